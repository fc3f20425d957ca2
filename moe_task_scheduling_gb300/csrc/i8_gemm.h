// i8_gemm.h -- the int8 product on the tensor cores: its shape of work, shared by
// the C entry points and the kernel.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "et_layout.h"

namespace et {

constexpr int kI8KBlock = 128;      // k of a block: one 128-byte row of weights
constexpr int kI8Sms = 152;         // CTAs of the persistent grid (pairs: half)
constexpr int kI8TokensMax = 256;   // tokens of a tile (UMMA N)
constexpr int kI8MaxStages = 12;    // of either ring

// The rows of one pass: [first, first + count) of a call's, the device's count where it is given.
struct I8Rows {
    const int32_t* d_M;
    int first, count, call_max;
};

struct I8TcArgs {
    const int8_t* x;     // [M, K] (a pair takes its tokens from the map of their fp16 form)
    const float* sx;     // [M]
    const float* sw;     // [N]
    bf16* y;             // [M, N]
    I8Rows rows;
    int N, K;
    EtHeader* hdr;
    int tn;              // tokens of a tile
    int nt;              // tiles over N
    int kblocks;
    int grid;            // CTAs, pairs or clusters that take tiles in turn (a cluster: one)
    int split;           // CTAs of a cluster that share a tile (1: none)
    int blocks;          // k-blocks that a CTA has in all, at most
    int stages_w, stages_x;
    uint64_t timeout_ns;
    int fault_cta;       // a test's: this CTA loads no weights, so that all that wait for them give up (-1: none)
};

struct I8ExpandArgs {
    const int8_t* x;     // [M, K]
    void* x16;           // fp16 [M, K]
    I8Rows rows;
    int K;
    EtHeader* hdr;
};

// `pair`: CTA pairs of 256 channels.  i8_tc_stages: stages of either ring, no more than there are
// blocks; returns the bytes of shared memory.
int i8_tc_stages(bool pair, int tn, int blocks, int* w, int* x);
cudaError_t launch_i8_tc(const I8TcArgs& a, const CUtensorMap* map_w, const CUtensorMap* map_x, bool pair, int dev, void* stream);
cudaError_t launch_i8_expand(const I8ExpandArgs& a, int sms, void* stream);

}  // namespace et
