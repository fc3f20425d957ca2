// row_ops.cuh -- rows of up to 16384 bf16 held by the threads of a warp, of a
// group or of a CTA: how columns fall to threads, loads, stores and row sums.
// Shared by the norm kernels.
#pragma once

#include <initializer_list>

#include "et_api.h"
#include "ops_device.cuh"

namespace et {
namespace {

constexpr int kNormHMax = 16384;

// Eight consecutive bf16 of a row, packed.
struct Vec8 {
    uint32_t u[4];
    __device__ __forceinline__ float operator[](int i) const {
        return (i & 1) ? bf_hi(u[i >> 1]) : bf_lo(u[i >> 1]);
    }
};

// The threads of a row, and how its columns fall to them.  A CTA holds one row, or
// several with a group of threads (a multiple of a warp) each.  A thread has
// sixteen columns in two vectors of eight.  VEC (H a multiple of 8, tensors
// 16-byte aligned): eight neighbours, one 16-byte access; else columns a group
// apart, so that neighbouring threads still read neighbouring elements.
enum RowMode { kRowsWarp = 0, kRowsGroup = 1, kRowsOne = 2 };  // a row a warp (eight columns a thread
                                                               // are enough), a group, a CTA
template <int MODE>
struct RowGroup {
    int threads, group;  // kRowsGroup only

    __device__ __forceinline__ explicit RowGroup(int row_threads) {
        if (MODE == kRowsGroup) {
            threads = row_threads;
            group = threadIdx.x / row_threads;
        }
    }
    __device__ __forceinline__ int th() const {  // threads of a row
        return MODE == kRowsWarp ? 32 : MODE == kRowsOne ? static_cast<int>(blockDim.x) : threads;
    }
    __device__ __forceinline__ int groups() const {  // rows of the CTA
        return MODE == kRowsOne ? 1 : MODE == kRowsWarp ? static_cast<int>(blockDim.x >> 5) : static_cast<int>(blockDim.x) / threads;
    }
    __device__ __forceinline__ int id() const {  // this thread's row of the CTA,
        return MODE == kRowsOne ? 0 : MODE == kRowsWarp ? static_cast<int>(threadIdx.x >> 5) : group;
    }
    __device__ __forceinline__ int lane() const {  // and its place in it
        return MODE == kRowsOne ? static_cast<int>(threadIdx.x)
             : MODE == kRowsWarp ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x) - group * threads;
    }
    template <bool VEC>
    __device__ __forceinline__ int col(int j, int i) const {
        return VEC ? (j * th() + lane()) * 8 + i : (j * 8 + i) * th() + lane();
    }
    __device__ __forceinline__ void sync() const {
        if (MODE == kRowsOne) __syncthreads();
        else if (MODE == kRowsWarp) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(threads) : "memory");
    }
};

constexpr int kNormCtaThreads = 256;  // of a CTA that holds several rows
__host__ __device__ constexpr int norm_v(int mode) { return mode == kRowsWarp ? 1 : 2; }  // vectors of a thread

// This thread's vector j of a row of H columns; zeros past its end.
template <bool VEC, int MODE>
__device__ __forceinline__ Vec8 load8(const bf16* row, const RowGroup<MODE>& g, int j, int H) {
    Vec8 v{};
    if (VEC) {
        const int c = g.template col<VEC>(j, 0);
        if (c < H) {
            const uint4 q = *reinterpret_cast<const uint4*>(row + c);
            v.u[0] = q.x; v.u[1] = q.y; v.u[2] = q.z; v.u[3] = q.w;
        }
    } else {
        const uint16_t* r = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = g.template col<VEC>(j, i);
            if (c < H) v.u[i >> 1] |= static_cast<uint32_t>(r[c]) << (16 * (i & 1));
        }
    }
    return v;
}

template <bool VEC, int MODE>
__device__ __forceinline__ void store8(bf16* row, const RowGroup<MODE>& g, int j, int H, const float* f) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
    if (VEC) {
        const int c = g.template col<VEC>(j, 0);
        if (c < H) *reinterpret_cast<uint4*>(row + c) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
        uint16_t* r = reinterpret_cast<uint16_t*>(row);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = g.template col<VEC>(j, i);
            if (c < H) r[c] = static_cast<uint16_t>(u[i >> 1] >> (16 * (i & 1)));
        }
    }
}

// One or two sums over the row's threads, the same bits in every one of them.
// Consecutive sums alternate between two slots of `red` (n counts them), so one
// barrier a sum is enough: who has passed the next sum's barrier knows that all
// have read this one.
template <int MODE>
__device__ __forceinline__ float row_sum(float v, float (*red)[32], const RowGroup<MODE>& g, int& n) {
    v = warp_sum(v);
    if (MODE != kRowsWarp) {
        const int slot = n++ & 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int first = g.id() * (g.th() >> 5);
        if (lane == 0) red[slot][warp] = v;
        g.sync();
        v = warp_sum(lane < (g.th() >> 5) ? red[slot][first + lane] : 0.0f);
    }
    return v;
}
template <int MODE>
__device__ __forceinline__ float2 row_sum2(float2 v, float (*red)[32], float (*red2)[32], const RowGroup<MODE>& g, int& n) {
    v.x = warp_sum(v.x);
    v.y = warp_sum(v.y);
    if (MODE != kRowsWarp) {
        const int slot = n++ & 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int first = g.id() * (g.th() >> 5);
        if (lane == 0) { red[slot][warp] = v.x; red2[slot][warp] = v.y; }
        g.sync();
        const bool in = lane < (g.th() >> 5);
        v.x = warp_sum(in ? red[slot][first + lane] : 0.0f);
        v.y = warp_sum(in ? red2[slot][first + lane] : 0.0f);
    }
    return v;
}

__device__ __forceinline__ float2 unpack2(uint32_t w) { return make_float2(bf_lo(w), bf_hi(w)); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Bytes of a staged row: without VEC it starts anywhere in its first 16-byte piece.
__host__ __device__ constexpr int norm_row_bytes(int H, bool vec) { return vec ? H * 2 : (H * 2 + 29) / 16 * 16; }

// 16-byte accesses: H a multiple of 8 and every bf16 tensor 16-byte aligned.
bool norm_vec(int H, std::initializer_list<const void*> ps) {
    if (H % 8) return false;
    for (const void* q : ps)
        if (!api_aligned(q, 16)) return false;
    return true;
}

// Threads of a row: sixteen columns each.
int norm_threads(int H) { return ((H + 15) / 16 + 31) / 32 * 32; }

// Rows of a CTA: as many as make 256 threads.  With fewer, a small H left most of
// an SM idle (forward and backward, T = 4096, H = 512: 62 us, with eight rows 20).
int norm_groups(int threads, int rows) {
    const int g = threads < kNormCtaThreads ? kNormCtaThreads / threads : 1;
    return g < rows ? g : rows;
}

RowMode norm_mode(int H, int threads) {
    return H <= 256 ? kRowsWarp : 2 * threads <= kNormCtaThreads ? kRowsGroup : kRowsOne;
}

}  // namespace
}  // namespace et
