// ops_device.cuh -- device helpers shared by the router, norm, dropout, 4-bit and
// 8-bit weight kernels: warp and block sums in a fixed order, 16-byte asynchronous
// copies, the symbolic row count and the sticky status word.  Nothing here waits on
// a flag or an mbarrier.  (i8_gemm_kernel.cu does, and bounds its waits itself.)
#pragma once

#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "et_layout.h"

namespace et {

// Most of these kernels are launched with programmatic stream serialisation: one
// may be scheduled while the kernel before it in the stream drains, so it waits
// for that kernel's end (and its writes) before it touches global memory, then
// lets its own successor be scheduled.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_begin() {
    grid_wait();
    grid_release();
}

// Status details of these kernels (et_status), after the wait sites of et_layout.h.
constexpr int kWhereExpertIndex = 13;  // an expert index outside [-1, E)

// The first error of a workspace stays (et_status reads it).
__device__ __forceinline__ void record_status(EtHeader* hdr, int code, int detail) {
    if (atomicCAS(&hdr->status_code, 0, code) == 0) atomicExch(&hdr->status_detail, detail);
}

// The row count of this call: the host's, or the device's where it is given.
// A device count outside [0, max] is recorded and taken as "no rows"; the
// caller then returns without writing (ok == false).
__device__ __forceinline__ int row_count(const int32_t* d_n, int n_host, int n_max, EtHeader* hdr,
                                         bool* ok) {
    *ok = true;
    if (!d_n) return n_host;
    const int n = *d_n;
    if (n < 0 || n > n_max) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0)
            record_status(hdr, ET_ERR_BOUNDS, kWhereBoundsT);
        *ok = false;
        return 0;
    }
    return n;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Three sums over a warp, of which lane 0 has the first, 16 the second and 8 the third:
// half of the lanes go on with one of them each time, nine shuffles less than one by one.
__device__ __forceinline__ float warp_sum3(const float (&v)[3]) {
    const int lane = threadIdx.x & 31;
    const bool b16 = lane & 16, b8 = lane & 8;
    float s = (b16 ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, b16 ? v[0] : v[1], 16);
    const float c = v[2] + __shfl_xor_sync(0xffffffffu, v[2], 16);
    s = (b8 ? c : s) + __shfl_xor_sync(0xffffffffu, b8 ? s : c, 8);
#pragma unroll
    for (int off = 4; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    return s;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two fp32 values as packed bf16, each rounded to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Four int8 of a word as two pairs of fp16, exact: with the sign bits turned over a byte is
// x + 128, 0x6400 | b is 1024 + b in fp16, and 1152 less is x.
__device__ __forceinline__ void int8_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
    w ^= 0x80808080u;
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off), y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// 16 bytes global -> shared; bytes past `valid` (0 or 16 here) are filled with zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The first `bytes` (1 to 16) of 16, the rest zeros: nothing behind them is read.
__device__ __forceinline__ void cp_async16_part(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace et
