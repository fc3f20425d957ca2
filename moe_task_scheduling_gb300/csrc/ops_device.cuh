// ops_device.cuh -- device helpers shared by the router, norm and 4-bit weight
// kernels: warp and block sums in a fixed order, 16-byte asynchronous copies,
// the symbolic row count and the sticky status word.  None of these kernels
// waits on a flag or an mbarrier, so none of them needs a wait budget.
#pragma once

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

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two fp32 values as packed bf16, each rounded to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
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
