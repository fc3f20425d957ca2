// et_api.h -- host-side helpers shared by the translation units that hold C
// entry points: the thread's error string, the current device, workspace checks.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

#include <string>
#include <utility>

#include "et_layout.h"

namespace et {

constexpr int kApiMaxDevices = 64;

// Defined in etmoe_api.cu.
void api_clear_error();
int api_fail(int code, const std::string& msg);
int api_fail_cuda(cudaError_t e, const char* what);
int api_device(int* dev, int* sms);  // current device (sm_103a checked) and its SM count
int api_check_ws(const void* ws, size_t have, size_t need);
uint64_t api_timeout_ns(const et_opts* opts);  // of a bounded wait
// Row-major [rows, cols] of 1-byte integers or fp16 as boxes of 128 bytes x box_rows with
// the 128-byte swizzle; zeros outside.  (api_device has been called.)
int api_map128(CUtensorMap* m, const void* base, int elem_bytes, uint64_t rows, uint64_t cols, uint32_t box_rows, const char* what);

inline bool api_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Runs a C entry point's body: clears the thread's error string first, and no
// C++ exception (an error message that cannot be allocated) leaves the call.
template <class F>
int api_entry(F&& body) noexcept {
    try {
        api_clear_error();
        return body();
    } catch (...) {
        return ET_ERR_CUDA;
    }
}

// One-time cudaFuncSetAttribute(MaxDynamicSharedMemorySize) of a kernel on each
// device; two threads that meet here both set the same value.
struct SmemOptIn {
    bool done[kApiMaxDevices] = {};
};
template <class K>
cudaError_t api_smem_opt_in(SmemOptIn& st, int dev, K kernel, int bytes) {
    if (__atomic_load_n(&st.done[dev], __ATOMIC_ACQUIRE)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) __atomic_store_n(&st.done[dev], true, __ATOMIC_RELEASE);
    return e;
}

// N numbers that queries of the runtime give for a kernel, kept for each device:
// another device may have other SMs and other places for clusters.  A query that
// fails is not kept, its error goes to the caller.
template <int N>
struct DeviceNumbers {
    int kept[kApiMaxDevices][N] = {};  // the number + 1; 0: not asked yet
    template <class Q>
    cudaError_t get(int dev, int at, int* value, Q&& query) {
        const int k = __atomic_load_n(&kept[dev][at], __ATOMIC_RELAXED);
        if (k) {
            *value = k - 1;
            return cudaSuccess;
        }
        *value = 0;
        const cudaError_t e = query(value);
        if (e == cudaSuccess) __atomic_store_n(&kept[dev][at], *value + 1, __ATOMIC_RELAXED);
        return e;
    }
};

// One launch; cluster: CTAs a cluster; early: it may be scheduled while the
// kernel before it drains (its kernel then waits, see grid_wait in ops_device.cuh).
// The error is this launch's own (cudaGetLastError could return an older one of
// the calling program).
template <class... P, class... A>
cudaError_t api_launch_cluster(void (*kernel)(P...), dim3 grid, dim3 block, int cluster, bool early, size_t smem,
                               void* stream, A&&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = early ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

template <class... P, class... A>
cudaError_t api_launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, void* stream, A&&... args) {
    return api_launch_cluster(kernel, grid, block, 1, true, smem, stream, std::forward<A>(args)...);
}

}  // namespace et
