"""et_i8_gemm behind other work of its stream: what is written right before the call is what it multiplies, however long
that takes."""
import ctypes
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu


def _weights(N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(N, K, generator=g, device="cuda").bfloat16()


# one CTA a tile and clusters of them, pairs and clusters of pairs, more than one pass of rows, integer and fp16 MMAs
FORMS = [(1, 4096, 1024), (16, 1024, 4096), (64, 4096, 1024), (200, 1000, 2064), (300, 256, 14336), (1000, 4096, 4096), (2048, 6144, 512),
         (4096, 2048, 1024), (8200, 1000, 144)]


@pytest.mark.parametrize("M,N,K", FORMS)
def test_weights_quantised_right_before(cuda_lib, M, N, K):
    """Two sets of weights quantised into one buffer in turn, each multiplied right behind, with no wait of the host
    anywhere: the bits that a call gives whose weights were there long before."""
    E = cuda_lib
    raw = [_weights(N, K, s) for s in (1, 2)]
    xq, sx = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    ws = E.alloc_workspace(max(E.et_i8_gemm_workspace_bytes(M, N, K), E.et_i8_quantize_workspace_bytes(max(M, N), K)))
    E.et_i8_quantize(_weights(M, K, 3), xq, sx, workspace=ws)
    want = []
    for w in raw:
        q, s, Y = torch.empty(N, K, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda"), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        E.et_i8_quantize(w, q, s, workspace=ws)
        torch.cuda.synchronize()
        E.et_i8_gemm(xq, sx, q, s, Y, workspace=ws)
        torch.cuda.synchronize()
        want.append(Y)
    assert not torch.equal(*want)
    q, s = torch.zeros(N, K, dtype=torch.int8, device="cuda"), torch.zeros(N, device="cuda")
    got = [torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(20)]
    torch.cuda.synchronize()
    for i, Y in enumerate(got):
        E.et_i8_quantize(raw[i % 2], q, s, workspace=ws)
        E.et_i8_gemm(xq, sx, q, s, Y, workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(Y, want[i % 2]) for i, Y in enumerate(got))
    assert E.et_status(ws) == (0, 0)


LATE = r"""
#include <cuda_runtime.h>
// Lets the stream's next kernel be scheduled at once, then takes its time, then copies.
__global__ void late_copy_kernel(const char* from, char* to, size_t n, unsigned long long ns) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        unsigned long long t0, t;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
        for (int i = 0; i < 1000000; ++i) {
            asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
            if (t - t0 > ns) break;
            __nanosleep(1000);
        }
    }
    __syncthreads();
    for (size_t i = threadIdx.x; i < n; i += blockDim.x) to[i] = from[i];
}
extern "C" int late_copy(const void* from, void* to, size_t n, unsigned long long ns, void* stream) {
    late_copy_kernel<<<1, 1024, 0, static_cast<cudaStream_t>(stream)>>>(static_cast<const char*>(from), static_cast<char*>(to), n, ns);
    return cudaGetLastError();
}
"""


@pytest.fixture(scope="module")
def late_copy(tmp_path_factory):
    from moe_task_scheduling_gb300 import build
    d = tmp_path_factory.mktemp("late")
    (d / "late.cu").write_text(LATE)
    r = subprocess.run([build.nvcc(), *build.ARCH, "-O2", "-Xcompiler", "-fPIC", "-shared", "-o", str(d / "late.so"), str(d / "late.cu")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    f = ctypes.CDLL(str(d / "late.so")).late_copy
    f.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint64, ctypes.c_void_p]
    return f


@pytest.mark.parametrize("M,N,K", FORMS)
@pytest.mark.parametrize("device_count", [False, True])
def test_behind_a_kernel_that_outlasts_the_limit_of_a_wait(cuda_lib, late_copy, M, N, K, device_count):
    """A kernel that lets the product start early, goes on for longer (0.3 s) than a wait of the product may take (0.2 s),
    and writes the weights only then: the time is not the product's, no wait runs out and the result is whole."""
    E = cuda_lib
    xq, sx = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    q, s = torch.empty(N, K, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    ws = E.alloc_workspace(max(E.et_i8_gemm_workspace_bytes(M, N, K), E.et_i8_quantize_workspace_bytes(max(M, N), K)))
    E.et_i8_quantize(_weights(M, K, 4), xq, sx, workspace=ws)
    E.et_i8_quantize(_weights(N, K, 5), q, s, workspace=ws)
    how = dict(d_M=torch.full((1,), M, dtype=torch.int32, device="cuda")) if device_count else {}
    want, Y = (torch.zeros(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    E.et_i8_gemm(xq, sx, q, s, want, workspace=ws, **how)
    late = torch.zeros_like(q)
    torch.cuda.synchronize()
    n = q.numel() if q.numel() < 1 << 20 else 1 << 20  # one CTA copies: the first rows
    late.view(-1)[n:] = q.view(-1)[n:]
    torch.cuda.synchronize()
    assert late_copy(q.data_ptr(), late.data_ptr(), n, 300_000_000, torch.cuda.current_stream().cuda_stream) == 0
    E.et_i8_gemm(xq, sx, late, s, Y, workspace=ws, **how)
    torch.cuda.synchronize()
    assert E.et_status(ws) == (0, 0)
    assert torch.equal(Y, want)
