"""Waits of et_i8_gemm that run out: the call ends by itself, the status says so, nothing outside Y's rows is written, and
the same workspace serves the next call."""
import pytest
import torch

pytestmark = pytest.mark.gpu

# one CTA a tile; clusters of 4 and 8; pairs, one and several tiles each, few blocks of k and many; clusters of 2 and 4
# pairs; two passes of rows
FORMS = [(64, 4096, 1024), (64, 14336, 4096), (200, 1000, 2064), (40, 128, 65536), (1000, 4096, 4096), (2048, 6144, 512),
         (4096, 2048, 1024), (1024, 1024, 8192), (600, 1000, 16384), (8200, 1000, 144)]


def _case(E, M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    x, w = (torch.randint(-127, 128, (n, K), generator=g, device="cuda", dtype=torch.int8) for n in (M, N))
    sx, sw = torch.rand(M, generator=g, device="cuda") + 0.1, torch.rand(N, generator=g, device="cuda") + 0.1
    ws = E.alloc_workspace(E.et_i8_gemm_workspace_bytes(M, N, K))
    around = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")  # a row on either side

    def call(**how):
        E.et_i8_gemm(x, sx, w, sw, around[1:-1], workspace=ws, **how)
        status = E.et_status(ws)
        E.et_reset_status(ws)
        assert (around[0] == 7).all() and (around[-1] == 7).all()
        return status, around[1:-1].clone()
    return call


@pytest.mark.parametrize("M,N,K", FORMS)
@pytest.mark.parametrize("cta", [0, 1])
def test_weights_that_never_come(cuda_lib, M, N, K, cta):
    call = _case(cuda_lib, M, N, K)
    status, want = call()
    assert status == (0, 0)
    status, _ = call(timeout_us=20000, fault_mode=1, fault_arg=cta)
    assert status[0] == cuda_lib.ET_ERR_TIMEOUT
    status, got = call()
    assert status == (0, 0) and torch.equal(got, want)


@pytest.mark.parametrize("M,N,K", FORMS)
def test_a_limit_shorter_than_the_product(cuda_lib, M, N, K):
    """Each role gives up where it happens to be, with copies and products in flight."""
    call = _case(cuda_lib, M, N, K)
    status, want = call()
    assert status == (0, 0)
    for us in (1, 2, 5, 10, 20):
        for _ in range(3):
            status, got = call(timeout_us=us)
            assert status[0] in (0, cuda_lib.ET_ERR_TIMEOUT)
            assert status[0] or torch.equal(got, want)
    status, got = call(timeout_us=1000000)
    assert status == (0, 0) and torch.equal(got, want)
