"""et_i8_gemm behind other work of its stream: what is written right before the call is what it multiplies."""
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
