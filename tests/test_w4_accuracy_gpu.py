"""The 4-bit products on the GPU where a loose bound would hide a fault: inputs whose result is exact, and inputs
far larger than the others whose weights are zero."""
import pytest
import torch

from tests import ref_ops as ref
from tests import ref_w4
from tests.test_w4_gpu import _cuda, _experts, _experts_inputs, _gemv, _gen

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _exact_weight(N, K, group, seed):
    """Every 4-bit value, scales 1/4, 1/2 and 1."""
    g = _gen(seed)
    q = torch.randint(0, 256, (N, K // 2), generator=g).to(torch.uint8)
    s = (2.0 ** torch.randint(-2, 1, (K // group, N), generator=g)).to(BF)
    return q, s


@pytest.mark.parametrize("N,K", [(200, 256), (4096, 512), (256, 2048), (2120, 7168)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_gemv_of_integers(cuda_lib, N, K, group):
    """Integers up to 8: every product and sum is a multiple of 1/4 below 7168 * 64 = 2^18.9, so fp32 holds each
    exactly and only the output's rounding is left.  Then some inputs of weight zero (q = 8) are made as large as
    2^120: they add nothing."""
    q, s = _exact_weight(N, K, group, N + K)
    at = [0, 5, K // 2 + 1, K - 1]
    for c in at:
        q[:, c // 2] = (q[:, c // 2] & 0xf0 | 8) if c % 2 == 0 else (q[:, c // 2] & 0x0f | 0x80)
    qc, sc = _cuda(q, s)
    w = ref.w4_values(q, s)
    for M in (1, 3, 8, 16, 33, 64):
        x = torch.randint(-8, 9, (M, K), generator=_gen(M)).to(BF)
        want = (x.double() @ w.t()).to(BF)
        y, ws = _gemv(cuda_lib, x.cuda(), qc, sc)
        assert torch.equal(y.cpu(), want)
        for row in range(M):
            for i, c in enumerate(at):
                x[row, c] = (-1.0) ** (row + i) * 2.0 ** (10, 14, 20, 120)[(row + i) % 4]
        assert torch.equal(_gemv(cuda_lib, x.cuda(), qc, sc, ws=ws)[0].cpu(), want)


@pytest.mark.parametrize("T,H,F,En,k,group", [(1, 256, 512, 8, 2, 128), (7, 2048, 768, 16, 8, 128), (40, 192, 320, 3, 2, 64),
                                              (64, 416, 288, 256, 8, 32), (64, 128, 1600, 128, 8, 64), (33, 4096, 320, 6, 2, 64)])
def test_experts_large_inputs_of_zero_weights(cuda_lib, T, H, F, En, k, group):
    """One input of every token, and one of every down product, is thousands of times the others, and no weight
    takes it in: the same bits as with zeros in their places."""
    x, idx, w, gate, up, down = _experts_inputs(T, H, F, En, k, group, T + H)
    c, f = H // 2 + 1, F // 2 + 1  # odd: the high half of a byte
    for q, at in ((gate[0], c), (up[0], c), (down[0], f)):
        q[:, :, at // 2] = q[:, :, at // 2] & 0x0f | 0x80
    for s in (gate[1], up[1]):  # h[f] of some thousands
        s[:, :, f] *= 256
    zero_up = (up[0], up[1].clone())
    zero_up[1][:, :, f] = 0
    x[:, c] = 0
    want, ws = _experts(cuda_lib, x, idx, w, gate, zero_up, down)
    x[:, c] = (2.0 ** (10 + torch.arange(T) % 12)).to(BF)
    got, _ = _experts(cuda_lib, x, idx, w, gate, up, down, ws=ws)
    assert torch.isfinite(want).all() and float(want.abs().max()) > 0
    assert torch.equal(got, want)


@pytest.mark.parametrize("T,H,F,En,k,group", ref_w4.SIZES)
def test_experts_of_exact_products(cuda_lib, T, H, F, En, k, group):
    """Gate and up products are exact here, which leaves a bound small enough to show one lost row or 32 lost inputs."""
    a = ref_w4.inputs(T, H, F, En, k, group, T + H)
    out, ws = _experts(cuda_lib, *a)
    want, bound = ref_w4.experts(*a)
    ref.check(out, want, ref_w4.tolerance(want, bound), "out")
    assert torch.equal(out, _experts(cuda_lib, *a, ws=ws)[0])
    assert cuda_lib.et_status(ws) == (0, 0)
