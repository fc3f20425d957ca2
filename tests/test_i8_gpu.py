"""et_i8_quantize and et_i8_gemm on the GPU against exact integers and the 64-bit definition."""
import math

import pytest
import torch

from tests import ref_more as ref
from tests.ref_ops import F32_HALF as U
from tests.ref_ops import check

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _off(t, shift):
    b = torch.empty(t.numel() + 64, dtype=t.dtype, device="cuda")
    v = b[shift:shift + t.numel()].view(t.shape)
    v.copy_(t)
    return v


# ------------------------------------------------------------------ quantiser

def _quantize(E, x, shift=0, M=None, d_M=None, ws=None):
    Mm, K = x.shape
    ws = ws if ws is not None else E.alloc_workspace(E.et_i8_quantize_workspace_bytes(Mm, K))
    q, s = torch.full((Mm, K), 77, dtype=torch.int8, device="cuda"), torch.full((Mm,), 7.0, device="cuda")
    E.et_i8_quantize(_off(x, shift), q, s, M=M, d_M=d_M, workspace=ws)
    return q, s, ws


@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (17, 256), (9, 272), (40, 512), (5, 1008), (33, 4096), (2, 4112), (7, 14336), (3, 16384),
                                 (2, 16400), (3, 32768), (2, 65536), (1000, 64)])
def test_quantize(cuda_lib, M, K):
    x = (torch.randn(M, K, generator=_gen(M + K)) * torch.logspace(-6, 6, M)[:, None]).bfloat16()
    x[:, ::5] = (torch.randint(-254, 255, (M, (K + 4) // 5), generator=_gen(K)).float() / 2).bfloat16()  # halves: ties
    x[:, 0] = 127.0
    want_q, want_s = ref.i8_quantize(x)
    for shift in (0, 1):
        q, s, ws = _quantize(cuda_lib, x, shift)
        assert torch.equal(s.cpu(), want_s) and torch.equal(q.cpu(), want_q)
    assert cuda_lib.et_status(ws) == (0, 0)


def test_quantize_special_rows(cuda_lib):
    """Zeros of either sign, one value, infinities, NaN, the smallest and the largest numbers."""
    x = torch.randn(9, 64, generator=_gen(1)).bfloat16()
    x[0] = 0.0
    x[1] = -0.0
    x[2] = 0.0
    x[2, 63] = -3.0
    x[3, 5] = math.inf
    x[4, 60] = math.nan
    x[5] = x[5] * 2.0 ** -126
    x[6] = 0.0
    x[6, 1:4] = torch.tensor([9.2e-41, -9.2e-41, 4.6e-41]).bfloat16()
    x[7] = (x[7].float() / x[7].float().abs().max() * 3.3895e38).bfloat16()
    q, s, _ = _quantize(cuda_lib, x)
    want_q, want_s = ref.i8_quantize(x)
    assert torch.equal(q.cpu(), want_q)
    assert torch.equal(torch.isnan(s.cpu()), torch.isnan(want_s)) and torch.isnan(s[3]) and torch.isnan(s[4])
    fin = torch.isfinite(want_s)
    assert torch.equal(s.cpu()[fin], want_s[fin])


# ------------------------------------------------------------------ products

def _random(M, N, K, seed, full=False):
    g = _gen(seed)
    lo = -128 if full else -127
    return (torch.randint(lo, 128, (M, K), generator=g).to(torch.int8), torch.rand(M, generator=g) * 0.02 + 1e-3,
            torch.randint(lo, 128, (N, K), generator=g).to(torch.int8), torch.rand(N, generator=g) * 0.01 + 1e-4)


def _gemm(E, xq, sx, wq, sw, M=None, d_M=None, ws=None, y_shift=0):
    Mm, K = xq.shape
    N = wq.shape[0]
    ws = ws if ws is not None else E.alloc_workspace(E.et_i8_gemm_workspace_bytes(Mm, N, K))
    Y = _off(torch.full((Mm, N), 7.0, dtype=torch.bfloat16), y_shift)
    E.et_i8_gemm(xq.cuda(), sx.cuda(), wq.cuda(), sw.cuda(), Y, M=M, d_M=d_M, workspace=ws)
    return Y, ws


def _check(Y, xq, sx, wq, sw, M=None):
    M = xq.shape[0] if M is None else M
    y, e = ref.i8_gemm(xq[:M], sx[:M], wq, sw)
    check(Y[:M], y, ref.bf16_bound(y, e), "Y")
    assert (Y[M:] == 7).all()


GEMM = [(1, 1, 16), (1, 8, 32), (1, 4096, 14336), (2, 5, 48), (2, 1000, 1024), (3, 130, 2064), (4, 127, 144), (5, 129, 4096), (7, 333, 528),
        (8, 128, 128), (8, 2000, 4096), (9, 64, 112), (12, 700, 2048), (16, 128, 1024), (16, 1024, 4096), (17, 257, 272), (31, 500, 768),
        (32, 384, 2064), (33, 1000, 144), (48, 96, 16384), (64, 512, 4096), (65, 130, 400), (100, 1000, 2048), (127, 129, 1040),
        (128, 256, 512), (129, 384, 640), (200, 1000, 2064), (255, 300, 256), (256, 1024, 1024), (257, 257, 272), (300, 2000, 528),
        (512, 512, 2048), (777, 1111, 1008), (1000, 136, 4096), (1500, 2048, 512), (2049, 770, 784), (2500, 2050, 272), (1111, 5000, 528), (4800, 2048, 80), (600, 6500, 1040), (8200, 1000, 144)]


@pytest.mark.parametrize("M,N,K", GEMM)
def test_gemm(cuda_lib, M, N, K):
    a = _random(M, N, K, M + N + K, full=True)
    Y, ws = _gemm(cuda_lib, *a)
    _check(Y, *a)
    Y2, _ = _gemm(cuda_lib, *a, ws=ws, y_shift=1)  # the same bits again, from the same workspace, to an odd address
    assert torch.equal(Y, Y2)
    assert cuda_lib.et_status(ws) == (0, 0)


@pytest.mark.parametrize("M", [1, 3, 8, 20, 64, 130, 300, 600])
def test_gemm_is_exact_to_the_integer(cuda_lib, M):
    """Sums below 2^8 with scales of 1 are bf16 integers: the result has to be the integer itself.  One lost or doubled
    16-byte piece of any row would show."""
    N, K = 390, 1936
    g = _gen(M)
    xq, wq = torch.zeros(M, K, dtype=torch.int8), torch.zeros(N, K, dtype=torch.int8)
    for r in range(K // 16):  # one nonzero in each 16-byte piece of a row
        xq[torch.arange(M), r * 16 + torch.randint(0, 16, (M,), generator=g)] = 1
    wq[:] = torch.randint(-2, 3, (N, K), generator=g).to(torch.int8)
    y = xq.double() @ wq.double().t()
    assert float(y.abs().max()) <= 256
    Y, _ = _gemm(cuda_lib, xq, torch.ones(M), wq, torch.ones(N))
    assert torch.equal(Y.cpu().double(), y)
    Y, _ = _gemm(cuda_lib, torch.full((M, K), -1, dtype=torch.int8), torch.ones(M), torch.ones(N, K, dtype=torch.int8), torch.ones(N))
    assert torch.equal(Y.cpu().double(), torch.full((M, N), -float(K)).bfloat16().double())


@pytest.mark.parametrize("M", [1, 5, 16, 100, 300])
def test_gemm_extreme_values(cuda_lib, M):
    """Every value of int8 against every other, the largest sums, scales of 0, NaN, infinity and the smallest numbers."""
    N, K = 256, 65536
    xq = torch.full((M, K), -128, dtype=torch.int8)
    wq = (torch.arange(N)[:, None] - 128).to(torch.int8).expand(N, K).contiguous()
    sx, sw = torch.ones(M), torch.ones(N)
    Y, _ = _gemm(cuda_lib, xq, sx, wq, sw)
    _check(Y, xq, sx, wq, sw)
    x2 = (torch.arange(M)[:, None] * 37 % 256 - 128).to(torch.int8).expand(M, 32).contiguous()
    w2 = wq[:, :32].contiguous()
    sw[3], sw[4], sw[5], sw[6] = 0.0, math.nan, math.inf, 1e-40
    sx[0] = 0.0
    Y, _ = _gemm(cuda_lib, x2, sx, w2, sw)
    y = (x2.double() @ w2.double().t()) * (sx.double()[:, None] * sw.double())
    fin = torch.isfinite(y)
    assert torch.equal(torch.isfinite(Y.cpu()), fin)
    check(torch.where(fin, Y.cpu().double(), 0.0), torch.where(fin, y, 0.0), ref.bf16_bound(torch.where(fin, y, 0.0), 2.0 ** -22 * torch.where(fin, y, 0.0).abs()) + 2.0 ** -130, "Y")


@pytest.mark.parametrize("Mm,N,K", [(8, 300, 512), (64, 500, 1040), (700, 260, 512)])
def test_device_count(cuda_lib, Mm, N, K):
    """One launch for every count: rows behind it stay; a count out of range is recorded and nothing is written."""
    a = _random(Mm, N, K, Mm)
    dM = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = cuda_lib.alloc_workspace(cuda_lib.et_i8_gemm_workspace_bytes(Mm, N, K))
    x = torch.randn(Mm, K, generator=_gen(3)).bfloat16()
    wantq, wants = ref.i8_quantize(x)
    for M in (Mm, 1, 0, Mm // 2 + 1):
        dM.fill_(M)
        for how in (dict(d_M=dM), dict(M=M)):
            Y, _ = _gemm(cuda_lib, *a, ws=ws, **how)
            if M:
                _check(Y, *a, M=M)
            else:
                assert (Y == 7).all()
            q, s, _ = _quantize(cuda_lib, x, ws=ws, **how)
            assert torch.equal(q[:M].cpu(), wantq[:M]) and torch.equal(s[:M].cpu(), wants[:M])
            assert (q[M:] == 77).all() and (s[M:] == 7).all()
    for M in (Mm + 1, -1):
        dM.fill_(M)
        Y, _ = _gemm(cuda_lib, *a, ws=ws, d_M=dM)
        assert (Y == 7).all() and cuda_lib.et_status(ws)[0] == cuda_lib.ET_ERR_BOUNDS
        cuda_lib.et_reset_status(ws)
        q, s, _ = _quantize(cuda_lib, x, ws=ws, d_M=dM)
        assert (q == 77).all() and (s == 7).all() and cuda_lib.et_status(ws)[0] == cuda_lib.ET_ERR_BOUNDS
        cuda_lib.et_reset_status(ws)
        Y, _ = _gemm(cuda_lib, *a, ws=ws)  # and the workspace serves the next call
        _check(Y, *a)


def test_shapes_in_turn_share_a_workspace(cuda_lib):
    """Calls of other shapes one after the other, with one workspace of the largest's size."""
    shapes = [(300, 500, 2064), (5, 129, 4096), (64, 1000, 1024), (1, 64, 16384), (700, 130, 272), (16, 384, 4096)]
    ws = cuda_lib.alloc_workspace(max(cuda_lib.et_i8_gemm_workspace_bytes(*s) for s in shapes))
    args = [_random(*s, i) for i, s in enumerate(shapes)]
    first = [_gemm(cuda_lib, *a, ws=ws)[0] for a in args]
    for a, f in zip(args, first):
        _check(f, *a)
    for i in (5, 0, 3, 1, 4, 2):
        assert torch.equal(_gemm(cuda_lib, *args[i], ws=ws)[0], first[i])


def test_quantised_linear(cuda_lib):
    """bf16 tokens and weights through both calls: within what the two quantisations can lose."""
    M, N, K = 50, 300, 1024
    g = _gen(9)
    x, w = torch.randn(M, K, generator=g).bfloat16(), (torch.randn(N, K, generator=g) / 32).bfloat16()
    xq, sx, ws = _quantize(cuda_lib, x)
    wq, sw, _ = _quantize(cuda_lib, w)
    Y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    ws = cuda_lib.alloc_workspace(cuda_lib.et_i8_gemm_workspace_bytes(M, N, K))
    cuda_lib.et_i8_gemm(xq, sx, wq, sw, Y, workspace=ws)
    want = x.double() @ w.double().t()
    ex, ew = sx.double().cpu()[:, None] * 0.5001, sw.double().cpu()[:, None] * 0.5001  # half a step of each value
    lost = ex * w.double().abs().sum(-1) + x.double().abs().sum(-1)[:, None] * ew.t() + ex * ew.t() * K
    check(Y, want, ref.bf16_bound(want, lost), "Y")


@pytest.mark.parametrize("M,N,K", [(3, 200, 65536), (12, 200, 65536), (40, 256, 65536), (64, 20000, 65536), (300, 256, 14336), (1000, 4096, 14336)])
@pytest.mark.parametrize("low", [1, 100])
def test_gemm_sums_that_rise_and_fall(cuda_lib, M, N, K, low):
    """Products of one sign for half of k, then of the other: partial sums up to 2^30 whose result is small, where every
    bit that a partial sum loses shows.  Up to 8 tokens nothing is lost."""
    g = torch.Generator(device="cuda").manual_seed(M + K)
    x = torch.randint(low, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(low, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    x[:, K // 2:] = -x[:, :K // 2]
    w[:, K // 2:] = w[:, :K // 2]
    x[:, 0] = 3
    y = x.double() @ w.double().t()
    Y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    ws = cuda_lib.alloc_workspace(cuda_lib.et_i8_gemm_workspace_bytes(M, N, K))
    cuda_lib.et_i8_gemm(x, torch.ones(M, device="cuda"), w, torch.ones(N, device="cuda"), Y, workspace=ws)
    # (its bound is written at ref.i8_gemm; the sums of |x w| are taken on the device, exact in 64 bits)
    e = 0.0 if M <= 8 else K * 2.0 ** -27 * (x.double().abs() @ w.double().t())
    check(Y, y.cpu(), ref.bf16_bound(y, e + 4 * U * y.abs()).cpu(), "Y")
