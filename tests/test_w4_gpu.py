"""The 4-bit weight calls on the GPU against the 64-bit definitions."""
import math

import pytest
import torch

from tests import ref_ops as ref

pytestmark = pytest.mark.gpu
U, B = ref.F32_HALF, ref.BF16_HALF
BF = torch.bfloat16


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _weight(shape, group, seed, std=None):
    K = shape[-1]
    w = (torch.randn(*shape, generator=_gen(seed)) * (std or 1 / math.sqrt(K))).to(BF)
    return ref.w4_pack(w, group)


def _cuda(*ts):
    return [t.cuda() for t in ts]


def _gemv(E, x, q, s, M=None, d_M=None, ws=None, stream=None):
    N = q.shape[0]
    y = torch.full((x.shape[0], N), 7.0, dtype=BF, device="cuda")
    ws = ws if ws is not None else E.alloc_workspace(E.et_w4_gemv_workspace_bytes(x.shape[0], N, x.shape[1], x.shape[1] // s.shape[0]))
    E.et_w4_gemv(x, q, s, y, M=M, d_M=d_M, workspace=ws, stream=stream)
    return y, ws


def _check_gemv(y, x, q, s, rows=None):
    rows = x.shape[0] if rows is None else rows
    want, mag = ref.gemv(x[:rows].cpu(), q.cpu(), s.cpu())
    # one rounding of the output; products are exact, and each of the K + K / group additions (in the tensor
    # core: at worst truncated, two half steps) is off by its partial sum's step
    ref.check(y[:rows], want, B * want.abs() + (2 * x.shape[1] + 16) * U * mag + 1e-38, "y")
    assert (y[rows:] == 7).all()


SIZES = [(8, 32), (8, 128), (64, 96), (72, 160), (200, 256), (256, 1024), (1000, 2048), (4096, 512), (48, 14336), (2056, 1120)]


@pytest.mark.parametrize("N,K", SIZES)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_gemv(cuda_lib, N, K, group):
    if K % group:
        K = (K // group + 1) * group
    q, s = _weight((N, K), group, N + K)
    qc, sc = _cuda(q, s)
    for M in (1, 2, 3, 8, 9, 16, 17, 33, 64):
        x = torch.randn(M, K, generator=_gen(M)).to(BF).cuda()
        y, ws = _gemv(cuda_lib, x, qc, sc)
        _check_gemv(y, x, q, s)
        assert torch.equal(y, _gemv(cuda_lib, x, qc, sc, ws=ws)[0])  # the same bits again
        # every row is the row it is alone within a bound, and exactly what a zero x gives
    x = torch.zeros(5, K, dtype=BF, device="cuda")
    assert (_gemv(cuda_lib, x, qc, sc)[0] == 0).all()


@pytest.mark.parametrize("M,N,K,group", [(16, 6144, 4096, 64), (11, 6144, 4096, 128), (33, 2120, 7168, 32), (64, 2120, 7168, 128),
                                         (50, 3000, 8192, 64)])
def test_gemv_many_rows_of_large_weights(cuda_lib, M, N, K, group):
    """Passes of sixteen rows, the last of them ragged."""
    q, s = _weight((N, K), group, N + M)
    qc, sc = _cuda(q, s)
    x = torch.randn(M, K, generator=_gen(M)).to(BF).cuda()
    y, ws = _gemv(cuda_lib, x, qc, sc)
    _check_gemv(y, x, q, s)
    assert torch.equal(y, _gemv(cuda_lib, x, qc, sc, ws=ws)[0])
    y, _ = _gemv(cuda_lib, x, qc, sc, d_M=torch.full((1,), M - 5, dtype=torch.int32, device="cuda"), ws=ws)
    _check_gemv(y, x, q, s, M - 5)


@pytest.mark.parametrize("T,H,F,En,k,group", [(64, 4096, 128, 4, 1, 128), (33, 4096, 320, 6, 2, 64), (64, 4128, 96, 2, 2, 32)])
def test_experts_with_many_rows_and_long_sums(cuda_lib, T, H, F, En, k, group):
    """Experts with more rows than a pass of sixteen takes, and with fewer."""
    a = _experts_inputs(T, H, F, En, k, group, T + H)
    out, ws = _experts(cuda_lib, *a)
    _check_experts(out, *a)
    dT = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    out, _ = _experts(cuda_lib, *a, d_T=dT, ws=ws)
    _check_experts(out, *a, T=9)
    assert cuda_lib.et_status(ws) == (0, 0)


@pytest.mark.parametrize("T,H,F,En,k,group", [(64, 416, 288, 256, 8, 32), (63, 448, 320, 250, 8, 64), (40, 1024, 128, 128, 8, 128),
                                              (64, 64, 1568, 200, 8, 32), (64, 128, 1600, 128, 8, 64), (50, 128, 3200, 60, 8, 128)])
def test_experts_of_many_units(cuda_lib, T, H, F, En, k, group):
    """So many (tile, rows of an expert) that a warp takes each alone: in both products, or in one of them; with
    experts left out, named twice and out of range, and fewer tokens by the device count."""
    x, idx, w, gate, up, down = _experts_inputs(T, H, F, En, k, group, T + H)
    idx[0] = -1
    idx[1, 3:] = idx[1, 0]
    idx[5, 2], w[5, 2] = -1, math.nan
    idx[6, 1], idx[7, 0] = En, -7
    seen = torch.where((idx >= 0) & (idx < En), idx, -1)
    out, ws = _experts(cuda_lib, x, idx, w, gate, up, down)
    assert (out[0] == 0).all()
    _check_experts(out, x, seen, w, gate, up, down)
    assert torch.equal(out, _experts(cuda_lib, x, idx, w, gate, up, down, ws=ws)[0])
    assert cuda_lib.et_status(ws)[0] == cuda_lib.ET_ERR_BOUNDS
    cuda_lib.et_reset_status(ws)
    dT = torch.zeros(1, dtype=torch.int32, device="cuda")
    for n in (5, 0, T + 1):
        dT.fill_(n)
        out, _ = _experts(cuda_lib, x, idx, w, gate, up, down, d_T=dT, ws=ws)
        if n <= T:
            _check_experts(out, x, seen, w, gate, up, down, T=n)
            assert cuda_lib.et_status(ws) == (0, 0)
        else:
            assert (out == 7).all() and cuda_lib.et_status(ws)[0] == cuda_lib.ET_ERR_BOUNDS


def test_gemv_device_count(cuda_lib):
    N, K = 264, 640
    q, s = _weight((N, K), 64, 1)
    qc, sc = _cuda(q, s)
    x = torch.randn(40, K, generator=_gen(2)).to(BF).cuda()
    dM = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = cuda_lib.alloc_workspace(256)
    for M in (40, 1, 0, 33):
        dM.fill_(M)
        y, _ = _gemv(cuda_lib, x, qc, sc, d_M=dM, ws=ws)
        _check_gemv(y, x, q, s, rows=M)
        y, _ = _gemv(cuda_lib, x, qc, sc, M=M, ws=ws)
        _check_gemv(y, x, q, s, rows=M)
    for M in (41, -1):
        dM.fill_(M)
        y, _ = _gemv(cuda_lib, x, qc, sc, d_M=dM, ws=ws)
        assert (y == 7).all() and cuda_lib.et_status(ws)[0] == cuda_lib.ET_ERR_BOUNDS
        cuda_lib.et_reset_status(ws)


def test_gemv_special_values(cuda_lib):
    """Negative and zero scales, a NaN scale in one row, an infinity in one row of x: only those outputs show it."""
    N, K = 64, 256
    q, s = _weight((N, K), 64, 3)
    s[1] = -s[1]
    s[2] = 0
    s[0, 5] = math.nan
    x = torch.randn(4, K, generator=_gen(4)).to(BF)
    x[2, 200] = math.inf
    q[:, 100] = 0xff - (q[:, 100] & 0x77)  # no zero weight meets the infinity's column in another order
    y, _ = _gemv(cuda_lib, x.cuda(), q.cuda(), s.cuda())
    y = y.float().cpu()
    assert torch.isnan(y[:, 5]).all()
    assert not torch.isfinite(y[2]).any()
    keep = [c for c in range(N) if c != 5]
    xs = x[[0, 1, 3]]
    want, mag = ref.gemv(xs, q[keep], s[:, keep])
    ref.check(y[[0, 1, 3]][:, keep], want, B * want.abs() + (2 * K + 16) * U * mag, "y")


# ------------------------------------------------------------------ conversion

@pytest.mark.parametrize("shape,group", [((8, 32), 32), ((1000, 2048), 32), ((72, 320), 64), ((3, 136, 384), 128), ((5, 8, 64), 32), ((2, 2048, 4096), 128)])
def test_quantize(cuda_lib, shape, group):
    w = (torch.randn(*shape, generator=_gen(5)) * 0.02).to(BF)
    w.view(-1)[:32] = 0                                    # a group of zeros
    w.view(-1, 32)[-1] = torch.arange(-16, 16).to(BF) / 2  # ties
    q, s = ref.w4_pack(w, group)
    qc = torch.full_like(q, 0xAA, device="cuda")
    sc = torch.full_like(s, 7.0, device="cuda")
    cuda_lib.et_w4_quantize(w.cuda(), qc, sc)
    assert torch.equal(qc.cpu(), q) and torch.equal(sc.cpu(), s)
    back = torch.empty(shape, dtype=BF, device="cuda")
    cuda_lib.et_w4_dequantize(qc, sc, back)
    want = ref.w4_values(q, s, torch.float32).to(BF)
    assert torch.equal(back.cpu(), want)


def test_quantize_special_values(cuda_lib):
    w = torch.randn(16, 128, generator=_gen(6)).to(BF)
    w[1, 40], w[2, 0], w[3, 127] = math.inf, math.nan, -math.inf
    w[4, :32] = torch.finfo(BF).max
    w[5, :32] = 9.2e-41  # the smallest subnormal: its seventh rounds to zero
    w[6, :32] = 4e-39    # subnormal with a scale
    q, s = ref.w4_pack(w, 32)
    qc, sc = torch.empty_like(q, device="cuda"), torch.empty_like(s, device="cuda")
    cuda_lib.et_w4_quantize(w.cuda(), qc, sc)
    assert torch.equal(qc.cpu(), q)
    assert torch.equal(torch.isnan(sc.cpu()), torch.isnan(s)) and torch.equal(sc.cpu().nan_to_num(1.0), s.nan_to_num(1.0))
    assert int(torch.isnan(s).sum()) == 3
    back = torch.empty(16, 128, dtype=BF, device="cuda")
    cuda_lib.et_w4_dequantize(qc, sc, back)
    want = ref.w4_values(q, s, torch.float32).to(BF)
    assert torch.equal(back.cpu().nan_to_num(7.0), want.nan_to_num(7.0))


def test_quantize_every_quotient(cuda_lib):
    """Every pair of significands of a weight and its group's largest: each quotient that can lie near a half."""
    top = (1 + torch.arange(128) / 128).to(BF)                        # the group's largest, times a power of two
    val = torch.cat([(1 + torch.arange(128) / 128) * 2.0 ** -e for e in range(5)]).to(BF)
    val = torch.cat([val, -val, torch.zeros(7 * 186 - 1280)]).view(186, 7)
    w = torch.zeros(128, 186, 32, dtype=BF)
    w[:, :, 0] = top[:, None] * 1.0
    w[:, :, 1:8] = val.to(BF)
    w[:, :, 1:8] = torch.minimum(torch.maximum(w[:, :, 1:8], -w[:, :, :1]), w[:, :, :1])
    for scale in (1.0, 2.0 ** -100, 2.0 ** 100):
        ws = (w.float() * scale).to(BF).reshape(128, 186 * 32)
        q, s = ref.w4_pack(ws, 32)
        qc, sc = torch.empty_like(q, device="cuda"), torch.empty_like(s, device="cuda")
        cuda_lib.et_w4_quantize(ws.cuda(), qc, sc)
        assert torch.equal(sc.cpu(), s) and torch.equal(qc.cpu(), q)


# ------------------------------------------------------------------ experts

def _experts_inputs(T, H, F, En, k, group, seed):
    g = _gen(seed)
    x = torch.randn(T, H, generator=g).to(BF)
    gate, up, down = (_weight(sh, group, seed + i) for i, sh in enumerate(((En, F, H), (En, F, H), (En, H, F))))
    L = torch.randn(T, En, generator=g)
    val, idx = torch.topk(L, k, -1)
    return x, idx.to(torch.int32), torch.softmax(val, -1), gate, up, down


def _experts(E, x, idx, w, gate, up, down, T=None, d_T=None, ws=None, stream=None):
    Tm, H = x.shape
    En, F = gate[0].shape[:2]
    dev = [t.cuda() for t in (x, idx, w, *gate, *up, *down)]
    out = torch.full((Tm, H), 7.0, dtype=BF, device="cuda")
    ws = ws if ws is not None else E.alloc_workspace(
        E.et_w4_experts_workspace_bytes(Tm, H, F, En, idx.shape[1], H // gate[1].shape[1]))
    E.et_w4_experts(*dev, out, T=T, d_T=d_T, workspace=ws, stream=stream)
    return out, ws


def _check_experts(out, x, idx, w, gate, up, down, T=None):
    T = x.shape[0] if T is None else T
    want, mag = ref.experts(x[:T], idx[:T], w[:T], gate, up, down)
    ref.check(out[:T], want, B * (want.abs() + mag) + mag + 1e-38, "out")
    assert (out[T:] == 7).all()


EXPERTS = [(1, 64, 32, 1, 1, 32), (1, 256, 512, 8, 2, 128), (16, 256, 512, 8, 2, 64), (5, 96, 160, 4, 4, 32),
           (3, 640, 128, 200, 8, 128), (64, 128, 128, 16, 8, 64), (33, 192, 320, 3, 2, 64), (64, 64, 64, 2, 2, 32),
           (7, 2048, 768, 16, 8, 128), (20, 160, 1120, 5, 1, 32), (64, 256, 256, 256, 8, 128)]


@pytest.mark.parametrize("T,H,F,En,k,group", EXPERTS)
def test_experts(cuda_lib, T, H, F, En, k, group):
    a = _experts_inputs(T, H, F, En, k, group, T + H)
    out, ws = _experts(cuda_lib, *a)
    _check_experts(out, *a)
    assert torch.equal(out, _experts(cuda_lib, *a, ws=ws)[0])
    assert cuda_lib.et_status(ws) == (0, 0)


def test_experts_all_on_one(cuda_lib):
    """Every token on the same experts: rows beyond one pass."""
    T, H, F, En, k = 64, 128, 96, 40, 2
    x, idx, w, gate, up, down = _experts_inputs(T, H, F, En, k, 32, 9)
    idx[:, 0], idx[:, 1] = 7, 39
    out, _ = _experts(cuda_lib, x, idx, w, gate, up, down)
    _check_experts(out, x, idx, w, gate, up, down)


def test_experts_left_out_and_twice(cuda_lib):
    """-1 leaves an expert out (its weight, even NaN, is not used); a token may name one expert twice; a token
    without any expert gives zeros."""
    T, H, F, En, k = 6, 128, 192, 5, 4
    x, idx, w, gate, up, down = _experts_inputs(T, H, F, En, k, 64, 10)
    idx[0] = -1
    idx[1] = 3
    idx[2, 1:] = -1
    idx[3, 2] = idx[3, 0]
    w[0], w[2, 1:] = math.nan, math.nan
    out, ws = _experts(cuda_lib, x, idx, w, gate, up, down)
    assert (out[0] == 0).all()
    _check_experts(out, x, idx, w, gate, up, down)
    assert cuda_lib.et_status(ws) == (0, 0)
    none = torch.full_like(idx, -1)
    assert (_experts(cuda_lib, x, none, w, gate, up, down, ws=ws)[0] == 0).all()


def test_experts_bad_index_is_recorded(cuda_lib):
    T, H, F, En, k = 4, 64, 64, 3, 2
    x, idx, w, gate, up, down = _experts_inputs(T, H, F, En, k, 32, 11)
    bad = idx.clone()
    bad[1, 0], bad[2, 1], bad[3, 0] = 3, -2, 1 << 30
    out, ws = _experts(cuda_lib, x, bad, w, gate, up, down)
    assert cuda_lib.et_status(ws)[0] == cuda_lib.ET_ERR_BOUNDS
    seen = torch.where((bad >= 0) & (bad < En), bad, -1)
    _check_experts(out, x, seen, w, gate, up, down)
    cuda_lib.et_reset_status(ws)
    _check_experts(_experts(cuda_lib, x, idx, w, gate, up, down, ws=ws)[0], x, idx, w, gate, up, down)
    assert cuda_lib.et_status(ws) == (0, 0)


def test_experts_device_count_stream_and_graph(cuda_lib):
    """Captured once; replayed with other inputs and counts, and run on a side stream."""
    T, H, F, En, k = 24, 256, 384, 12, 3
    x, idx, w, gate, up, down = _experts_inputs(T, H, F, En, k, 128, 12)
    dT = torch.full((1,), T, dtype=torch.int32, device="cuda")
    dev = [t.cuda() for t in (x, idx, w, *gate, *up, *down)]
    out = torch.empty((T, H), dtype=BF, device="cuda")
    ws = cuda_lib.alloc_workspace(cuda_lib.et_w4_experts_workspace_bytes(T, H, F, En, k, 128))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cuda_lib.et_w4_experts(*dev, out, d_T=dT, workspace=ws, stream=s)
    torch.cuda.synchronize()
    _check_experts(out, x, idx, w, gate, up, down)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cuda_lib.et_w4_experts(*dev, out, d_T=dT, workspace=ws)
    for seed, n in ((13, T), (14, 1), (15, 0), (16, 9)):
        x2, idx2, w2, _, _, _ = _experts_inputs(T, H, 64, En, k, 32, seed)
        for d, v in zip(dev, (x2, idx2, w2)):
            d.copy_(v)
        dT.fill_(n)
        out.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        _check_experts(out, x2, idx2, w2, gate, up, down, T=n)
    dT.fill_(T + 1)
    out.fill_(7)
    g.replay()
    torch.cuda.synchronize()
    assert (out == 7).all() and cuda_lib.et_status(ws)[0] == cuda_lib.ET_ERR_BOUNDS
