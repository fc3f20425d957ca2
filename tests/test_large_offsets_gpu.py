"""Tensors of more than 2^31 and 2^32 elements: the last rows, whose offsets pass 32 bits, against the definitions."""
import numpy as np
import pytest
import torch

from tests import ref_more as ref
from tests.ref_ops import F32_HALF as U
from tests.ref_ops import check

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _room(gb):
    if torch.cuda.get_device_properties(0).total_memory < (gb + 8) * 2 ** 30:
        pytest.skip(f"needs {gb} GB")


def _keep(rows, H, p, seed, offset):
    """The kept elements of these rows alone."""
    thr = round(p * 65536)
    h = np.arange(H)
    out = np.zeros((len(rows), H), dtype=bool)
    for i, t in enumerate(rows):
        w = ref.philox([h // 8, np.full(H, t), np.full(H, offset), np.zeros(H)], [seed, 0])
        half = np.choose(h % 8 // 2, w) >> (16 * (h % 2)).astype(np.uint64) & np.uint64(65535)
        out[i] = half >= thr
    return torch.from_numpy(out), 65536 / (65536 - thr)


@pytest.mark.parametrize("T,H", [(530000, 8192), (300011, 7501)])
def test_dropout_and_layer_norm(cuda_lib, T, H):
    _room(30)
    E = cuda_lib
    base = torch.randn(64, H, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    x = base.repeat(T // 64 + 1, 1)[:T]
    y = x.flip(1).contiguous()
    out = torch.empty_like(x)
    rows = [0, 2 ** 31 // H, T - 2, T - 1]
    kept, mul = _keep(rows, H, 0.25, 9, 3)
    xs, ys = x[rows].cpu(), y[rows].cpu()
    z = xs.double() + torch.where(kept, ys.double() * mul, 0.0)
    mag = xs.double().abs() + ys.double().abs() * mul
    ws = E.alloc_workspace(E.et_layer_norm_workspace_bytes(T, H))
    E.et_dropout(x, y, out, p=0.25, seed=9, offset=3, workspace=ws)
    check(out[rows], z, ref.bf16_bound(z, 2 * U * mag), "dropout")
    E.et_layer_norm(x, y, None, out, eps=1e-5, p=0.25, seed=9, offset=3, workspace=ws)
    hat, n, r = ref.layer_norm(z)
    e_n, rel_r = ref.norm_error(xs, ys, mul, z, n, r)
    check(out[rows], hat, ref.bf16_bound(hat, e_n + 2 * U * n.abs()), "x_hat")
    E.et_layer_norm_bwd(x, y, None, x, out, None, eps=1e-5, p=0.25, seed=9, offset=3, workspace=ws)
    D, _, _ = ref.layer_norm_grad(z, n, r, None, None, xs)
    e, _, _ = ref.layer_norm_grad_bounds(n, r, e_n, rel_r, None, None, xs)
    check(out[rows], D, ref.bf16_bound(D, e), "dx")
    assert E.et_status(ws) == (0, 0)


def test_router_groups(cuda_lib):
    _room(40)
    E, T, En, k = cuda_lib, 2 ** 24 - 5, 256, 8
    base = torch.randn(64, En, generator=torch.Generator().manual_seed(2))
    logits = base.cuda().repeat(T // 64 + 1, 1)[:T]
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    counts, n = torch.empty(En, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    ws = E.alloc_workspace(E.et_router_groups_workspace_bytes(T, En, k))
    E.et_router_groups(logits, idx, w, score=E.ET_SCORE_SIGMOID, n_groups=8, k_groups=4, expert_counts=counts, n_routed=n, workspace=ws)
    want = ref.router_groups(base, k, 8, 4)
    times = T // 64 + (torch.arange(64) < T % 64)
    c = torch.zeros(En, dtype=torch.float64)
    for t in range(64):
        c[want["idx"][t]] += float(times[t])
    assert torch.equal(counts.cpu().double(), c) and int(n) == T
    at = torch.arange(64)
    for first in (0, 2 ** 23 // 64 * 64, T // 64 * 64 - 64):  # every row of three blocks, from the start to the end
        assert torch.equal(idx[first:first + 64].cpu().long(), want["idx"][at])
    d = torch.empty(T, En, device="cuda")
    dw = torch.ones(T, k, device="cuda")
    E.et_router_groups_bwd(logits, idx, w, counts, n, d, score=E.ET_SCORE_SIGMOID, renorm=False, d_topk_w=dw, workspace=ws)
    # every row's gradient is that of the row 64 before it, to the bit: no term knows the row
    assert torch.equal(d[:64], d[T // 64 * 64 - 64:T // 64 * 64]) and float(d[-1].abs().sum()) > 0


@pytest.mark.parametrize("M", [1, 12, 40])
def test_int8(cuda_lib, M):
    _room(12)
    E, N, K = cuda_lib, 70001, 65536
    w = torch.empty(N, K, dtype=torch.int8, device="cuda")
    w[:] = torch.randint(-127, 128, (K,), device="cuda", dtype=torch.int8)
    last = torch.randint(-127, 128, (3, K), device="cuda", dtype=torch.int8)
    w[-3:] = last
    x = torch.randint(-127, 128, (M, K), device="cuda", dtype=torch.int8)
    sx, sw = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    Y = torch.empty(M, N, dtype=BF, device="cuda")
    ws = E.alloc_workspace(E.et_i8_gemm_workspace_bytes(M, N, K))
    E.et_i8_gemm(x, sx, w, sw, Y, workspace=ws)
    cols = [0, 2 ** 31 // K, 2 ** 32 // K, N - 3, N - 2, N - 1]
    y, e = ref.i8_gemm(x.cpu(), sx.cpu(), w[cols].cpu(), sw[cols].cpu())
    check(Y[:, cols], y, ref.bf16_bound(y, e), "Y")
    assert E.et_status(ws) == (0, 0)


def test_int8_many_rows_with_a_device_count(cuda_lib):
    """More rows than one pass takes, counted on the device: whole passes, parts of one, none."""
    E, Mm, N, K = cuda_lib, 8500, 264, 272
    g = torch.Generator().manual_seed(3)
    x, w = (torch.randint(-127, 128, (s, K), generator=g).to(torch.int8) for s in (Mm, N))
    sx, sw = torch.rand(Mm, generator=g), torch.rand(N, generator=g)
    y, e = ref.i8_gemm(x, sx, w, sw)
    d_M = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = E.alloc_workspace(E.et_i8_gemm_workspace_bytes(Mm, N, K))
    a = [t.cuda() for t in (x, sx, w, sw)]
    for M in (Mm, 8192, 8193, 5, 0, 8191):
        Y = torch.full((Mm, N), 7.0, dtype=BF, device="cuda")
        d_M.fill_(M)
        E.et_i8_gemm(*a, Y, d_M=d_M, workspace=ws)
        if M:
            check(Y[:M], y[:M], ref.bf16_bound(y[:M], e[:M]), "Y")
        assert (Y[M:] == 7).all()
    assert E.et_status(ws) == (0, 0)


def test_dropout_in_place(cuda_lib):
    """out may be x or y, whatever H and alignment."""
    E = cuda_lib
    g = torch.Generator().manual_seed(4)
    for T, H, shift in ((40, 4096, 0), (33, 1001, 0), (17, 64, 1), (9, 5000, 3)):
        x, y = (torch.randn(T, H, generator=g).to(BF) for _ in range(2))
        want = torch.empty(T, H, dtype=BF, device="cuda")
        ws = E.alloc_workspace(E.et_dropout_workspace_bytes(T, H))
        E.et_dropout(x.cuda(), y.cuda(), want, p=0.3, seed=1, workspace=ws)
        for into in (0, 1):
            t = [torch.zeros(T * H + 8, dtype=BF, device="cuda")[shift:shift + T * H].view(T, H).copy_(v) for v in (x, y)]
            E.et_dropout(t[0], t[1], t[into], p=0.3, seed=1, workspace=ws)
            assert torch.equal(t[into], want) and torch.equal(t[1 - into].cpu(), (y, x)[into])
