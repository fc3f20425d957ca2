"""et_router_topk and its gradient on the GPU against the 64-bit definitions."""
import math

import pytest
import torch

from tests import ref_ops as ref

pytestmark = pytest.mark.gpu
U = ref.F32_HALF


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _forward(E, logits, k, mask=None, T=None, d_T=None, ws=None, stream=None):
    Tm, En = logits.shape
    L = logits.cuda()
    m = None if mask is None else mask.cuda()
    o = dict(idx=torch.full((Tm, k), -7, dtype=torch.int32, device="cuda"),
             w=torch.full((Tm, k), 9.0, device="cuda"), counts=torch.full((En,), -7, dtype=torch.int32, device="cuda"),
             n=torch.full((1,), -7, dtype=torch.int32, device="cuda"), mean_prob=torch.full((En,), 9.0, device="cuda"),
             losses=torch.full((2,), 9.0, device="cuda"))
    ws = ws if ws is not None else E.alloc_workspace(E.et_router_topk_workspace_bytes(Tm, En, k))
    E.et_router_topk(L, o["idx"], o["w"], token_mask=m, expert_counts=o["counts"], n_routed=o["n"],
                     mean_prob=o["mean_prob"], losses=o["losses"], T=T, d_T=d_T, workspace=ws, stream=stream)
    return o, ws, L, m


def _check_forward(o, logits, k, mask=None, T=None):
    T = logits.shape[0] if T is None else T
    r = ref.router(logits[:T], k, None if mask is None else mask[:T])
    En = logits.shape[1]
    assert torch.equal(o["idx"][:T].cpu(), r["idx"].to(torch.int32))
    assert torch.equal(o["counts"].cpu(), r["counts"].to(torch.int32)) and int(o["n"]) == r["n"]
    # exp (2 ulp = 4 half steps), its argument's subtraction (relative to the largest |L - L0|), the sum over
    # up to E entries and a division: relative to the weight
    fin = torch.where(torch.isfinite(logits[:T]), logits[:T].double(), 0.0)
    spread = float(fin.max() - fin.min()) if T else 0.0
    rel = (8 + spread + En) * U
    ref.check(o["w"][:T], r["w"], rel * r["w"] + 1e-38, "w")
    ref.check(o["mean_prob"], r["mean_prob"], (rel + 64 * U) * r["mean_prob"] + 1e-38, "mean_prob")
    top = float(fin.abs().max()) if T else 0.0
    lse_err = (2 * top + 16 + spread + En) * U
    b = torch.stack((r["losses"][0] * (2 * rel + 128 * U), 2 * r["lse"].abs().sum() / max(r["n"], 1) * lse_err + r["losses"][1] * 64 * U))
    ref.check(o["losses"], r["losses"], b + 1e-38, "losses")
    assert (o["idx"][T:] == -7).all() and (o["w"][T:] == 9).all()  # rows behind the last: as they were
    return r, rel, lse_err


def _backward(E, o, ws, L, m, dl, dw, T=None, d_T=None, stream=None):
    d = torch.full_like(L, 7.0)
    E.et_router_topk_bwd(L, o["idx"], o["w"], o["counts"], o["n"], d, token_mask=m,
                         d_losses=None if dl is None else dl.cuda(), d_topk_w=None if dw is None else dw.cuda(),
                         T=T, d_T=d_T, workspace=ws, stream=stream)
    return d


def _check_backward(d, logits, k, mask, dl, dw, r, rel, lse_err, T=None):
    T = logits.shape[0] if T is None else T
    zl = torch.zeros(2) if dl is None else dl
    zw = torch.zeros(T, k) if dw is None else dw[:T]
    g = ref.router_grad(logits[:T], k, zl, zw, None if mask is None else mask[:T])
    p, n, En = r["p"], max(r["n"], 1), logits.shape[1]
    c = En * r["counts"] / (n * k) / n
    mag = abs(float(zl[0])) * p * (c + (p * c).sum(-1, keepdim=True)) + abs(float(zl[1])) * 2 / n * r["lse"].abs()[:, None] * p
    on = r["idx"] >= 0
    dwa = torch.where(on, zw.double().abs(), 0.0)
    sel = torch.where(on, r["w"] * (dwa + (r["w"] * dwa).sum(-1, keepdim=True)), 0.0)
    mag = mag.scatter_add(1, r["idx"].clamp(min=0), sel)
    extra = abs(float(zl[1])) * 2 / n * lse_err * p
    ref.check(d[:T], g, (2 * rel + 32 * U) * mag + extra + 1e-38, "d_logits")
    assert (d[T:] == 7).all()


CASES = [(1, 1, 1), (1, 8, 2), (3, 7, 7), (16, 8, 2), (33, 31, 4), (40, 33, 8), (64, 64, 8), (129, 65, 3), (257, 128, 8),
         (31, 200, 1), (5000, 256, 8), (4096, 128, 8), (9000, 16, 2)]


@pytest.mark.parametrize("T,En,k", CASES)
@pytest.mark.parametrize("masked", [False, True])
def test_router(cuda_lib, T, En, k, masked):
    g = _gen(T * 1000 + En)
    logits = torch.randn(T, En, generator=g) * 2
    mask = (torch.rand(T, generator=g) > 0.3).to(torch.uint8) if masked else None
    dl, dw = torch.tensor([0.7, -0.3]), torch.randn(T, k, generator=g)
    o, ws, L, m = _forward(cuda_lib, logits, k, mask)
    r, rel, le = _check_forward(o, logits, k, mask)
    _check_backward(_backward(cuda_lib, o, ws, L, m, dl, dw), logits, k, mask, dl, dw, r, rel, le)
    _check_backward(_backward(cuda_lib, o, ws, L, m, None, dw), logits, k, mask, None, dw, r, rel, le)
    _check_backward(_backward(cuda_lib, o, ws, L, m, dl, None), logits, k, mask, dl, None, r, rel, le)
    # the same bits again, from the same workspace
    o2, _, _, _ = _forward(cuda_lib, logits, k, mask, ws=ws)
    assert all(torch.equal(o[n], o2[n]) for n in o)
    assert cuda_lib.et_status(ws) == (0, 0)


def test_ties_and_masks(cuda_lib):
    """Equal logits, -0.0, -inf, rows with fewer than k finite logits or none, the lowest finite value."""
    ninf, low = -math.inf, torch.finfo(torch.float32).min
    rows = [[0.0, -0.0, 0.0, 0.0, -1.0], [ninf] * 5, [ninf, 2.0, ninf, ninf, 1.0], [ninf, ninf, ninf, ninf, 3.0],
            [low, low, 0.0, low, low], [1.0, 1.0, 1.0, 1.0, 1.0], [low, 1.0, ninf, low, 1.0], [5.0, 4.0, 3.0, 2.0, 1.0]]
    logits = torch.tensor(rows)
    for mask in (None, torch.tensor([1, 1, 1, 0, 1, 1, 255, 1], dtype=torch.uint8)):
        dl, dw = torch.tensor([0.5, 0.25]), torch.randn(8, 3, generator=_gen(3))
        o, ws, L, m = _forward(cuda_lib, logits, 3, mask)
        r = ref.router(logits, 3, mask)
        assert torch.equal(o["idx"].cpu(), r["idx"].to(torch.int32))
        assert torch.equal(o["counts"].cpu(), r["counts"].to(torch.int32)) and int(o["n"]) == r["n"]
        ref.check(o["w"], r["w"], 32 * U, "w")
        ref.check(o["losses"], r["losses"], 64 * U * r["losses"].abs(), "losses")
        d = _backward(cuda_lib, o, ws, L, m, dl, dw)
        ref.check(d, ref.router_grad(logits, 3, dl, dw, mask), 64 * U, "d_logits")


@pytest.mark.parametrize("En,k", [(5, 3), (8, 8), (40, 8), (64, 4), (100, 8), (128, 8), (200, 7), (256, 8)])
def test_close_and_equal_logits(cuda_lib, En, k):
    """Logits that differ in their last bits only, equal ones among them, of either sign, at the k-th place and
    elsewhere; logits rounded to bf16; -inf and the lowest finite values side by side."""
    T = 600
    g = _gen(En)
    near = 1 + torch.randint(0, 30, (T, En), generator=g) * 2.0 ** -23
    near[100:200] = -near[100:200]
    near[200:300] = torch.randn(100, En, generator=g).bfloat16().float()
    near[300:400] = torch.where(torch.rand(100, En, generator=g) < 0.5, near[300:400], torch.randn(100, En, generator=g))
    low = torch.tensor([-math.inf, torch.finfo(torch.float32).min, -3.4e38, 0.0, -0.0, 1e-45, -1e-45])
    near[400:500] = low[torch.randint(0, 7, (100, En), generator=g)]
    near[500:] = torch.randint(-2, 3, (100, En), generator=g).float()
    o, _, _, _ = _forward(cuda_lib, near, k)
    r = ref.router(near, k)
    assert torch.equal(o["idx"].cpu(), r["idx"].to(torch.int32))
    assert torch.equal(o["counts"].cpu(), r["counts"].to(torch.int32)) and int(o["n"]) == r["n"]
    # weights: each logit's distance from the largest, exp and the sum over k (as above), 0 far below
    fin = torch.where(torch.isfinite(near), near.double(), 0.0).abs()
    fin = torch.where(fin < 1e30, fin, 0.0)
    ref.check(o["w"], r["w"], (8 + 2 * float(fin.max()) + k) * U * r["w"] + 1e-38, "w")


def test_nothing_is_routed(cuda_lib):
    """All tokens masked, all logits -inf, no tokens at all: zeros, not NaN."""
    for logits, mask, T in ((torch.randn(9, 6), torch.zeros(9, dtype=torch.uint8), None),
                            (torch.full((9, 6), -math.inf), None, None), (torch.randn(9, 6), None, 0)):
        o, ws, L, m = _forward(cuda_lib, logits, 2, mask, T=T)
        assert (o["counts"] == 0).all() and int(o["n"]) == 0
        assert (o["losses"] == 0).all() and (o["mean_prob"] == 0).all()
        d = _backward(cuda_lib, o, ws, L, m, torch.ones(2), torch.ones(9, 2), T=T)
        if T is None:
            assert (o["idx"] == -1).all() and (o["w"] == 0).all() and (d == 0).all()
        else:
            assert (o["idx"] == -7).all() and (d == 7).all()


def test_nan_and_infinity_show(cuda_lib):
    """A NaN or +inf logit makes its token's weights and the losses NaN; other tokens keep theirs."""
    logits = torch.randn(4, 8, generator=_gen(5))
    logits[1, 3], logits[2, 6] = math.nan, math.inf
    o, ws, L, m = _forward(cuda_lib, logits, 2)
    assert int(o["idx"][1, 0]) == 3 and int(o["idx"][2, 0]) == 6
    assert torch.isnan(o["w"][1]).all() and torch.isnan(o["losses"]).all()
    keep = [0, 3]
    r = ref.router(logits[keep], 2)
    assert torch.equal(o["idx"][keep].cpu(), r["idx"].to(torch.int32))
    ref.check(o["w"][keep], r["w"], 32 * U, "w")
    d = _backward(cuda_lib, o, ws, L, m, torch.ones(2), None)
    assert torch.isnan(d[1]).all() and torch.isnan(d[2]).all()
    # masked out, they change nothing
    mask = torch.tensor([1, 0, 0, 1], dtype=torch.uint8)
    o, ws, L, m = _forward(cuda_lib, logits, 2, mask)
    _check = ref.router(logits[keep], 2)
    ref.check(o["losses"], _check["losses"], 64 * U * _check["losses"].abs(), "losses")
    d = _backward(cuda_lib, o, ws, L, m, torch.ones(2), torch.ones(4, 2))
    assert (d[1] == 0).all() and (d[2] == 0).all() and torch.isfinite(d).all()


def test_device_count(cuda_lib):
    """One launch for every count: rows behind it stay; a count out of range is recorded and nothing is written."""
    logits = torch.randn(300, 24, generator=_gen(6))
    dT = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = cuda_lib.alloc_workspace(cuda_lib.et_router_topk_workspace_bytes(300, 24, 4))
    dl, dw = torch.tensor([0.5, 0.1]), torch.randn(300, 4, generator=_gen(7))
    for T in (300, 1, 0, 37):
        dT.fill_(T)
        o, _, L, m = _forward(cuda_lib, logits, 4, d_T=dT, ws=ws)
        d = _backward(cuda_lib, o, ws, L, m, dl, dw, d_T=dT)
        r, rel, le = _check_forward(o, logits, 4, T=T)
        if T:
            _check_backward(d, logits, 4, None, dl, dw, r, rel, le, T=T)
    for T in (301, -1):
        dT.fill_(T)
        o, _, L, m = _forward(cuda_lib, logits, 4, d_T=dT, ws=ws)
        assert (o["idx"] == -7).all() and (o["counts"] == -7).all() and (o["losses"] == 9).all()
        assert cuda_lib.et_status(ws)[0] == cuda_lib.ET_ERR_BOUNDS
        cuda_lib.et_reset_status(ws)


def test_gradient_against_differences(cuda_lib):
    """The kernel's gradient along random directions against differences of the 64-bit forward."""
    T, En, k = 20, 12, 3
    logits = torch.randn(T, En, generator=_gen(8))
    dl, dw = torch.tensor([0.9, 0.4]), torch.randn(T, k, generator=_gen(9))
    o, ws, L, m = _forward(cuda_lib, logits, k)
    d = _backward(cuda_lib, o, ws, L, m, dl, dw).double().cpu()

    def f(v):
        r = ref.router(v, k)
        return (r["losses"] * dl.double()).sum() + (r["w"] * dw.double()).sum()
    for s in range(4):
        v = torch.randn(T, En, generator=_gen(20 + s), dtype=torch.float64)
        h = 1e-6
        num = (f(logits.double() + h * v) - f(logits.double() - h * v)) / (2 * h)
        assert abs(float(num - (d * v).sum())) <= 1e-4


def test_streams_and_graph(cuda_lib):
    """On a side stream, and captured once and replayed with other inputs and counts."""
    T, En, k = 600, 40, 4
    s = torch.cuda.Stream()
    logits = torch.randn(T, En, generator=_gen(10))
    L = logits.cuda()
    dT = torch.full((1,), T, dtype=torch.int32, device="cuda")
    idx, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    counts, n = torch.empty(En, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    P, ls = torch.empty(En, device="cuda"), torch.empty(2, device="cuda")
    dl, dw, d = torch.ones(2, device="cuda"), torch.randn(T, k, device="cuda"), torch.empty_like(L)
    ws = cuda_lib.alloc_workspace(cuda_lib.et_router_topk_workspace_bytes(T, En, k))

    def step(stream):
        cuda_lib.et_router_topk(L, idx, w, expert_counts=counts, n_routed=n, mean_prob=P, losses=ls, d_T=dT,
                                workspace=ws, stream=stream)
        cuda_lib.et_router_topk_bwd(L, idx, w, counts, n, d, d_losses=dl, d_topk_w=dw, d_T=dT, workspace=ws, stream=stream)
    s.wait_stream(torch.cuda.current_stream())
    step(s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(None)
    for seed, rows in ((11, T), (12, 77), (13, 1)):
        logits = torch.randn(T, En, generator=_gen(seed))
        L.copy_(logits)
        dT.fill_(rows)
        g.replay()
        torch.cuda.synchronize()
        r = ref.router(logits[:rows], k)
        assert torch.equal(idx[:rows].cpu(), r["idx"].to(torch.int32)) and int(n) == rows
        ref.check(ls, r["losses"], 256 * U * r["losses"].abs(), "losses")
        gr = ref.router_grad(logits[:rows], k, torch.ones(2), dw[:rows].cpu())
        ref.check(d[:rows], gr, 256 * U * (1 + gr.abs()) * float(dw.abs().max()), "d_logits")
