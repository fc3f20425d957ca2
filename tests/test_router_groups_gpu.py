"""et_router_groups and its gradient on the GPU against the 64-bit definitions."""
import math

import pytest
import torch

from tests import ref_more as ref
from tests.ref_ops import check

pytestmark = pytest.mark.gpu
U = ref.U


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _forward(E, logits, k, G, kg, best=2, sigmoid=True, bias=None, renorm=True, scale=1.0, mask=None, T=None, d_T=None, ws=None):
    Tm, En = logits.shape
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    o = dict(idx=torch.full((Tm, k), -7, dtype=torch.int32, device="cuda"), w=torch.full((Tm, k), 9.0, device="cuda"),
             counts=torch.full((En,), -7, dtype=torch.int32, device="cuda"), n=torch.full((1,), -7, dtype=torch.int32, device="cuda"),
             mean_prob=torch.full((En,), 9.0, device="cuda"), loss=torch.full((1,), 9.0, device="cuda"))
    ws = ws if ws is not None else E.alloc_workspace(E.et_router_groups_workspace_bytes(Tm, En, k))
    E.et_router_groups(c(logits), o["idx"], o["w"], score=E.ET_SCORE_SIGMOID if sigmoid else E.ET_SCORE_SOFTMAX, n_groups=G,
                       k_groups=kg, group_best=best, bias=c(bias), renorm=renorm, scale=scale, token_mask=c(mask),
                       expert_counts=o["counts"], n_routed=o["n"], mean_prob=o["mean_prob"], loss=o["loss"], T=T, d_T=d_T,
                       workspace=ws)
    return o, ws


def _weight_bound(logits, r, renorm, scale):
    """(20 + E + |x - x0|) 2^-24 of the weight: x0 the row's largest logit, with renorm the largest chosen one."""
    L = torch.where(torch.isfinite(logits), logits.double(), torch.zeros((), dtype=torch.float64))
    x = torch.gather(L, 1, r["idx"].clamp(min=0))
    on = r["idx"] >= 0
    low = torch.full_like(x, -math.inf)
    x0 = torch.where(on, x, low).amax(-1, keepdim=True) if renorm else torch.where(logits > -math.inf, L, torch.full_like(L, -math.inf)).amax(-1, keepdim=True)
    d = torch.where(on, (x - x0).abs(), torch.zeros_like(x))
    return (20 + logits.shape[1] + d) * U * r["w"].abs() + abs(scale) * 2.0 ** -126


def _check(o, logits, k, G, kg, T=None, **how):
    T = logits.shape[0] if T is None else T
    how = dict(how)
    if how.get("mask") is not None:
        how["mask"] = how["mask"][:T]
    r = ref.router_groups(logits[:T], k, G, kg, **how)
    assert torch.equal(o["idx"][:T].cpu(), r["idx"].to(torch.int32))
    assert torch.equal(o["counts"].cpu(), r["counts"].to(torch.int32)) and int(o["n"]) == r["n"]
    check(o["w"][:T], r["w"], _weight_bound(logits[:T], r, how.get("renorm", True), how.get("scale", 1.0)), "w")
    L = torch.where(torch.isfinite(logits[:T]), logits[:T].double(), torch.zeros((), dtype=torch.float64))
    far = (L.amax(-1, keepdim=True) - L).abs() if T else L
    rel = (48 + logits.shape[1] + 4 * far + 5 * L.abs()) * U
    # a token's p, then sums over tokens: 32, and as many as follow
    bP = (r["p"] * (rel + 128 * U)).sum(0) / max(r["n"], 1) + 2.0 ** -126
    check(o["mean_prob"], r["mean_prob"], bP, "mean_prob")
    En = logits.shape[1]
    b = En * (r["counts"] / (max(r["n"], 1) * k) * (bP + 64 * U * r["mean_prob"])).sum()
    check(o["loss"], r["loss"], b.reshape(1) + 2.0 ** -120, "loss")
    assert (o["idx"][T:] == -7).all() and (o["w"][T:] == 9).all()  # rows behind the last: as they were
    return r, rel


def _backward(E, o, ws, logits, dl, dw, sigmoid=True, renorm=True, scale=1.0, mask=None, T=None, d_T=None):
    d = torch.full(logits.shape, 7.0, device="cuda")
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    E.et_router_groups_bwd(c(logits), o["idx"], o["w"], o["counts"], o["n"], d,
                           score=E.ET_SCORE_SIGMOID if sigmoid else E.ET_SCORE_SOFTMAX, renorm=renorm, scale=scale,
                           token_mask=c(mask), d_loss=c(dl), d_topk_w=c(dw), T=T, d_T=d_T, workspace=ws)
    return d


def _check_backward(d, logits, k, r, rel, dl, dw, sigmoid=True, renorm=True, scale=1.0, T=None):
    """Terms of the formula, each off by its weight's or p's error and a few roundings of their magnitudes."""
    T = logits.shape[0] if T is None else T
    zl = torch.zeros(1) if dl is None else dl
    zw = torch.zeros(T, k) if dw is None else dw[:T]
    g = ref.router_groups_grad(logits[:T], r, k, zl, zw, sigmoid=sigmoid, renorm=renorm, scale=scale)
    p, n, En = r["p"], max(r["n"], 1), logits.shape[1]
    C = En * r["counts"] / (n * k) / n
    mag = abs(float(zl)) * p * (C + (p * C).sum(-1, keepdim=True))
    on = r["idx"] >= 0
    W = torch.where(on, (r["w"] * zw.double()).abs(), torch.zeros(T, k, dtype=torch.float64))
    inner = W + (r["w"].abs() / abs(scale) * W.sum(-1, keepdim=True) if renorm and scale else 0.0)
    wrel = rel.amax(-1, keepdim=True)  # above every weight's own bound
    mag = mag.scatter_add(1, r["idx"].clamp(min=0), torch.where(on, inner, torch.zeros_like(inner)))
    if not renorm and not sigmoid:
        mag = mag + p * W.sum(-1, keepdim=True)
    check(d[:T], g, (3 * wrel + 64 * U) * mag + 2.0 ** -120, "d_logits")
    assert (d[T:] == 7).all()


# T, E, k, G, kg, best
CASES = [(1, 1, 1, 1, 1, 2), (1, 8, 2, 4, 2, 2), (3, 7, 7, 1, 1, 1), (16, 128, 8, 8, 4, 2), (33, 30, 4, 5, 3, 2),
         (40, 36, 8, 4, 3, 1), (64, 64, 8, 32, 8, 2), (129, 65, 3, 13, 2, 2), (257, 256, 8, 8, 4, 2), (31, 200, 1, 8, 1, 2),
         (300, 160, 6, 8, 3, 2), (700, 128, 8, 16, 6, 1), (900, 96, 8, 8, 8, 2), (1200, 16, 2, 2, 1, 2)]


@pytest.mark.parametrize("T,En,k,G,kg,best", CASES)
@pytest.mark.parametrize("sigmoid,bias,renorm,masked", [(True, True, True, False), (True, False, False, True), (False, True, False, True),
                                                        (False, False, True, False), (True, True, False, True), (False, True, True, False)])
def test_router_groups(cuda_lib, T, En, k, G, kg, best, sigmoid, bias, renorm, masked):
    g = _gen(T * 1000 + En)
    logits = torch.randn(T, En, generator=g) * 2
    b = torch.randn(En, generator=g) * 0.1 if bias else None
    mask = (torch.rand(T, generator=g) > 0.3).to(torch.uint8) if masked else None
    dl, dw = torch.tensor([0.7]), torch.randn(T, k, generator=g)
    how = dict(sigmoid=sigmoid, renorm=renorm, scale=2.5)
    o, ws = _forward(cuda_lib, logits, k, G, kg, best, bias=b, mask=mask, **how)
    r, rel = _check(o, logits, k, G, kg, best=best, bias=b, mask=mask, **how)
    for l, w in ((dl, dw), (None, dw), (dl, None)):
        d = _backward(cuda_lib, o, ws, logits, l, w, mask=mask, **how)
        _check_backward(d, logits, k, r, rel, l, w, **how)
    o2, _ = _forward(cuda_lib, logits, k, G, kg, best, bias=b, mask=mask, ws=ws, **how)
    assert all(torch.equal(o[n], o2[n]) for n in o)
    assert cuda_lib.et_status(ws) == (0, 0)


@pytest.mark.parametrize("En,k,G,kg", [(8, 2, 2, 1), (32, 8, 4, 2), (40, 8, 5, 3), (64, 4, 8, 4), (128, 8, 8, 4), (256, 8, 8, 4), (256, 8, 1, 1)])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_close_and_equal_scores(cuda_lib, En, k, G, kg, sigmoid):
    """Candidates that 32 bits cannot tell apart: logits in their last bits, scores and biases that nearly cancel, equal
    ones, logits and biases on coarse grids (ties at every place, across groups too), all equal."""
    g = _gen(En + sigmoid)
    T = 700
    near = torch.randn(T, En, generator=g)
    near[:100] = 1 + torch.randint(0, 30, (100, En), generator=g) * 2.0 ** -23
    near[100:200] = (torch.randn(100, En, generator=g) * 2).round() / 2
    near[200:300] = torch.randn(100, En, generator=g).bfloat16().float()
    near[300:400] = 0.5
    near[400:450] = torch.randn(50, 1, generator=g) + torch.randn(50, En, generator=g) * 1e-6
    near[450:500] = 12 + torch.randint(0, 5, (50, En), generator=g).float()  # sigmoid scores within 2^-17 of 1
    biases = [None, torch.zeros(En), torch.randint(-2, 3, (En,), generator=g) * 0.001]
    if sigmoid:  # score + bias alike to 2^-20 or so
        biases.append(0.5 - torch.sigmoid(near[600].double()).float())
        near[600:] = near[600] + torch.randn(100, En, generator=g) * 1e-6
    for b in biases:
        for best in (1, 2):
            o, _ = _forward(cuda_lib, near, k, G, kg, best, sigmoid=sigmoid, bias=b)
            r = ref.router_groups(near, k, G, kg, best, sigmoid=sigmoid, bias=b)
            assert torch.equal(o["idx"].cpu(), r["idx"].to(torch.int32))
            assert torch.equal(o["counts"].cpu(), r["counts"].to(torch.int32))
            check(o["w"], r["w"], _weight_bound(near, r, True, 1.0), "w")


def test_unavailable_experts(cuda_lib):
    """-inf logits and biases: whole groups, whole rows, fewer than k left; the lowest finite logits."""
    ninf, low = -math.inf, torch.finfo(torch.float32).min
    rows = torch.randn(10, 8, generator=_gen(1))
    rows[1] = ninf
    rows[2, 1:] = ninf
    rows[3, :4] = ninf
    rows[4] = low
    rows[5, ::2] = ninf
    rows[6, 4:] = low
    rows[7] = torch.tensor([-200.0, -201, -150, -149, -300, -151, -152, -400])  # scores below the smallest fp32
    rows[8] = torch.tensor([90.0, 100, 110, 30, -90, -100, 50, 60])
    b = torch.randn(8, generator=_gen(2)) * 0.1
    off = b.clone()
    off[[0, 1, 6]] = ninf
    dl, dw = torch.tensor([0.5]), torch.randn(10, 3, generator=_gen(3))
    for sigmoid in (True, False):
        for renorm in (True, False):
            for bias in (None, b, off, torch.full((8,), ninf)):
                for mask in (None, torch.tensor([1, 1, 1, 0, 1, 255, 1, 1, 1, 1], dtype=torch.uint8)):
                    how = dict(sigmoid=sigmoid, renorm=renorm, scale=1.5)
                    o, ws = _forward(cuda_lib, rows, 3, 4, 2, bias=bias, mask=mask, **how)
                    r, rel = _check(o, rows, 3, 4, 2, bias=bias, mask=mask, **how)
                    d = _backward(cuda_lib, o, ws, rows, dl, dw, mask=mask, **how).cpu()
                    g = ref.router_groups_grad(torch.where(rows > ninf, rows, torch.full_like(rows, -1e4)).clamp(min=-1e4), r, 3, dl, dw, **how)
                    ok = torch.isfinite(rows) & (rows > -100)  # elsewhere scores and their gradients are 0 in fp32
                    keep = ok | (rows == ninf)
                    row_ok = (rows[:, :] > -100).any(-1)  # rows of tiny scores are ratios, not what -1e4 above makes of them
                    assert torch.isfinite(d).all() and (d[~r["live"]] == 0).all()
                    sel = keep & row_ok[:, None]
                    tol = (3 * rel[ok].amax() + 64 * U) * 10  # terms of the order of 1, ten of them at most
                    assert ((d.double() - g).abs()[sel] <= float(tol)).all()


def test_tiny_scores_are_ratios(cuda_lib):
    """Sigmoid scores that underflow still give weights, probabilities and gradients as their ratios."""
    base = torch.randn(50, 16, generator=_gen(4))
    k, G, kg = 4, 4, 2
    # exact in 64 bits down to e^-700; the shifted logits are the rounded ones in both
    for shift in (-70.0, -120.0, -400.0):
        L = base + shift
        dl, dw = torch.tensor([0.3]), torch.randn(50, k, generator=_gen(5))
        o, ws = _forward(cuda_lib, L, k, G, kg)
        r, rel = _check(o, L, k, G, kg)
        d = _backward(cuda_lib, o, ws, L, dl, dw)
        _check_backward(d, L, k, r, rel, dl, dw)


def test_nan_and_infinity(cuda_lib):
    """A NaN logit ranks above all and shows; +inf is a score of 1 for sigmoid, shows for softmax; other tokens keep theirs."""
    logits = torch.randn(4, 8, generator=_gen(6))
    logits[1, 5], logits[2, 6] = math.nan, math.inf
    for bias in (None, torch.randn(8, generator=_gen(7)) * 0.1):
        o, ws = _forward(cuda_lib, logits, 2, 4, 2, bias=bias)
        assert int(o["idx"][1, 0]) == 5 and torch.isnan(o["w"][1]).all() and torch.isnan(o["loss"]).all()
        assert int((o["idx"][2] == 6).sum()) == 1 and torch.isfinite(o["w"][2]).all()
        d = _backward(cuda_lib, o, ws, logits, torch.ones(1), None)
        assert torch.isnan(d[1]).any()
        keep = [0, 3]
        r = ref.router_groups(logits[keep], 2, 4, 2, bias=bias)
        assert torch.equal(o["idx"][keep].cpu(), r["idx"].to(torch.int32))
        check(o["w"][keep], r["w"], _weight_bound(logits[keep], r, True, 1.0), "w")
        for renorm in (True, False):
            o, _ = _forward(cuda_lib, logits, 2, 4, 2, sigmoid=False, bias=bias, renorm=renorm)
            assert torch.isnan(o["w"][1]).all() and torch.isnan(o["w"][2]).all() and torch.isnan(o["loss"]).all()
            assert torch.isfinite(o["w"][keep]).all()
        mask = torch.tensor([1, 0, 0, 1], dtype=torch.uint8)  # masked out, they change nothing
        o, ws = _forward(cuda_lib, logits, 2, 4, 2, bias=bias, mask=mask)
        r = ref.router_groups(logits[keep], 2, 4, 2, bias=bias)
        check(o["loss"], r["loss"], 512 * U * r["loss"], "loss")
        d = _backward(cuda_lib, o, ws, logits, torch.ones(1), torch.ones(4, 2), mask=mask)
        assert (d[1] == 0).all() and (d[2] == 0).all() and torch.isfinite(d).all()
    for v in (math.inf, math.nan):  # a bias as large as that: its expert first, its weight as it is
        bias = torch.zeros(8)
        bias[3] = v
        o, _ = _forward(cuda_lib, logits[keep], 2, 1, 1, bias=bias)
        assert (o["idx"][:, 0] == 3).all() and torch.isfinite(o["w"]).all()


def test_large_biases(cuda_lib):
    """Biases far larger than the scores round them away in 32 bits; the choice is the exact one."""
    g = _gen(8)
    logits = torch.randn(200, 64, generator=g)
    for b in (torch.full((64,), 1e6), torch.randint(0, 2, (64,), generator=g) * 1e4 - 5e3, torch.randn(64, generator=g) * 1e7):
        for sigmoid in (True, False):
            o, _ = _forward(cuda_lib, logits, 6, 8, 3, bias=b, sigmoid=sigmoid)
            r = ref.router_groups(logits, 6, 8, 3, bias=b, sigmoid=sigmoid)
            assert torch.equal(o["idx"].cpu(), r["idx"].to(torch.int32))


def test_nothing_is_routed(cuda_lib):
    for logits, mask, T in ((torch.randn(9, 6), torch.zeros(9, dtype=torch.uint8), None), (torch.full((9, 6), -math.inf), None, None),
                            (torch.randn(9, 6), None, 0)):
        o, ws = _forward(cuda_lib, logits, 2, 3, 2, mask=mask, T=T)
        assert (o["counts"] == 0).all() and int(o["n"]) == 0 and (o["loss"] == 0).all() and (o["mean_prob"] == 0).all()
        d = _backward(cuda_lib, o, ws, logits, torch.ones(1), torch.ones(9, 2), mask=mask, T=T)
        if T is None:
            assert (o["idx"] == -1).all() and (o["w"] == 0).all() and (d == 0).all()
        else:
            assert (o["idx"] == -7).all() and (d == 7).all()


def test_device_count(cuda_lib):
    """One launch for every count: rows behind it stay; a count out of range is recorded and nothing is written."""
    logits = torch.randn(300, 24, generator=_gen(9))
    b = torch.randn(24, generator=_gen(10)) * 0.1
    dT = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = cuda_lib.alloc_workspace(cuda_lib.et_router_groups_workspace_bytes(300, 24, 4))
    dl, dw = torch.tensor([0.5]), torch.randn(300, 4, generator=_gen(11))
    for T in (300, 1, 0, 37):
        dT.fill_(T)
        o, _ = _forward(cuda_lib, logits, 4, 6, 3, bias=b, d_T=dT, ws=ws)
        d = _backward(cuda_lib, o, ws, logits, dl, dw, d_T=dT)
        if T:
            r, rel = _check(o, logits, 4, 6, 3, T=T, bias=b)
            _check_backward(d, logits, 4, r, rel, dl, dw, T=T)
        else:
            assert (o["counts"] == 0).all() and (o["idx"] == -7).all() and (d == 7).all()
    for T in (301, -1):
        dT.fill_(T)
        o, _ = _forward(cuda_lib, logits, 4, 6, 3, bias=b, d_T=dT, ws=ws)
        assert (o["idx"] == -7).all() and (o["counts"] == -7).all() and (o["loss"] == 9).all()
        assert cuda_lib.et_status(ws)[0] == cuda_lib.ET_ERR_BOUNDS
        cuda_lib.et_reset_status(ws)


@pytest.mark.parametrize("sigmoid,renorm", [(True, True), (True, False), (False, True), (False, False)])
def test_gradient_against_differences(cuda_lib, sigmoid, renorm):
    """The kernel's gradient along random directions against differences of the 64-bit forward, the choice held."""
    T, En, k = 20, 12, 3
    logits = torch.randn(T, En, generator=_gen(12))
    dl, dw = torch.tensor([0.9]), torch.randn(T, k, generator=_gen(13))
    how = dict(sigmoid=sigmoid, renorm=renorm, scale=1.7)
    o, ws = _forward(cuda_lib, logits, k, 4, 2, **how)
    d = _backward(cuda_lib, o, ws, logits, dl, dw, **how).double().cpu()
    idx = o["idx"].cpu().long()

    def f(v):
        r = ref.router_groups(v, k, 4, 2, idx=idx, **how)
        return (r["loss"] * dl.double()).sum() + (r["w"] * dw.double()).sum()
    for s in range(4):
        v = torch.randn(T, En, generator=_gen(20 + s), dtype=torch.float64)
        h = 1e-6
        num = (f(logits.double() + h * v) - f(logits.double() - h * v)) / (2 * h)
        # the kernel's 240 entries off by some 100 x 2^-24 of terms of order 1; the difference's own error is h^2
        assert abs(float(num - (d * v).sum())) <= 240 * 400 * U


def test_no_bias_and_one_group_choose_as_the_plain_router(cuda_lib):
    """Without bias, with one group, the choice and the renormalised softmax weights are et_router_topk's."""
    T, En, k = 500, 96, 6
    logits = torch.randn(T, En, generator=_gen(14)).cuda()
    o, _ = _forward(cuda_lib, logits.cpu(), k, 1, 1, sigmoid=False)
    idx, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    ws = cuda_lib.alloc_workspace(cuda_lib.et_router_topk_workspace_bytes(T, En, k))
    cuda_lib.et_router_topk(logits, idx, w, workspace=ws)
    assert torch.equal(o["idx"], idx)
    check(o["w"], w, 64 * U * w.double().cpu(), "w")
    o, _ = _forward(cuda_lib, logits.cpu(), k, 1, 1, sigmoid=True)  # sigmoid orders as its logits do
    assert torch.equal(o["idx"], idx)


@pytest.mark.parametrize("T,En", [(77, 40), (77, 128), (77, 160), (77, 256), (1030, 64), (1030, 160), (1030, 256)])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_any_alignment(cuda_lib, T, En, sigmoid):
    """Logits and gradients that start anywhere: what aligned ones give."""
    k = 4
    g = _gen(En)
    logits, dl, dw = torch.randn(T, En, generator=g), torch.randn(1, generator=g), torch.randn(T, k, generator=g).cuda()
    o, ws = _forward(cuda_lib, logits, k, 4, 2, sigmoid=sigmoid)
    want = _backward(cuda_lib, o, ws, logits, dl, dw, sigmoid=sigmoid)
    score = cuda_lib.ET_SCORE_SIGMOID if sigmoid else cuda_lib.ET_SCORE_SOFTMAX
    for shift in (1, 2, 3):
        lo, d = (torch.zeros(T * En + 4, device="cuda")[shift:shift + T * En].view(T, En) for _ in range(2))
        lo.copy_(logits)
        idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
        cuda_lib.et_router_groups(lo, idx, w, score=score, n_groups=4, k_groups=2, workspace=ws)
        assert torch.equal(idx, o["idx"]) and torch.equal(w, o["w"])
        cuda_lib.et_router_groups_bwd(lo, idx, w, o["counts"], o["n"], d, score=score, d_loss=dl.cuda(), d_topk_w=dw, workspace=ws)
        # other lanes hold other experts: the sums over a row go in another order, a few roundings of their terms
        check(d, want.cpu().double(), 96 * U * (want.cpu().double().abs() + want.cpu().double().abs().amax(-1, keepdim=True)), "d_logits")


# ------------------------------------------------------------------ many rows: four share a warp

MANY = [(En, G) for En in (32, 64, 128, 256) for G in (1, 2, 4, 8, 16, 32)] + [(96, 4), (96, 32), (160, 8), (160, 32), (192, 16), (192, 3), (224, 2), (224, 8), (120, 8)]


@pytest.mark.parametrize("En,G", MANY)
@pytest.mark.parametrize("sigmoid,bias,renorm,masked", [(True, True, True, True), (False, False, False, False)])
def test_many_rows(cuda_lib, En, G, sigmoid, bias, renorm, masked):
    T, kg = 1027, max(1, G // 2)
    k, best = min(8, En // G * kg), 1 + G % 4 // 2
    g = _gen(En * 100 + G)
    logits = torch.randn(T, En, generator=g) * 2
    b = torch.randn(En, generator=g) * 0.1 if bias else None
    mask = (torch.rand(T, generator=g) > 0.3).to(torch.uint8) if masked else None
    how = dict(sigmoid=sigmoid, renorm=renorm, scale=2.5)
    o, ws = _forward(cuda_lib, logits, k, G, kg, best, bias=b, mask=mask, **how)
    _check(o, logits, k, G, kg, best=best, bias=b, mask=mask, **how)
    o2, _ = _forward(cuda_lib, logits, k, G, kg, best, bias=b, mask=mask, ws=ws, **how)
    assert all(torch.equal(o[n], o2[n]) for n in o)
    assert cuda_lib.et_status(ws) == (0, 0)


def _hard_rows(T, En, G, g):
    """Rows where choosing goes wrong if it goes wrong anywhere, in turn."""
    L = torch.randn(T, En, generator=g)
    i = torch.arange(T) % 12
    gs = En // G
    L[i == 1] = L[i == 1].bfloat16().float()                                    # coarse: equal logits
    L[i == 2] = torch.randint(-2, 3, (int((i == 2).sum()), En), generator=g).float()  # many ties
    L[i == 3] = 0.25                                                            # all equal
    L[i == 4] = 0.5 + torch.randint(-3, 4, (int((i == 4).sum()), En), generator=g) * 2.0 ** -24  # a few ulp apart
    L[i == 5] = torch.where(torch.rand(int((i == 5).sum()), En, generator=g) < 0.8, torch.tensor(-math.inf), L[i == 5])
    L[i == 6, :gs] = -math.inf                                                  # a group that nobody can choose
    L[i == 7] = -math.inf                                                       # a row that is not routed
    L[i == 7, En // 2] = torch.where(torch.arange(int((i == 7).sum())) % 2 == 0, -math.inf, 1.0)
    L[i == 8] = L[i == 8] * 3 - 100.0                                           # tiny scores
    L[i == 9] = L[i == 9] * 4 + 25.0                                            # sigmoids that are 1
    L[i == 10, ::5] = math.inf
    L[i == 11, 3] = math.nan
    return L


@pytest.mark.parametrize("En,G,kg", [(32, 8, 4), (32, 32, 9), (64, 16, 5), (64, 1, 1), (128, 4, 2), (128, 16, 6), (256, 8, 4), (256, 32, 8), (256, 2, 1), (96, 16, 4),
                                      (160, 8, 3), (192, 32, 11), (224, 4, 2)])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("bias", [None, "random", "zero", "some"])
def test_four_rows_a_warp_choose_as_one(cuda_lib, En, G, kg, sigmoid, bias):
    """Many rows in one call, and the same rows in short calls: the same choice, for hard rows in every place of a warp."""
    T, k = 2051, min(8, En // G * kg)
    g = _gen(En + G)
    L = _hard_rows(T, En, G, g)
    L = L[torch.randperm(T, generator=g)]
    b = None
    if bias is not None:
        b = torch.randn(En, generator=g) * 0.05 if bias == "random" else torch.zeros(En)
        if bias == "some":
            b[1], b[En // 2 + 1], b[En - 1] = -math.inf, 3.0, -1e-7
    for best in (1, 2):
        for renorm in (True, False):
            how = dict(sigmoid=sigmoid, bias=b, renorm=renorm)
            o, _ = _forward(cuda_lib, L, k, G, kg, best, **how)
            parts = [_forward(cuda_lib, L[t:t + 500], k, G, kg, best, **how)[0] for t in range(0, T, 500)]
            assert torch.equal(o["idx"], torch.cat([q["idx"] for q in parts]))
            assert torch.equal(o["counts"], sum(q["counts"] for q in parts)) and int(o["n"]) == sum(int(q["n"]) for q in parts)
            w, v = o["w"].cpu().double(), torch.cat([q["w"] for q in parts]).cpu().double()
            assert torch.equal(torch.isnan(w), torch.isnan(v))
            # the same terms summed in another order: the sum's 256 roundings at most
            check(torch.where(torch.isnan(w), 0.0, w), torch.where(torch.isnan(v), 0.0, v), 256 * U * torch.where(torch.isnan(v), 0.0, v).abs(), "w")
    # and against the definition, rows without NaN or infinity above
    rows = torch.isfinite(torch.where(L == -math.inf, 0.0, L)).all(-1).nonzero()[:, 0][:150]
    want = ref.router_groups(L[rows], k, G, kg, 2, sigmoid=sigmoid, bias=b)
    assert torch.equal(o["idx"][rows.cuda()].cpu().long(), want["idx"])


def test_many_rows_device_count(cuda_lib):
    """One call for up to 3000 rows, whatever the device says."""
    T, En, k = 3000, 64, 4
    g = _gen(8)
    logits = torch.randn(T, En, generator=g)
    d_T = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = cuda_lib.alloc_workspace(cuda_lib.et_router_groups_workspace_bytes(T, En, k))
    for n in (3000, 1, 0, 1501, 6):
        d_T.fill_(n)
        o, _ = _forward(cuda_lib, logits, k, 8, 3, d_T=d_T, ws=ws)
        _check(o, logits, k, 8, 3, T=n)
    for n in (3001, -1):
        d_T.fill_(n)
        o, _ = _forward(cuda_lib, logits, k, 8, 3, d_T=d_T, ws=ws)
        assert (o["idx"] == -7).all() and cuda_lib.et_status(ws)[0] == cuda_lib.ET_ERR_BOUNDS
        cuda_lib.et_reset_status(ws)


def test_long_batches_of_rows(cuda_lib):
    """More rows than a lane adds up at a time: probabilities and loss to their bound."""
    T, En, k = 700000, 32, 2
    g = _gen(5)
    rows = torch.randn(64, En, generator=g)
    o, _ = _forward(cuda_lib, rows.repeat(T // 64 + 1, 1)[:T], k, 4, 2)
    w = T // 64 + (torch.arange(64) < T % 64)
    r = ref.router_groups(rows, k, 4, 2)
    counts = torch.zeros(En, dtype=torch.float64)
    for t in range(64):
        counts[r["idx"][t]] += float(w[t])
    assert torch.equal(o["counts"].cpu().double(), counts)
    want = (r["p"] * w[:, None].double()).sum(0) / T
    # a p's own bound, 32 rows of a lane, then batches: T / (152 16 4 32) = 2.3, 4, 16 warps, 152 CTAs
    far = (rows.amax(-1, keepdim=True) - rows).abs().double()
    rel = (48 + En + 4 * far + 5 * rows.abs().double()).amax() * U
    check(o["mean_prob"], want, (rel + 256 * U) * want, "mean_prob")
