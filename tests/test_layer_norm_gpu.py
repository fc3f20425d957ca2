"""et_dropout and et_layer_norm with its gradient on the GPU against the 64-bit definitions."""
import math

import pytest
import torch

from tests import ref_more as ref
from tests.ref_ops import check

pytestmark = pytest.mark.gpu
U = ref.U
SEED, OFFSET = 0x1234567890ABCDEF, 0xFEDCBA0987654321


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(g, *shape, scale=1.0, add=0.0):
    return (torch.randn(*shape, generator=g) * scale + add).bfloat16()


def _c(t):
    return None if t is None else t.cuda()


def _off(t, shift):
    """The tensor on the GPU, `shift` elements behind an aligned address."""
    if t is None:
        return None
    b = torch.empty(t.numel() + 64, dtype=t.dtype, device="cuda")
    v = b[shift:shift + t.numel()].view(t.shape)
    v.copy_(t)
    return v


# ------------------------------------------------------------------ dropout

@pytest.mark.parametrize("T,H", [(1, 1), (1, 8), (3, 7), (2, 4096), (17, 33), (64, 40), (5, 2047), (3, 2056), (9, 2049), (1000, 24),
                                 (2, 20000), (1, 262144), (700, 512)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9999])
@pytest.mark.parametrize("with_x", [False, True])
def test_dropout(cuda_lib, T, H, p, with_x):
    g = _gen(T * 31 + H)
    y, x = _randn(g, T, H), _randn(g, T, H) if with_x else None
    ws = cuda_lib.alloc_workspace(cuda_lib.et_dropout_workspace_bytes(T, H))
    want = ref.residual(x, y, p, SEED, OFFSET)
    mul = ref.keep(1, 1, p, 0, 0)[1]
    mag = y.double().abs() * mul + (x.double().abs() if with_x else 0.0)
    bound = ref.bf16_bound(want, 2 * U * mag)
    for shift in (0, 3):
        out = _off(torch.full((T, H), 7.0, dtype=torch.bfloat16), shift)
        cuda_lib.et_dropout(_off(x, shift), _off(y, shift), out, p=p, seed=SEED, offset=OFFSET, workspace=ws)
        check(out, want, bound, f"out, {shift} elements off")
    a = _c(y)  # in place, and the gradient of y: the same call
    cuda_lib.et_dropout(None, a, a, p=p, seed=SEED, offset=OFFSET, workspace=ws)
    k, _ = ref.keep(T, H, p, SEED, OFFSET)
    check(a, torch.where(k, y.double() * mul, 0.0), ref.bf16_bound(y.double() * mul, U * mag), "dy in place")
    assert ((a.cpu() == 0) | k).all()
    assert cuda_lib.et_status(ws) == (0, 0)


def test_dropped_values_do_not_matter(cuda_lib):
    """NaN and infinities where the mask drops them leave no trace."""
    T, H, p = 40, 96, 0.3
    k, mul = ref.keep(T, H, p, 5, 6)
    y = _randn(_gen(1), T, H)
    bad = torch.where(k, y.float(), torch.tensor([math.nan, math.inf, -math.inf] * (T * H // 3)).view(T, H)).bfloat16()
    x = _randn(_gen(2), T, H)
    ws = cuda_lib.alloc_workspace(cuda_lib.et_layer_norm_workspace_bytes(T, H))
    out = [torch.empty(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    for i, v in enumerate((y, bad)):
        cuda_lib.et_dropout(_c(x), _c(v), out[i], p=p, seed=5, offset=6, workspace=ws)
        cuda_lib.et_layer_norm(_c(x), _c(v), None, out[2 + i], eps=1e-5, p=p, seed=5, offset=6, workspace=ws)
    assert torch.equal(out[0], out[1]) and torch.equal(out[2], out[3])


def test_dropout_rate_and_independence(cuda_lib):
    """The kept share, and other masks for another seed, offset, row and column."""
    T, H, p = 512, 4096, 0.25
    ws = cuda_lib.alloc_workspace(cuda_lib.et_dropout_workspace_bytes(T, H))
    one = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")

    def mask(seed, offset):
        out = torch.empty_like(one)
        cuda_lib.et_dropout(None, one, out, p=p, seed=seed, offset=offset, workspace=ws)
        return out > 0
    a = mask(1, 0)
    n = T * H
    five = 5 * math.sqrt(p * (1 - p) / n)  # five deviations
    assert abs(float(a.double().mean()) - (1 - p)) < five
    both = (1 - p) ** 2
    five2 = 5 * math.sqrt(both * (1 - both) / n)
    for b in (mask(2, 0), mask(1, 1), mask(1 << 32, 0), mask(1, 1 << 32), a.roll(1, 0), a.roll(1, 1), a.roll(8, 1)):
        assert abs(float((a & b).double().mean()) - both) < 2 * five2


def test_rng_on_the_device(cuda_lib):
    """{seed, offset} read from the device at run time, in a captured graph too."""
    T, H = 33, 200
    y = _randn(_gen(3), T, H)
    Y, out = _c(y), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    hat = torch.empty_like(out)
    ws = cuda_lib.alloc_workspace(cuda_lib.et_layer_norm_workspace_bytes(T, H))
    rng = torch.tensor([77, 5], dtype=torch.int64, device="cuda")

    def step():
        cuda_lib.et_dropout(None, Y, out, p=0.4, d_rng=rng, workspace=ws)
        cuda_lib.et_layer_norm(Y, Y, None, hat, eps=1e-5, p=0.4, d_rng=rng, workspace=ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for off in (5, 6, 1 << 40):
        rng[1] = off
        graph.replay()
        check(out, ref.residual(None, y, 0.4, 77, off), ref.bf16_bound(y.double() * 2, 2 * U * y.double().abs() * 2), "out")
        z = ref.residual(y, y, 0.4, 77, off)
        want, n, r = ref.layer_norm(z)
        e, _ = ref.norm_error(y, y, 2.0, z, n, r)
        check(hat, want, ref.bf16_bound(want, e + 2 * U * n.abs()), "hat")


# ------------------------------------------------------------------ layer norm

SHAPES = [(1, 1), (1, 8), (2, 3), (5, 32), (33, 256), (9, 255), (12, 257), (40, 264), (7, 512), (300, 520), (64, 1000), (31, 1001),
          (20, 2048), (6, 2049), (700, 4096), (9, 4104), (3, 8192), (4, 8191), (2, 8200), (3, 16384), (2, 16383)]


def _run(E, x, y, gamma, beta, p, dxo, dh, shift=0, T=None, d_T=None, ws=None, want_dy=True, in_place=False):
    Tm, H = x.shape
    ws = ws if ws is not None else E.alloc_workspace(E.et_layer_norm_workspace_bytes(Tm, H))
    t = dict(x=_off(x, shift), y=_off(y, shift), gamma=_off(gamma, shift), beta=_off(beta, shift), dxo=_off(dxo, shift), dh=_off(dh, shift))
    seven = torch.full((Tm, H), 7.0, dtype=torch.bfloat16)
    o = {n: _off(seven, shift) for n in ("x_out", "x_hat", "dx", "dy")}
    if y is None or not want_dy:
        o["dy"] = None
    o["dg"] = None if gamma is None else torch.full((H,), 7.0, device="cuda")
    o["db"] = torch.full((H,), 7.0, device="cuda")
    how = dict(eps=1e-5, p=p, seed=SEED, offset=OFFSET, T=T, d_T=d_T, workspace=ws)
    E.et_layer_norm(t["x"], t["y"], o["x_out"], o["x_hat"], gamma=t["gamma"], beta=t["beta"], **how)
    if in_place:
        o["dx"], o["dy"] = t["dxo"], t["y"]
    E.et_layer_norm_bwd(t["x"], t["y"], t["dxo"], t["dh"], o["dx"], o["dy"], gamma=t["gamma"], d_gamma=o["dg"], d_beta=o["db"], **how)
    return o, ws


def _check(o, x, y, gamma, beta, p, dxo, dh, T=None):
    T = x.shape[0] if T is None else T
    x, y, dxo, dh = (None if v is None else v[:T] for v in (x, y, dxo, dh))
    k, mul = (None, 1.0) if y is None else ref.keep(*y.shape, p, SEED, OFFSET)
    z = ref.residual(x, y, p, SEED, OFFSET)
    want, n, r = ref.layer_norm(z, gamma, beta)
    mag = x.double().abs() + (0.0 if y is None else y.double().abs() * mul)
    check(o["x_out"][:T], z, ref.bf16_bound(z, 2 * U * mag), "x_out")
    e_n, rel_r = ref.norm_error(x, y, mul, z, n, r)
    g = 1.0 if gamma is None else gamma.double().abs()
    e = e_n * g + 2 * U * (n.abs() * g + (0.0 if beta is None else beta.double().abs()))
    check(o["x_hat"][:T], want, ref.bf16_bound(want, e), "x_hat")
    D, dg, db = ref.layer_norm_grad(z, n, r, gamma, dxo, dh)
    eD, eg, eb = ref.layer_norm_grad_bounds(n, r, e_n, rel_r, gamma, dxo, dh)
    check(o["dx"][:T], D, ref.bf16_bound(D, eD), "dx")
    if o["dy"] is not None:
        check(o["dy"][:T], torch.where(k, D * mul, 0.0), ref.bf16_bound(D * mul, (eD + U * D.abs()) * mul), "dy")
    if o["dg"] is not None:
        check(o["dg"], dg, eg + 2.0 ** -126, "d_gamma")
    check(o["db"], db, eb + 2.0 ** -126, "d_beta")


def _inputs(T, H, seed, with_y=True, affine=True, dxo=True):
    g = _gen(seed)
    x, dh = _randn(g, T, H), _randn(g, T, H)
    return (x, _randn(g, T, H, scale=2.0) if with_y else None, _randn(g, H, scale=0.2, add=1.0) if affine else None,
            _randn(g, H, scale=0.2) if affine else None, _randn(g, T, H) if dxo else None, dh)


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("p,with_y,affine,dxo", [(0.1, True, True, True), (0.0, False, True, False), (0.5, True, False, False), (0.0, True, True, True)])
def test_layer_norm(cuda_lib, T, H, p, with_y, affine, dxo):
    x, y, gamma, beta, d, dh = _inputs(T, H, T * 7 + H, with_y, affine, dxo)
    for shift in (0, 1):
        o, ws = _run(cuda_lib, x, y, gamma, beta, p, d, dh, shift=shift)
        _check(o, x, y, gamma, beta, p, d, dh)
        o2, _ = _run(cuda_lib, x, y, gamma, beta, p, d, dh, shift=shift, ws=ws)
        assert all(o[n] is None or torch.equal(o[n], o2[n]) for n in o)
    assert cuda_lib.et_status(ws) == (0, 0)


@pytest.mark.parametrize("H", [64, 250, 600, 4096])
def test_in_place_and_optional_outputs(cuda_lib, H):
    x, y, gamma, beta, d, dh = _inputs(21, H, H)
    a, ws = _run(cuda_lib, x, y, gamma, beta, 0.2, d, dh)
    b, _ = _run(cuda_lib, x, y, gamma, beta, 0.2, d, dh, in_place=True)  # dx over d_x_out, dy over y
    assert all(torch.equal(a[n], b[n]) for n in a)
    X = _c(x)
    hat = torch.empty_like(X)
    cuda_lib.et_layer_norm(X, _c(y), X, hat, gamma=_c(gamma), beta=_c(beta), eps=1e-5, p=0.2, seed=SEED, offset=OFFSET, workspace=ws)
    assert torch.equal(X, a["x_out"]) and torch.equal(hat, a["x_hat"])
    dx = torch.empty_like(X)
    cuda_lib.et_layer_norm_bwd(_c(x), _c(y), _c(d), _c(dh), dx, None, gamma=_c(gamma), eps=1e-5, p=0.2, seed=SEED, offset=OFFSET,
                               workspace=ws)  # no dy, no parameter gradients
    assert torch.equal(dx, a["dx"])


def test_constant_and_extreme_rows(cuda_lib):
    """Rows without deviation (all equal, all zero), a large mean, one far element, the smallest and large values."""
    T, H = 8, 384
    x, _, gamma, beta, d, dh = _inputs(T, H, 5, with_y=False)
    x[0] = 0
    x[1] = 3.0
    x[2] = (x[2].float() + 100).bfloat16()
    x[3, 5] = 1000.0
    x[4] = x[4] * 2.0 ** -100
    x[5] = (x[5].float() * 2.0 ** 50).bfloat16()
    o, _ = _run(cuda_lib, x, None, gamma, beta, 0.0, d, dh)
    _check(o, x, None, gamma, beta, 0.0, d, dh)
    assert torch.equal(o["x_hat"][0].cpu(), beta) and torch.equal(o["x_hat"][1].cpu(), beta)


def test_nan_stays_in_its_row(cuda_lib):
    x, y, gamma, beta, d, dh = _inputs(6, 520, 6)
    ref_o, _ = _run(cuda_lib, x, y, gamma, beta, 0.0, d, dh)
    x = x.clone()
    x[2, 100], x[4, 7] = math.nan, math.inf
    o, _ = _run(cuda_lib, x, y, gamma, beta, 0.0, d, dh)
    keep = [0, 1, 3, 5]
    for n in ("x_out", "x_hat", "dx", "dy"):
        assert torch.equal(o[n][keep], ref_o[n][keep])
        assert n == "x_out" or (torch.isnan(o[n][2]).any() and torch.isnan(o[n][4]).any())


@pytest.mark.parametrize("T,H", [(200000, 8), (90000, 33), (40000, 300)])
def test_long_batches(cuda_lib, T, H):
    """More rows than a thread adds up in one chain: the parameter gradients of equal rows stay exact to their bound."""
    g = _gen(H)
    row, dh = _randn(g, 1, H), _randn(g, 1, H)
    x, d = row.expand(T, H).contiguous(), dh.expand(T, H).contiguous()
    ws = cuda_lib.alloc_workspace(cuda_lib.et_layer_norm_workspace_bytes(T, H))
    dg, db, dx = torch.empty(H, device="cuda"), torch.empty(H, device="cuda"), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    gamma = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    cuda_lib.et_layer_norm_bwd(_c(x), None, None, _c(d), dx, None, gamma=gamma, eps=1e-5, d_gamma=dg, d_beta=db, workspace=ws)
    z = row.double()
    _, n, r = ref.layer_norm(z)
    e_n, _ = ref.norm_error(row, None, 1.0, z, n, r)
    # chains of at most 256 rows, of T / 256 / 300 such sums, 10 and 5: T / 76800 + 271 roundings
    adds = (T // 76800 + 280) * U
    check(db, T * dh.double()[0], adds * T * dh.double()[0].abs(), "d_beta")
    m = T * dh.double()[0].abs()
    check(dg, T * (dh.double() * n)[0], m * e_n[0] + adds * m * (n.abs() + e_n)[0], "d_gamma")


def test_device_count(cuda_lib):
    T, H = 40, 136
    x, y, gamma, beta, d, dh = _inputs(T, H, 9)
    dT = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = cuda_lib.alloc_workspace(cuda_lib.et_layer_norm_workspace_bytes(T, H))
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    for n in (40, 1, 0, 17):
        for dev in (True, False):
            dT.fill_(n)
            o, _ = _run(cuda_lib, x, y, gamma, beta, 0.3, d, dh, ws=ws, **(dict(d_T=dT) if dev else dict(T=n)))
            if n:
                _check(o, x, y, gamma, beta, 0.3, d, dh, T=n)
            else:
                assert (o["dg"] == 0).all() and (o["db"] == 0).all()
            assert all((o[v][n:] == 7).all() for v in ("x_out", "x_hat", "dx", "dy"))
            out.fill_(7)
            cuda_lib.et_dropout(_c(x), _c(y), out, p=0.3, workspace=ws, **(dict(d_T=dT) if dev else dict(T=n)))
            assert (out[n:] == 7).all() and (n == 0 or not (out[:n] == 7).all())
    for n in (41, -1):
        dT.fill_(n)
        o, _ = _run(cuda_lib, x, y, gamma, beta, 0.3, d, dh, ws=ws, d_T=dT)
        assert all((o[v] == 7).all() for v in o)
        assert cuda_lib.et_status(ws)[0] == cuda_lib.ET_ERR_BOUNDS
        cuda_lib.et_reset_status(ws)
        out.fill_(7)
        cuda_lib.et_dropout(None, _c(y), out, p=0.3, workspace=ws, d_T=dT)
        assert (out == 7).all() and cuda_lib.et_status(ws)[0] == cuda_lib.ET_ERR_BOUNDS
        cuda_lib.et_reset_status(ws)


def test_gradient_against_differences(cuda_lib):
    """dx, dy and the parameters' gradients along random directions against differences of the 64-bit forward."""
    T, H, p = 6, 40, 0.25
    x, y, gamma, beta, d, dh = _inputs(T, H, 11)
    o, _ = _run(cuda_lib, x, y, gamma, beta, p, d, dh)
    k, mul = ref.keep(T, H, p, SEED, OFFSET)

    def f(x, y, gamma, beta):
        z = x + torch.where(k, y * mul, torch.zeros_like(y))
        hat, _, _ = ref.layer_norm(z, gamma, beta)
        return (z * d.double()).sum() + (hat * dh.double()).sum()
    at = [v.double() for v in (x, y, gamma, beta)]
    grads = [o[n].double().cpu() for n in ("dx", "dy", "dg", "db")]
    for s in range(4):
        v = [torch.randn(t.shape, generator=_gen(30 + s), dtype=torch.float64) for t in at]
        h = 1e-6
        num = (f(*[a + h * b for a, b in zip(at, v)]) - f(*[a - h * b for a, b in zip(at, v)])) / (2 * h)
        got = sum((gr * b).sum() for gr, b in zip(grads, v))
        # dx and dy are rounded to bf16: 2^-8 of each entry, signs at random but counted in full; the rest is far below
        slack = sum(float((gr.abs() * b.abs()).sum()) for gr, b in zip(grads[:2], v[:2])) * 2.0 ** -8
        assert abs(float(num - got)) <= slack + 1e-3
