"""et_block_norm and its gradient on the GPU against the 64-bit definitions."""
import itertools

import pytest
import torch

from tests import ref_ops as ref

pytestmark = pytest.mark.gpu
U, B = ref.F32_HALF, ref.BF16_HALF
EPS = 1e-5


def _inputs(T, H, gate, post, pre, y, seed, device="cuda", offset=0):
    """bf16 inputs; `offset` elements into a larger buffer (another alignment)."""
    g = torch.Generator().manual_seed(seed)

    def rn(*s, mean=0.0, std=1.0, dtype=torch.bfloat16):
        v = (mean + std * torch.randn(*s, generator=g)).to(dtype)
        buf = torch.zeros(v.numel() + offset, dtype=dtype, device=device)
        buf[offset:] = v.reshape(-1).to(device)
        return buf[offset:].view(*s)
    d = dict(x=rn(T, H), y=rn(T, H, std=2.0) if y else None, gamma_post=rn(H, mean=1.0, std=0.1) if post else None,
             gamma_pre=rn(H, mean=1.0, std=0.1) if pre else None, d_x_out=rn(T, H), d_x_hat=rn(T, H) if pre else None)
    d["gate"] = {"none": lambda: None, "channel": lambda: rn(H, mean=0.5, std=0.3),
                 "token": lambda: rn(T, mean=0.5, std=0.3, dtype=torch.float32), "full": lambda: rn(T, H, mean=0.5, std=0.3)}[gate]()
    return d


def _ref(d, gate, scale, T, back=True):
    """64-bit values, gradients and the magnitudes for their bounds, of the first T rows."""
    L = {n: (None if d[n] is None else d[n].double().cpu()) for n in ("x", "y", "gamma_post", "gamma_pre", "gate", "d_x_out", "d_x_hat")}
    for n in ("x", "y", "d_x_out", "d_x_hat"):
        L[n] = None if L[n] is None else L[n][:T].clone()
    if gate == "token":
        L["gate"] = L["gate"][:T, None].clone()
    elif gate == "full":
        L["gate"] = L["gate"][:T].clone()
    leaves = [n for n in ("x", "y", "gamma_post", "gamma_pre", "gate") if L[n] is not None]
    for n in leaves:
        L[n].requires_grad_(True)
    z, hat = ref.block_norm(L["x"], L["y"], L["gamma_post"], L["gate"], scale, L["gamma_pre"], EPS)
    total = (0 if L["d_x_out"] is None else (z * L["d_x_out"]).sum()) + (0 if hat is None or L["d_x_hat"] is None else (hat * L["d_x_hat"]).sum())
    grads = dict(zip(leaves, torch.autograd.grad(total, [L[n] for n in leaves], allow_unused=True))) if back else {}
    a = {n: (None if L[n] is None else L[n].detach()) for n in L}
    zmag = a["x"].abs()
    n_ = None
    ry = 1.0
    if a["y"] is not None:
        n_ = a["y"]
        if a["gamma_post"] is not None:
            ry = 1 / torch.sqrt((n_ * n_).mean(-1, keepdim=True) + EPS)
            n_ = n_ * ry * a["gamma_post"]
        zmag = zmag + abs(scale) * (n_ if a["gate"] is None else a["gate"] * n_).abs()
    z = z.detach()
    rz = 1 / torch.sqrt((z * z).mean(-1, keepdim=True) + EPS) if a["gamma_pre"] is not None else None
    return L, grads, a, z, (None if hat is None else hat.detach()), zmag, n_, ry, rz


# fp32 roundings on the way: a handful per value, a sum's depth (16 columns a thread, 5 + 5 levels of the
# tree) in a statistic, whose error reaches a value by a factor of at most 1; what the rounding of z moves in
# mean(z^2) is at most 2 mean(|z| zmag): all covered by 64 roundings of the magnitudes below.
N = 64 * U


def _run_case(E, T, H, gate, post, pre, y, scale, seed, offset=0, T_used=None, d_T=None, back=True, ws=None):
    d = _inputs(T, H, gate, post, pre, y, seed, offset=offset)
    n = T if T_used is None else T_used
    ws = ws if ws is not None else E.alloc_workspace(E.et_block_norm_workspace_bytes(T, H))
    xo = torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda")
    xh = torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda") if pre else None
    kw = dict(gamma_post=d["gamma_post"], gate=d["gate"], scale=scale, gamma_pre=d["gamma_pre"], eps=EPS, workspace=ws,
              T=None if d_T is not None else T_used, d_T=d_T)
    E.et_block_norm(d["x"], d["y"], xo, xh, **kw)
    L, grads, a, z, hat, zmag, nn, ry, rz = _ref(d, gate, scale, n, back)
    ref.check(xo[:n], z, B * z.abs() + N * zmag + 1e-38, "x_out")
    assert (xo[n:] == 7).all()
    if pre:
        hmag = (rz * a["gamma_pre"]).abs() * (zmag + z.abs() * (zmag * z.abs()).mean(-1, keepdim=True) * rz * rz)
        ref.check(xh[:n], hat, B * hat.abs() + N * hmag + 1e-38, "x_hat")
        assert (xh[n:] == 7).all()
    if not back:
        return
    o = dict(dx=torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda"),
             dy=torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda") if y else None,
             d_gamma_post=torch.full((H,), 7.0, device="cuda") if post else None,
             d_gamma_pre=torch.full((H,), 7.0, device="cuda") if pre else None,
             d_gate={"none": None, "channel": torch.full((H,), 7.0, device="cuda"), "token": torch.full((T,), 7.0, device="cuda"),
                     "full": torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda")}[gate])
    E.et_block_norm_bwd(d["x"], d["y"], d["d_x_out"], d["d_x_hat"], o["dx"], o["dy"], d_gamma_post=o["d_gamma_post"],
                        d_gamma_pre=o["d_gamma_pre"], d_gate=o["d_gate"], **kw)
    # magnitudes: dz = d_x_out + rz gp dh - z k2,  k2 = mean(gp dh z) rz^3
    dmag = torch.zeros_like(z) if a["d_x_out"] is None else a["d_x_out"].abs()
    if pre:
        ah = (a["d_x_hat"] * a["gamma_pre"]).abs()
        # zmag / |z| is what cancellation in z costs the statistics
        cond = 1 + (zmag * z.abs()).mean(-1, keepdim=True) * rz * rz
        dmag = dmag + cond * rz * ah + (z.abs() + zmag) * cond * (ah * (z.abs() + zmag)).mean(-1, keepdim=True) * rz ** 3
    ref.check(o["dx"][:n], grads["x"], B * grads["x"].abs() + N * dmag + 1e-38, "dx")
    assert (o["dx"][n:] == 7).all()
    rows = (n + 64) * U
    if pre:
        m = (a["d_x_hat"] * rz).abs() * (zmag + z.abs() * cond)
        ref.check(o["d_gamma_pre"], grads["gamma_pre"], (rows + N) * m.sum(0) + 1e-38, "d_gamma_pre")
    if not y:
        return
    ga = 1.0 if a["gate"] is None else a["gate"].abs()
    dn = abs(scale) * ga * dmag
    if post:
        b = dn * a["gamma_post"].abs()
        ymag = ry * b + a["y"].abs() * (b * a["y"].abs()).mean(-1, keepdim=True) * ry ** 3
        ref.check(o["d_gamma_post"], grads["gamma_post"], (rows + N) * (dn * a["y"].abs() * ry).sum(0) + 1e-38, "d_gamma_post")
    else:
        ymag = dn
    ref.check(o["dy"][:n], grads["y"], B * grads["y"].abs() + N * ymag + 1e-38, "dy")
    assert (o["dy"][n:] == 7).all()
    gm = abs(scale) * nn.abs() * dmag
    if gate == "channel":
        ref.check(o["d_gate"], grads["gate"], (rows + N) * gm.sum(0) + 1e-38, "d_gate")
    elif gate == "token":
        ref.check(o["d_gate"][:n], grads["gate"][:, 0], 2 * N * gm.sum(-1) + 1e-38, "d_gate")
        assert (o["d_gate"][n:] == 7).all()
    elif gate == "full":
        ref.check(o["d_gate"][:n], grads["gate"], B * grads["gate"].abs() + N * gm + 1e-38, "d_gate")
        assert (o["d_gate"][n:] == 7).all()
    return o


SHAPES = [(1, 1), (1, 4096), (3, 7), (2, 8), (5, 31), (9, 256), (8, 257), (17, 264), (33, 1000), (700, 128), (1300, 520),
          (40, 2048), (12, 4104), (6, 5003), (20, 8192), (3, 8200), (2, 16384), (3, 16383)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
def test_block_norm(cuda_lib, T, H, gate):
    _run_case(cuda_lib, T, H, gate, True, True, True, 0.5, seed=T + H)


@pytest.mark.parametrize("post,pre,y", [c for c in itertools.product([False, True], repeat=3) if c[2] or not c[0]])
@pytest.mark.parametrize("H", [96, 1027])
def test_parts(cuda_lib, post, pre, y, H):
    """Every combination of the optional parts."""
    for gate in (["none", "token"] if y else ["none"]):
        _run_case(cuda_lib, 11, H, gate, post, pre, y, -1.5, seed=5)


@pytest.mark.parametrize("offset", [1, 3, 8])
def test_other_alignment(cuda_lib, offset):
    """Inputs that start off a 16-byte boundary."""
    for H in (64, 512, 77):
        _run_case(cuda_lib, 9, H, "full", True, True, True, 1.0, seed=7, offset=offset)


@pytest.mark.parametrize("T,H,offset", [(4000, 33, 0), (1500, 1001, 0), (1500, 1001, 1), (1500, 1000, 3), (700, 4099, 5)])
@pytest.mark.parametrize("gate", ["token", "channel", "full"])
def test_many_rows_off_alignment(cuda_lib, T, H, offset, gate):
    """Rows of odd width, or that start off a 16-byte boundary, with several for each thread group to take in turn."""
    _run_case(cuda_lib, T, H, gate, True, True, True, 0.5, seed=H, offset=offset)


@pytest.mark.parametrize("H", [129, 1001])
def test_in_place_off_alignment(cuda_lib, H):
    """dx over d_x_out and dy over y where rows share 16-byte pieces with their neighbours."""
    T = 1200
    d = _inputs(T, H, "full", True, True, True, 4)
    ws = cuda_lib.alloc_workspace(cuda_lib.et_block_norm_workspace_bytes(T, H))
    kw = dict(gamma_post=d["gamma_post"], gate=d["gate"], scale=0.7, gamma_pre=d["gamma_pre"], eps=EPS, workspace=ws)
    res = []
    for place in (False, True, True):
        y2, dz2 = d["y"].clone(), d["d_x_out"].clone()
        dx, dy = (dz2, y2) if place else (torch.empty_like(y2), torch.empty_like(y2))
        dg, dgf = torch.empty(H, device="cuda"), torch.empty_like(y2)
        cuda_lib.et_block_norm_bwd(d["x"], y2, dz2, d["d_x_hat"], dx, dy, d_gamma_post=dg, d_gate=dgf, **kw)
        res.append((dx, dy, dg, dgf))
    for got in res[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got, res[0]))


def test_one_gradient_missing(cuda_lib):
    """No gradient into x_out, or none into x_hat."""
    T, H = 9, 320
    for lost in ("d_x_out", "d_x_hat"):
        d = _inputs(T, H, "none", True, True, True, 3)
        d[lost] = None
        ws = cuda_lib.alloc_workspace(cuda_lib.et_block_norm_workspace_bytes(T, H))
        dx, dy, dgr = torch.empty_like(d["x"]), torch.empty_like(d["x"]), torch.full((H,), 7.0, device="cuda")
        cuda_lib.et_block_norm_bwd(d["x"], d["y"], d["d_x_out"], d["d_x_hat"], dx, dy, gamma_post=d["gamma_post"],
                                   gamma_pre=d["gamma_pre"], eps=EPS, d_gamma_pre=dgr, workspace=ws)
        L, grads, a, *_ = _ref(d, "none", 1.0, T)
        top = float(grads["x"].abs().max())
        ref.check(dx, grads["x"], B * grads["x"].abs() + 64 * N * top, "dx")
        ref.check(dy, grads["y"], B * grads["y"].abs() + 64 * N * top, "dy")
        if lost == "d_x_hat":
            assert (dgr == 0).all()


def test_zero_rows_and_zero_tokens(cuda_lib):
    """All-zero rows stay finite; T = 0 leaves rows as they were and gives zero parameter gradients."""
    T, H = 4, 128
    d = _inputs(T, H, "channel", True, True, True, 9)
    d["x"][1] = 0
    d["y"][1:3] = 0
    ws = cuda_lib.alloc_workspace(cuda_lib.et_block_norm_workspace_bytes(T, H))
    kw = dict(gamma_post=d["gamma_post"], gate=d["gate"], gamma_pre=d["gamma_pre"], eps=EPS, workspace=ws)
    xo, xh = torch.empty_like(d["x"]), torch.empty_like(d["x"])
    cuda_lib.et_block_norm(d["x"], d["y"], xo, xh, **kw)
    assert (xo[1] == 0).all() and (xh[1] == 0).all() and torch.equal(xo[2], d["x"][2])
    dx, dy = torch.full_like(xo, 7.0), torch.full_like(xo, 7.0)
    ps = [torch.full((H,), 7.0, device="cuda") for _ in range(3)]
    cuda_lib.et_block_norm_bwd(d["x"], d["y"], d["d_x_out"], d["d_x_hat"], dx, dy, d_gamma_post=ps[0], d_gamma_pre=ps[1],
                               d_gate=ps[2], **kw)
    assert all(torch.isfinite(t).all() for t in (dx, dy, *ps))
    for T_, d_T in ((0, None), (None, torch.zeros(1, dtype=torch.int32, device="cuda"))):
        dx.fill_(7), dy.fill_(7)
        cuda_lib.et_block_norm_bwd(d["x"], d["y"], d["d_x_out"], d["d_x_hat"], dx, dy, d_gamma_post=ps[0], d_gamma_pre=ps[1],
                                   d_gate=ps[2], T=T_, d_T=d_T, **kw)
        assert (dx == 7).all() and (dy == 7).all() and all((t == 0).all() for t in ps)


def test_device_count(cuda_lib):
    T, H = 400, 136
    dT = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = cuda_lib.alloc_workspace(cuda_lib.et_block_norm_workspace_bytes(T, H))
    for n in (400, 1, 63):
        dT.fill_(n)
        _run_case(cuda_lib, T, H, "channel", True, True, True, 0.5, seed=n, T_used=n, d_T=dT, ws=ws)
    for n in (401, -3):
        dT.fill_(n)
        d = _inputs(T, H, "none", True, True, True, 1)
        xo = torch.full_like(d["x"], 7.0)
        dg = torch.full((H,), 7.0, device="cuda")
        cuda_lib.et_block_norm(d["x"], d["y"], xo, None, gamma_post=d["gamma_post"], eps=EPS, d_T=dT, workspace=ws)
        assert (xo == 7).all() and cuda_lib.et_status(ws)[0] == cuda_lib.ET_ERR_BOUNDS
        cuda_lib.et_reset_status(ws)
        cuda_lib.et_block_norm_bwd(d["x"], d["y"], d["d_x_out"], None, xo, xo.clone(), gamma_post=d["gamma_post"], eps=EPS,
                                   d_gamma_post=dg, d_T=dT, workspace=ws)
        assert (xo == 7).all() and (dg == 7).all() and cuda_lib.et_status(ws)[0] == cuda_lib.ET_ERR_BOUNDS
        cuda_lib.et_reset_status(ws)


def test_in_place_and_same_bits(cuda_lib):
    """x_out over x, dx over d_x_out, dy over y; a second run gives the same bits."""
    T, H = 900, 768
    d = _inputs(T, H, "full", True, True, True, 4)
    ws = cuda_lib.alloc_workspace(cuda_lib.et_block_norm_workspace_bytes(T, H))
    kw = dict(gamma_post=d["gamma_post"], gate=d["gate"], scale=0.7, gamma_pre=d["gamma_pre"], eps=EPS, workspace=ws)
    xo, xh, xh2 = (torch.empty_like(d["x"]) for _ in range(3))
    cuda_lib.et_block_norm(d["x"], d["y"], xo, xh, **kw)
    x2 = d["x"].clone()
    cuda_lib.et_block_norm(x2, d["y"], x2, xh2, **kw)
    assert torch.equal(x2, xo) and torch.equal(xh2, xh)
    res = []
    for _ in range(2):
        y2, dz2 = d["y"].clone(), d["d_x_out"].clone()
        ps = [torch.empty(H, device="cuda") for _ in range(2)]
        dgf = torch.empty_like(xo)
        cuda_lib.et_block_norm_bwd(d["x"], y2, dz2, d["d_x_hat"], dz2, y2, d_gamma_post=ps[0], d_gamma_pre=ps[1], d_gate=dgf, **kw)
        res.append((dz2, y2, *ps, dgf))
    dx, dy = torch.empty_like(xo), torch.empty_like(xo)
    ps = [torch.empty(H, device="cuda") for _ in range(2)]
    dgf = torch.empty_like(xo)
    cuda_lib.et_block_norm_bwd(d["x"], d["y"], d["d_x_out"], d["d_x_hat"], dx, dy, d_gamma_post=ps[0], d_gamma_pre=ps[1], d_gate=dgf, **kw)
    for got in res:
        assert all(torch.equal(a, b) for a, b in zip(got, (dx, dy, *ps, dgf)))


def test_streams_and_graph(cuda_lib):
    """Forward and backward captured once, replayed with other inputs; and a call on a side stream."""
    T, H = 50, 640
    d = _inputs(T, H, "channel", True, True, True, 4)
    ws = cuda_lib.alloc_workspace(cuda_lib.et_block_norm_workspace_bytes(T, H))
    kw = dict(gamma_post=d["gamma_post"], gate=d["gate"], gamma_pre=d["gamma_pre"], eps=EPS, workspace=ws)
    outs = [torch.empty_like(d["x"]) for _ in range(4)] + [torch.empty(H, device="cuda") for _ in range(3)]

    def step(o, stream=None):
        cuda_lib.et_block_norm(d["x"], d["y"], o[0], o[1], stream=stream, **kw)
        cuda_lib.et_block_norm_bwd(d["x"], d["y"], d["d_x_out"], d["d_x_hat"], o[2], o[3], d_gamma_post=o[4], d_gamma_pre=o[5],
                                   d_gate=o[6], stream=stream, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step(outs, s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(outs)
    for seed in (5, 6):
        n = _inputs(T, H, "channel", True, True, True, seed)
        for key in ("x", "y", "d_x_out", "d_x_hat"):
            d[key].copy_(n[key])
        g.replay()
        torch.cuda.synchronize()
        want = [torch.empty_like(t) for t in outs]
        step(want)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_gradient_against_differences(cuda_lib):
    """The kernel's gradients along random directions against differences of the 64-bit forward."""
    T, H = 5, 40
    d = _inputs(T, H, "channel", True, True, True, 8)
    ws = cuda_lib.alloc_workspace(cuda_lib.et_block_norm_workspace_bytes(T, H))
    dx, dy = torch.empty_like(d["x"]), torch.empty_like(d["x"])
    ps = [torch.empty(H, device="cuda") for _ in range(3)]
    cuda_lib.et_block_norm_bwd(d["x"], d["y"], d["d_x_out"], d["d_x_hat"], dx, dy, gamma_post=d["gamma_post"], gate=d["gate"],
                               scale=0.5, gamma_pre=d["gamma_pre"], eps=EPS, d_gamma_post=ps[0], d_gamma_pre=ps[1], d_gate=ps[2],
                               workspace=ws)
    a = {k: v.double().cpu() for k, v in d.items()}

    def f(**over):
        b = dict(a, **over)
        z, hat = ref.block_norm(b["x"], b["y"], b["gamma_post"], b["gate"], 0.5, b["gamma_pre"], EPS)
        return (z * a["d_x_out"]).sum() + (hat * a["d_x_hat"]).sum()
    h = 1e-6
    for name, grad in (("x", dx), ("y", dy), ("gamma_post", ps[0]), ("gamma_pre", ps[1]), ("gate", ps[2])):
        gd = grad.double().cpu()
        for s in range(3):
            v = torch.randn(gd.shape, generator=torch.Generator().manual_seed(s), dtype=torch.float64)
            num = (f(**{name: a[name] + h * v}) - f(**{name: a[name] - h * v})) / (2 * h)
            # bf16 gradients carry half a step each
            assert abs(float(num - (gd * v).sum())) <= float((gd.abs() * v.abs()).sum()) * (B + 1e-4) + 1e-5
