"""The router, norm and 4-bit weight calls without a GPU: workspace sizes, refusals by the C ABI before any
device work, refusals by the binding, and the 64-bit references against differences and hand values."""
import math

import pytest
import torch

from moe_task_scheduling_gb300 import etmoe as E
from tests import ref_ops as ref


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return E.load()


# ------------------------------------------------------------------ sizes and refusals of the C ABI

def test_workspace_sizes(lib):
    assert E.et_router_topk_workspace_bytes(1, 1, 1) >= 256
    assert E.et_router_topk_workspace_bytes(65536, 256, 8) % 256 == 0
    for bad in ((0, 8, 2), (16, 0, 1), (16, 257, 2), (16, 8, 9), (16, 2, 3), (16, 8, 0)):
        assert E.et_router_topk_workspace_bytes(*bad) == 0
    assert E.et_block_norm_workspace_bytes(1, 1) >= 256
    assert E.et_block_norm_workspace_bytes(4096, 4096) >= 256 + 3 * 4096 * 4
    assert E.et_block_norm_workspace_bytes(0, 8) == 0 and E.et_block_norm_workspace_bytes(4, 16385) == 0
    assert E.et_w4_gemv_workspace_bytes(64, 8, 32, 32) >= 256
    for bad in ((0, 8, 32, 32), (65, 8, 32, 32), (1, 9, 32, 32), (1, 8, 48, 32), (1, 8, 64, 48), (1, 8, 0, 32)):
        assert E.et_w4_gemv_workspace_bytes(*bad) == 0
    assert E.et_w4_experts_workspace_bytes(64, 256, 512, 8, 2, 128) >= 64 * 2 * 512 * 2
    for bad in ((65, 256, 512, 8, 2, 128), (4, 256, 512, 8, 9, 128), (4, 256, 480, 8, 2, 128), (4, 256, 512, 257, 2, 128)):
        assert E.et_w4_experts_workspace_bytes(*bad) == 0


def _with(base, over):
    return list(dict(base, **over).values())


ROUTER = dict(L=16, m=None, idx=16, w=16, c=None, n=None, P=None, ls=None, T=4, dT=None, Tm=16, E=8, k=2, ws=256,
              wsb=1 << 30, st=None)
ROUTER_BWD = dict(L=16, m=None, idx=16, w=16, c=16, n=16, dl=None, dw=None, d=16, T=4, dT=None, Tm=16, E=8, k=2,
                  ws=256, wsb=1 << 30, st=None)
NORM = dict(x=16, y=16, gp=16, g=None, kind=0, s=1.0, gr=16, eps=1e-5, xo=16, xh=16, T=2, dT=None, Tm=4, H=64,
            ws=256, wsb=1 << 30, st=None)
NORM_BWD = dict(x=16, y=16, gp=16, g=None, kind=0, s=1.0, gr=16, eps=1e-5, do=16, dh=16, dx=16, dy=16, dgp=None,
                dgr=None, dg=None, T=2, dT=None, Tm=4, H=64, ws=256, wsb=1 << 30, st=None)
GEMV = dict(X=16, q=16, s=16, Y=16, M=2, dM=None, Mm=4, N=64, K=128, G=32, ws=256, wsb=1 << 30, st=None)
EXPERTS = dict(x=16, idx=16, w=16, qg=16, sg=16, qu=16, su=16, qd=16, sd=16, out=16, T=2, dT=None, Tm=4, H=64, F=128,
               E=8, k=2, G=32, ws=256, wsb=1 << 30, st=None)
CONV = dict(w=16, q=16, s=16, E=1, N=8, K=64, G=32, st=None)

INV, UNS, WS = E.ET_ERR_INVALID, E.ET_ERR_UNSUPPORTED, E.ET_ERR_WORKSPACE
REFUSALS = [
    ("et_router_topk", ROUTER, [(dict(L=None), INV), (dict(idx=None), INV), (dict(w=None), INV), (dict(L=18), INV),
                                (dict(E=257), UNS), (dict(E=0), UNS), (dict(k=9), UNS), (dict(E=1), UNS),
                                (dict(k=0), UNS), (dict(T=17), INV), (dict(T=-1), INV), (dict(Tm=0), UNS),
                                (dict(ws=None), WS), (dict(ws=264), WS), (dict(wsb=256), WS), (dict(ls=2), INV)]),
    ("et_router_topk_bwd", ROUTER_BWD, [(dict(c=None), INV), (dict(n=None), INV), (dict(d=None), INV),
                                        (dict(dw=2), INV), (dict(E=300), UNS), (dict(T=17), INV), (dict(wsb=8), WS)]),
    ("et_block_norm", NORM, [(dict(x=None), INV), (dict(xo=None, xh=None, gr=None), INV), (dict(gr=None), INV),
                             (dict(xh=None), INV), (dict(kind=1), INV), (dict(g=16), INV), (dict(kind=4, g=16), INV),
                             (dict(y=None), INV), (dict(eps=0.0), INV), (dict(eps=math.nan), INV),
                             (dict(eps=math.inf), INV), (dict(s=math.inf), INV), (dict(H=0), UNS),
                             (dict(H=16385), UNS), (dict(T=5), INV), (dict(x=17), INV), (dict(kind=2, g=18), INV),
                             (dict(ws=None), WS), (dict(wsb=128), WS)]),
    ("et_block_norm_bwd", NORM_BWD, [(dict(dx=None), INV), (dict(dy=None), INV), (dict(y=None, gp=None), INV),
                                     (dict(do=None, dh=None), INV), (dict(gr=None), INV), (dict(gr=None, dh=None, dgr=16), INV),
                                     (dict(dg=16), INV), (dict(dgp=18), INV), (dict(wsb=256), WS), (dict(Tm=0), UNS)]),
    ("et_w4_gemv", GEMV, [(dict(X=None), INV), (dict(Y=8), INV), (dict(G=16), UNS), (dict(G=256), UNS),
                          (dict(K=120), UNS), (dict(K=0), UNS), (dict(N=60), UNS), (dict(N=0), UNS),
                          (dict(Mm=65), UNS), (dict(M=5), INV), (dict(M=-1), INV), (dict(ws=None), WS), (dict(wsb=0), WS),
                          (dict(dM=2), INV)]),
    ("et_w4_experts", EXPERTS, [(dict(idx=None), INV), (dict(w=None), INV), (dict(qu=None), INV), (dict(sd=8), INV),
                                (dict(Tm=65), UNS), (dict(E=257), UNS), (dict(k=9), UNS), (dict(E=1), UNS),
                                (dict(H=48), UNS), (dict(F=100), UNS), (dict(T=5), INV), (dict(idx=18), INV),
                                (dict(wsb=512), WS)]),
    ("et_w4_quantize", CONV, [(dict(w=None), INV), (dict(q=8), INV), (dict(G=8), UNS), (dict(K=72), UNS),
                              (dict(N=4), UNS), (dict(E=0), UNS)]),
    ("et_w4_dequantize", CONV, [(dict(s=None), INV), (dict(w=8), INV), (dict(G=0), UNS), (dict(N=12), UNS)]),
]


@pytest.mark.parametrize("name,base,over,code", [(n, b, o, c) for n, b, cases in REFUSALS for o, c in cases])
def test_refusals(lib, name, base, over, code):
    assert getattr(lib, name)(*_with(base, over)) == code
    assert lib.et_last_error_string() != b""


def test_nothing_to_do(lib):
    """A host count of 0 launches nothing where nothing is written."""
    assert lib.et_router_topk_bwd(*_with(ROUTER_BWD, dict(T=0))) == E.ET_OK
    assert lib.et_block_norm(*_with(NORM, dict(T=0))) == E.ET_OK
    assert lib.et_w4_gemv(*_with(GEMV, dict(M=0))) == E.ET_OK
    assert lib.et_w4_experts(*_with(EXPERTS, dict(T=0))) == E.ET_OK


# ------------------------------------------------------------------ refusals of the binding

def test_binding_refuses_wrong_tensors(lib):
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA device"):
        E.et_router_topk(torch.zeros(4, 8), torch.zeros(4, 2, dtype=i32), torch.zeros(4, 2), workspace=ws)
    with pytest.raises(ValueError, match="CUDA device"):
        E.et_w4_gemv(torch.zeros(4, 64, dtype=bf), ws, ws, torch.zeros(4, 8, dtype=bf), workspace=ws)
    for t, dt, sh, msg in ((torch.zeros(4, 8, dtype=bf), f32, (4, 8), "must be torch.float32"),
                           (torch.zeros(4, 7), f32, (4, 8), r"\(4, 8\)"),
                           (torch.zeros(8, 4).t(), f32, (4, 8), "contiguous"),
                           (torch.zeros(4, 8), f32, (4, 8), "must be on CUDA device 0")):
        with pytest.raises(ValueError, match=msg):
            E._arg(t, "logits", dt, sh, 0)
    assert E._arg(None, "gate", f32, (4,), 0) is None
    with pytest.raises(ValueError, match="workspace"):
        E._workspace_args(None, 0)
    with pytest.raises(ValueError, match="workspace"):
        E._workspace_args(ws, 0)
    with pytest.raises(ValueError, match="device count"):
        E._count_arg(torch.zeros(2, dtype=i32), 0)
    q = torch.zeros(4, 64, 32, dtype=torch.uint8)
    for s in (torch.zeros(64, dtype=bf), torch.zeros(4, 3, 64, dtype=bf), torch.zeros(4, 0, 64, dtype=bf)):
        with pytest.raises(ValueError, match="scale of q"):
            E._w4(q, s, "q", (4,), 64, 64, 0)


def test_call_runs_on_the_tensors_device(monkeypatch):
    """Tensors on a device that is not current: it is made current around the call, its stream is used."""
    import contextlib
    seen = []

    @contextlib.contextmanager
    def device(dev):
        seen.append(("enter", dev))
        yield
        seen.append(("exit", dev))
    monkeypatch.setattr(E, "_current_device", lambda: 0)
    monkeypatch.setattr(E, "_raw_stream", lambda dev: 100 + dev)
    monkeypatch.setattr(torch.cuda, "device", device)
    assert E._call(lambda *a: seen.append(a) or 0, 1, None, (7,), True) == 0
    assert seen == [("enter", 1), (7, 101), ("exit", 1)]
    seen.clear()
    assert E._call(lambda *a: seen.append(a) or 0, 0, 55, (7,), True) == 0
    assert seen == [(7, 55)]
    assert E._call(lambda *a: E.ET_ERR_CUDA, 0, 55, (), False) == E.ET_ERR_CUDA


# ------------------------------------------------------------------ the 64-bit references

def _differences(f, x, g, h=1e-6):
    """Directional central differences of f at x against the gradient g, along random directions."""
    gen = torch.Generator().manual_seed(11)
    for _ in range(4):
        v = torch.randn(x.shape, generator=gen, dtype=torch.float64)
        num = (f(x + h * v) - f(x - h * v)) / (2 * h)
        ana = (g * v).sum()
        assert abs(float(num - ana)) <= 1e-6 * (1 + abs(float(ana)))


@pytest.mark.parametrize("T,En,k", [(5, 8, 2), (3, 33, 8), (1, 1, 1)])
def test_router_reference(T, En, k):
    gen = torch.Generator().manual_seed(1)
    L = torch.randn(T, En, generator=gen, dtype=torch.float64)
    mask = torch.ones(T, dtype=torch.uint8)
    mask[T // 2] = T == 1
    dl, dw = torch.tensor([0.3, -0.2], dtype=torch.float64), torch.randn(T, k, generator=gen, dtype=torch.float64)
    r = ref.router(L, k, mask)
    assert r["n"] == int(mask.sum()) and int(r["counts"].sum()) == k * r["n"]

    def f(v):
        o = ref.router(v, k, mask)
        return (o["losses"] * dl).sum() + (o["w"] * dw * (o["idx"] >= 0)).sum()
    g = ref.router_grad(L, k, dl, dw, mask)
    _differences(f, L, g)
    # the written formula
    p, n = r["p"], r["n"]
    c = En * r["counts"] / (n * k) / n
    want = dl[0] * p * (c - (p * c).sum(-1, keepdim=True)) + dl[1] * 2 / n * r["lse"][:, None] * p
    ds = r["w"] * (dw - (r["w"] * dw).sum(-1, keepdim=True))
    want = want.scatter_add(1, r["idx"].clamp(min=0), torch.where(r["idx"] >= 0, ds, 0.0))
    assert torch.allclose(g, want, rtol=1e-12, atol=1e-12)


def test_router_reference_masks():
    ninf = -math.inf
    L = torch.tensor([[ninf, 1.0, ninf, ninf], [ninf] * 4, [0.0, -0.0, 0.0, 0.0]], dtype=torch.float64)
    r = ref.router(L, 2)
    assert r["idx"].tolist() == [[1, -1], [-1, -1], [0, 1]]
    assert r["w"].tolist() == [[1, 0], [0, 0], [0.5, 0.5]] and r["n"] == 2
    assert torch.isfinite(ref.router_grad(L, 2, torch.ones(2), torch.ones(3, 2))).all()


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
def test_norm_reference(gate):
    """The written gradient against differences of the 64-bit forward."""
    gen = torch.Generator().manual_seed(2)
    T, H = 3, 7
    rn = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, y, gp, gr, dz, dh = rn(T, H), rn(T, H), rn(H), rn(H), rn(T, H), rn(T, H)
    g = {"none": None, "channel": rn(H), "token": rn(T, 1), "full": rn(T, H)}[gate]
    leaves = [t.clone().requires_grad_(True) for t in (x, y, gp, gr)] + ([] if g is None else [g.clone().requires_grad_(True)])

    def total(x, y, gp, gr, g=None):
        z, hat = ref.block_norm(x, y, gp, g, 0.5, gr)
        return (z * dz).sum() + (hat * dh).sum()
    grads = torch.autograd.grad(total(*leaves), leaves)
    for i in range(len(leaves)):
        def f(v, i=i):
            a = [t.detach() for t in leaves]
            a[i] = v
            return total(*a)
        _differences(f, leaves[i].detach(), grads[i])


def test_w4_reference():
    """A hand value, the layout, ties and degenerate groups."""
    w = torch.zeros(8, 32)
    w[0, 0], w[0, 1], w[0, 3] = 7.0, -7.0, 2.5          # scale 1; 2.5 rounds to 2 (half to even)
    w[1, 2] = math.inf
    w[2, 5] = math.nan
    q, s = ref.w4_pack(w.to(torch.bfloat16), 32)
    assert q.shape == (8, 16) and s.shape == (1, 8)
    assert int(q[0, 0]) == 15 | (1 << 4) and int(q[0, 1]) == 8 | (10 << 4)
    assert float(s[0, 0]) == 1.0 and math.isnan(float(s[0, 1])) and math.isnan(float(s[0, 2])) and float(s[0, 3]) == 0
    assert (q[1:] == 0x88).all()
    v = ref.w4_values(q, s)
    assert v[0, :4].tolist() == [7, -7, 0, 2] and (v[3:] == 0).all()
