"""The grouped router, dropout, layer norm and int8 calls without a GPU: workspace sizes, refusals by the C ABI before any
device work, refusals by the binding, and the 64-bit references against known answers, library routines and differences."""
import math

import pytest
import torch

from moe_task_scheduling_gb300 import etmoe as E
from tests import ref_more as ref


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return E.load()


# ------------------------------------------------------------------ sizes and refusals of the C ABI

def test_workspace_sizes(lib):
    assert E.et_router_groups_workspace_bytes(65536, 256, 8) % 256 == 0 and E.et_router_groups_workspace_bytes(1, 1, 1) >= 256
    for bad in ((0, 8, 2), (16, 257, 2), (16, 8, 9), (16, 2, 3), (16, 8, 0), ((1 << 24) + 1, 8, 2)):
        assert E.et_router_groups_workspace_bytes(*bad) == 0
    assert E.et_dropout_workspace_bytes(1 << 24, 1 << 18) >= 256
    for bad in ((0, 8), (4, 0), (4, (1 << 18) + 1), ((1 << 24) + 1, 8)):
        assert E.et_dropout_workspace_bytes(*bad) == 0
    assert E.et_layer_norm_workspace_bytes(4096, 4096) >= 256 + 2 * 4096 * 4
    assert E.et_layer_norm_workspace_bytes(0, 8) == 0 and E.et_layer_norm_workspace_bytes(4, 16385) == 0
    assert E.et_i8_quantize_workspace_bytes(1 << 20, 65536) >= 256 and E.et_i8_gemm_workspace_bytes(1, 1, 16) >= 256
    for bad in ((0, 8, 32), (1, 0, 32), (1, 8, 24), (1, 8, 0), (1, 8, 65552), ((1 << 20) + 1, 8, 32), (1, (1 << 20) + 1, 32)):
        assert E.et_i8_gemm_workspace_bytes(*bad) == 0
    for bad in ((0, 32), (1, 8), (1 << 33, 32), (1, 65552)):
        assert E.et_i8_quantize_workspace_bytes(*bad) == 0


def _with(base, over):
    return list(dict(base, **over).values())


GROUPS = dict(L=16, b=None, m=None, score=1, G=4, kg=2, best=2, renorm=1, scale=1.0, idx=16, w=16, c=None, n=None, P=None, ls=None,
              T=4, dT=None, Tm=16, E=8, k=2, ws=256, wsb=1 << 30, st=None)
GROUPS_BWD = dict(L=16, m=None, score=1, renorm=1, scale=1.0, idx=16, w=16, c=16, n=16, dl=None, dw=None, d=16, T=4, dT=None, Tm=16,
                  E=8, k=2, ws=256, wsb=1 << 30, st=None)
DROP = dict(x=None, y=16, out=16, p=0.1, seed=1, off=2, rng=None, T=2, dT=None, Tm=4, H=64, ws=256, wsb=1 << 30, st=None)
LN = dict(x=16, y=16, g=16, b=16, eps=1e-5, p=0.1, seed=1, off=2, rng=None, xo=16, xh=16, T=2, dT=None, Tm=4, H=64, ws=256,
          wsb=1 << 30, st=None)
LN_BWD = dict(x=16, y=16, g=16, eps=1e-5, p=0.1, seed=1, off=2, rng=None, do=16, dh=16, dx=16, dy=16, dg=None, db=None, T=2, dT=None,
              Tm=4, H=64, ws=256, wsb=1 << 30, st=None)
QUANT = dict(x=16, q=16, s=16, M=2, dM=None, Mm=4, K=64, ws=256, wsb=1 << 30, st=None)
GEMM = dict(x=16, sx=16, w=16, sw=16, Y=16, M=2, dM=None, Mm=4, N=64, K=64, ws=256, wsb=1 << 40, st=None)

INV, UNS, WS = E.ET_ERR_INVALID, E.ET_ERR_UNSUPPORTED, E.ET_ERR_WORKSPACE
REFUSALS = [
    ("et_router_groups", GROUPS, [(dict(L=None), INV), (dict(idx=None), INV), (dict(w=None), INV), (dict(b=18), INV), (dict(E=257), UNS),
                                  (dict(k=9), UNS), (dict(k=0), UNS), (dict(score=2), INV), (dict(score=-1), INV), (dict(G=3), UNS),
                                  (dict(G=0), UNS), (dict(E=66, G=33), UNS), (dict(kg=0), UNS), (dict(kg=5), UNS), (dict(k=5), UNS),
                                  (dict(best=0), UNS), (dict(best=3), UNS), (dict(scale=math.nan), INV), (dict(scale=math.inf), INV),
                                  (dict(T=17), INV), (dict(T=-1), INV), (dict(Tm=0), UNS), (dict(ws=None), WS), (dict(ws=264), WS),
                                  (dict(wsb=256), WS), (dict(ls=2), INV)]),
    ("et_router_groups_bwd", GROUPS_BWD, [(dict(c=None), INV), (dict(n=None), INV), (dict(d=None), INV), (dict(dw=2), INV),
                                          (dict(E=300), UNS), (dict(score=7), INV), (dict(scale=math.inf), INV), (dict(T=17), INV),
                                          (dict(wsb=8), WS)]),
    ("et_dropout", DROP, [(dict(y=None), INV), (dict(out=None), INV), (dict(x=17), INV), (dict(p=1.0), INV), (dict(p=-0.1), INV),
                          (dict(p=math.nan), INV), (dict(rng=12), INV), (dict(T=5), INV), (dict(T=-1), INV), (dict(Tm=0), UNS),
                          (dict(H=0), UNS), (dict(H=(1 << 18) + 1), UNS), (dict(ws=None), WS), (dict(wsb=128), WS), (dict(dT=2), INV)]),
    ("et_layer_norm", LN, [(dict(x=None), INV), (dict(xh=None), INV), (dict(y=None), INV), (dict(eps=0.0), INV), (dict(eps=math.nan), INV),
                           (dict(eps=math.inf), INV), (dict(p=1.0), INV), (dict(p=math.nan), INV), (dict(p=-0.5), INV), (dict(H=0), UNS),
                           (dict(H=16385), UNS), (dict(T=5), INV), (dict(x=17), INV), (dict(b=17), INV), (dict(rng=4), INV),
                           (dict(ws=None), WS), (dict(wsb=128), WS)]),
    ("et_layer_norm_bwd", LN_BWD, [(dict(dx=None), INV), (dict(dh=None), INV), (dict(y=None, p=0.0), INV), (dict(g=None, dg=16), INV),
                                   (dict(dg=18), INV), (dict(db=2), INV), (dict(wsb=256), WS), (dict(Tm=0), UNS), (dict(p=2.0), INV)]),
    ("et_i8_quantize", QUANT, [(dict(x=None), INV), (dict(q=None), INV), (dict(s=None), INV), (dict(q=8), INV), (dict(x=17), INV),
                               (dict(K=24), UNS), (dict(K=0), UNS), (dict(K=65552), UNS), (dict(Mm=0), UNS), (dict(M=5), INV),
                               (dict(dM=2), INV), (dict(ws=None), WS), (dict(wsb=255), WS)]),
    ("et_i8_gemm", GEMM, [(dict(x=None), INV), (dict(sx=None), INV), (dict(w=None), INV), (dict(sw=None), INV), (dict(Y=None), INV),
                          (dict(x=8), INV), (dict(w=24), INV), (dict(Y=17), INV), (dict(sw=18), INV), (dict(K=24), UNS), (dict(K=0), UNS),
                          (dict(K=65552), UNS), (dict(N=0), UNS), (dict(N=(1 << 20) + 1), UNS), (dict(Mm=0), UNS), (dict(M=5), INV),
                          (dict(M=-1), INV), (dict(dM=2), INV), (dict(ws=None), WS), (dict(ws=264), WS), (dict(wsb=255), WS)]),
]


@pytest.mark.parametrize("name,base,over,code", [(n, b, o, c) for n, b, cases in REFUSALS for o, c in cases])
def test_refusals(lib, name, base, over, code):
    assert getattr(lib, name)(*_with(base, over)) == code
    assert lib.et_last_error_string() != b""


def test_nothing_to_do(lib):
    """A host count of 0 launches nothing where nothing is written."""
    assert lib.et_router_groups_bwd(*_with(GROUPS_BWD, dict(T=0))) == E.ET_OK
    assert lib.et_dropout(*_with(DROP, dict(T=0))) == E.ET_OK
    assert lib.et_layer_norm(*_with(LN, dict(T=0))) == E.ET_OK
    assert lib.et_i8_quantize(*_with(QUANT, dict(M=0))) == E.ET_OK
    assert lib.et_i8_gemm(*_with(GEMM, dict(M=0))) == E.ET_OK


# ------------------------------------------------------------------ refusals of the binding

def test_binding_refuses_wrong_tensors(lib):
    bf, f32, i32, i8 = torch.bfloat16, torch.float32, torch.int32, torch.int8
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    x = torch.zeros(4, 8, dtype=bf)
    with pytest.raises(ValueError, match="CUDA device"):
        E.et_router_groups(torch.zeros(4, 8), torch.zeros(4, 2, dtype=i32), torch.zeros(4, 2), score=1, workspace=ws)
    with pytest.raises(ValueError, match="CUDA device"):
        E.et_dropout(None, x, x, p=0.1, workspace=ws)
    with pytest.raises(ValueError, match="CUDA device"):
        E.et_layer_norm(x, None, None, x, eps=1e-5, workspace=ws)
    with pytest.raises(ValueError, match="CUDA device"):
        E.et_i8_quantize(x, torch.zeros(4, 8, dtype=i8), torch.zeros(4, dtype=f32), workspace=ws)
    with pytest.raises(ValueError, match="CUDA device"):
        E.et_i8_gemm(torch.zeros(4, 16, dtype=i8), torch.zeros(4), torch.zeros(8, 16, dtype=i8), torch.zeros(8), x, workspace=ws)
    for bad in ((-1, 0), (0, 1 << 64)):
        with pytest.raises(ValueError, match="seed and offset"):
            E._rng_args(0.1, *bad, None, 0)
    for bad in (torch.zeros(2), torch.zeros(3, dtype=torch.int64), torch.zeros(2, dtype=torch.int64)):
        with pytest.raises(ValueError, match="d_rng"):
            E._rng_args(0.1, 0, 0, bad, 0)
    assert E._rng_args(0.5, 3, 1 << 63, None, 0) == (0.5, 3, 1 << 63, None)


# ------------------------------------------------------------------ the references

def test_philox_known_answers():
    """The published vectors of Philox4x32-10."""
    for counter, key, want in (([0] * 4, [0] * 2, (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
                               ([0xffffffff] * 4, [0xffffffff] * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
                               ([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0],
                                (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))):
        assert tuple(int(v) for v in ref.philox(counter, key)) == want
    k, mul = ref.keep(3, 17, 0.5, 0xa4093822 | 0x299f31d0 << 32, 0x13198a2e | 0x03707344 << 32)
    assert mul == 2.0 and k.shape == (3, 17)
    w = [int(v) for v in ref.philox([2, 1, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0])]
    assert bool(k[1, 16]) == ((w[0] & 65535) >= 32768)  # column 16: element 0 of the third eight


def test_references_against_library_routines():
    g = torch.Generator().manual_seed(1)
    z = torch.randn(5, 24, generator=g, dtype=torch.float64, requires_grad=True)
    gamma, beta = torch.randn(24, generator=g, dtype=torch.float64), torch.randn(24, generator=g, dtype=torch.float64)
    hat, n, r = ref.layer_norm(z, gamma, beta)
    want = torch.nn.functional.layer_norm(z, (24,), gamma, beta, 1e-5)
    assert torch.allclose(hat, want, atol=1e-12)
    dh, dxo = torch.randn(5, 24, generator=g, dtype=torch.float64), torch.randn(5, 24, generator=g, dtype=torch.float64)
    (D,) = torch.autograd.grad((want * dh).sum() + (z * dxo).sum(), z)
    got, _, db = ref.layer_norm_grad(z.detach(), n.detach(), r.detach(), gamma, dxo, dh)
    assert torch.allclose(got, D, atol=1e-11) and torch.allclose(db, dh.sum(0))
    logits = torch.randn(6, 12, generator=g)
    q = ref.router_groups(logits, 3, 1, 1, sigmoid=False)
    assert torch.equal(q["idx"], logits.topk(3).indices)
    assert torch.allclose(q["w"], torch.softmax(logits.double().topk(3).values, -1))
    q = ref.router_groups(logits, 4, 4, 2, best=2, bias=torch.tensor([0.0] * 9 + [50.0] * 3))
    assert set(q["idx"][0, :3].tolist()) == {9, 10, 11} and q["loss"].shape == (1,)


def test_quantiser_reference():
    x = torch.tensor([[127.0, 0.5, -1.5, 2.5, -127, 3, 0, 1], [0] * 8, [1.0, math.inf, 0, 0, 0, 0, 0, 0]]).bfloat16()
    q, s = ref.i8_quantize(x)
    assert s[0] == 1.0 and q[0].tolist() == [127, 0, -2, 2, -127, 3, 0, 1] and s[1] == 0.0 and (q[1:] == 0).all() and torch.isnan(s[2])
