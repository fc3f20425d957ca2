"""The grouped router, the layer norm with dropout and the int8 products run together, as a block of a model uses
them: decoding with 4-bit experts and an int8 projection (one captured graph for every token count), the training
direction with dropout drawn anew at each replay, and many calls after one another without a wait."""
import math
import os
import subprocess
import sys

import pytest
import torch

from tests import ref_more as ref
from tests import ref_ops
from tests.ref_ops import BF16_HALF as B
from tests.ref_ops import F32_HALF as U
from tests.ref_ops import check

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
EPS = 1e-5
GROUPS = dict(n_groups=4, k_groups=2, renorm=True, scale=2.5)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rn(g, *s, std=1.0, mean=0.0, dtype=BF):
    return (mean + std * torch.randn(s, generator=g, device="cuda")).to(dtype)


class Block:
    """x + experts(LayerNorm(x)), normalised once more and projected with int8 weights."""

    def __init__(self, E, T, H, F, En, k, N, seed, ws=None):
        g = _gen(seed)
        self.E, self.k, self.T, self.En = E, k, T, En
        self.norms = [(_rn(g, H, std=0.1, mean=1.0), _rn(g, H, std=0.1)) for _ in range(2)]
        self.wr, self.bias = torch.randn(H, En, generator=g, device="cuda") / math.sqrt(H), 0.1 * torch.randn(En, generator=g, device="cuda")
        self.q = []
        for n, kk in ((F, H), (F, H), (H, F)):
            w = _rn(g, En, n, kk, std=1 / math.sqrt(kk))
            q = torch.empty(En, n, kk // 2, dtype=torch.uint8, device="cuda")
            s = torch.empty(En, kk // 64, n, dtype=BF, device="cuda")
            E.et_w4_quantize(w, q, s)
            self.q += [q, s]
        self.wq, self.sw = torch.empty(N, H, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
        E.et_i8_quantize(_rn(g, N, H, std=1 / math.sqrt(H)), self.wq, self.sw, workspace=E.alloc_workspace(E.et_i8_quantize_workspace_bytes(N, H)))
        self.x = torch.zeros(T, H, dtype=BF, device="cuda")
        self.h, self.y, self.z, self.n = (torch.full((T, H), 7.0, dtype=BF, device="cuda") for _ in range(4))
        self.xq, self.sx = torch.zeros(T, H, dtype=torch.int8, device="cuda"), torch.zeros(T, device="cuda")
        self.out = torch.full((T, N), 7.0, dtype=BF, device="cuda")
        self.logits = torch.zeros(T, En, device="cuda")
        self.idx, self.w = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
        self.counts = torch.zeros(En, dtype=torch.int32, device="cuda")
        self.dT = torch.full((1,), T, dtype=torch.int32, device="cuda")
        need = max(E.et_layer_norm_workspace_bytes(T, H), E.et_router_groups_workspace_bytes(T, En, k), E.et_i8_gemm_workspace_bytes(T, N, H),
                   E.et_w4_experts_workspace_bytes(T, H, F, En, k, 64), E.et_i8_quantize_workspace_bytes(T, H))
        self.ws = E.alloc_workspace(need) if ws is None else ws

    def run(self):
        E, kw = self.E, dict(d_T=self.dT, workspace=self.ws)
        (g0, b0), (g1, b1) = self.norms
        E.et_layer_norm(self.x, None, None, self.h, gamma=g0, beta=b0, eps=EPS, **kw)
        torch.matmul(self.h.float(), self.wr, out=self.logits)
        E.et_router_groups(self.logits, self.idx, self.w, score=E.ET_SCORE_SIGMOID, bias=self.bias, expert_counts=self.counts, **GROUPS, **kw)
        E.et_w4_experts(self.h, self.idx, self.w, *self.q, self.y, **kw)
        E.et_layer_norm(self.x, self.y, self.z, self.n, gamma=g1, beta=b1, eps=EPS, **kw)
        E.et_i8_quantize(self.n, self.xq, self.sx, d_M=self.dT, workspace=self.ws)
        E.et_i8_gemm(self.xq, self.sx, self.wq, self.sw, self.out, d_M=self.dT, workspace=self.ws)

    def check(self, T):
        """Every stage against its 64-bit definition on the inputs it was given."""
        c = lambda t: t[:T].cpu()  # noqa: E731
        for (gam, bet), x, y, z, got in ((self.norms[0], c(self.x), None, None, c(self.h)), (self.norms[1], c(self.x), c(self.y), c(self.z), c(self.n))):
            s = ref.residual(x, y)
            if z is not None:
                check(z, s, ref.bf16_bound(s, 2 * U * s.abs()), "z")
            hat, n, r = ref.layer_norm(s, gam.cpu(), bet.cpu(), EPS)
            e, _ = ref.norm_error(x, y, 1.0, s, n, r)
            check(got, hat, ref.bf16_bound(hat, e * gam.cpu().double().abs() + 4 * U * (hat.abs() + bet.cpu().double().abs())), "x_hat")
        how = dict(best=2, sigmoid=True, bias=self.bias.cpu(), renorm=True, scale=2.5)
        r = ref.router_groups(c(self.logits), self.k, 4, 2, **how)
        assert torch.equal(c(self.idx).long(), r["idx"]) and torch.equal(self.counts.cpu().double(), r["counts"])
        L = c(self.logits).double()
        check(self.w[:T], r["w"], (20 + self.En + 2 * float(L.abs().max())) * 2 * U * r["w"], "w")
        q = [t.cpu() for t in self.q]
        want, mag = ref_ops.experts(c(self.h), c(self.idx), c(self.w), q[0:2], q[2:4], q[4:6])
        check(self.y[:T], want, B * (want.abs() + mag) + mag, "experts")
        xq, sx = ref.i8_quantize(c(self.n))
        assert torch.equal(c(self.xq), xq) and torch.equal(c(self.sx), sx)
        Y, e = ref.i8_gemm(xq, sx, self.wq.cpu(), self.sw.cpu())
        check(self.out[:T], Y, ref.bf16_bound(Y, e), "out")
        for t in (self.h, self.y, self.z, self.n, self.out):
            assert (t[T:] == 7).all()
        assert self.E.et_status(self.ws) == (0, 0)


@pytest.mark.parametrize("T,N", [(12, 400), (40, 1000)])
def test_decoding_block(cuda_lib, T, N):
    """Eager, on another stream, then one captured graph replayed for other inputs and token counts."""
    b = Block(cuda_lib, T, 256, 384, 16, 4, N, 1)
    b.x.copy_(_rn(_gen(2), T, 256))
    b.run()
    torch.cuda.synchronize()
    b.check(T)
    eager = b.out.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.run()
    torch.cuda.synchronize()
    assert torch.equal(b.out, eager)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(b.out, eager)
    for seed, n in ((3, 1), (4, 7), (5, T)):
        b.x.copy_(_rn(_gen(seed), T, 256))
        b.dT.fill_(n)
        for t in (b.h, b.y, b.z, b.n, b.out):
            t.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        b.check(n)


def test_two_graphs_share_a_workspace(cuda_lib):
    """Two captured blocks of other shapes, one workspace, replayed in turn on one stream: each gives what it gives alone."""
    shapes = ((12, 256, 384, 16, 4, 400), (40, 512, 256, 32, 2, 1000))
    alone = [Block(cuda_lib, *s, seed=10 + i) for i, s in enumerate(shapes)]
    one = cuda_lib.alloc_workspace(max(b.ws.numel() for b in alone))
    bs = [Block(cuda_lib, *s, seed=10 + i, ws=one) for i, s in enumerate(shapes)]
    graphs = []
    for i, (a, b) in enumerate(zip(alone, bs)):
        a.x.copy_(_rn(_gen(i), *a.x.shape))
        b.x.copy_(a.x)
        a.run()
        b.run()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            b.run()
    for _ in range(10):
        for b in bs:
            b.out.zero_()
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.out, b.out) and torch.equal(a.w, b.w) for a, b in zip(alone, bs))
    assert cuda_lib.et_status(one) == (0, 0)


def test_two_blocks_on_two_streams(cuda_lib):
    """Two blocks at once, each with its own workspace, give what they give alone."""
    bs = [Block(cuda_lib, 40, 256, 384, 16, 4, 1000, s) for s in (11, 12)]
    want = []
    for i, b in enumerate(bs):
        b.x.copy_(_rn(_gen(20 + i), 40, 256))
        b.run()
        torch.cuda.synchronize()
        want.append(b.out.clone())
    streams = [torch.cuda.Stream() for _ in bs]
    for _ in range(20):
        for b, s in zip(bs, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                b.run()
        torch.cuda.synchronize()
        assert all(torch.equal(b.out, w) for b, w in zip(bs, want))


class Step:
    """z = x + dropout(y), LayerNorm, grouped router with its loss; and the way back to x, y, gamma and beta."""

    def __init__(self, E, sigmoid, T=96, H=512, En=24, k=3):
        g = _gen(51)
        self.E, self.k = E, k
        self.x, self.y, self.dz = _rn(g, T, H), _rn(g, T, H, std=2.0), _rn(g, T, H, std=0.01)
        self.gam, self.bet = _rn(g, H, std=0.1, mean=1.0), _rn(g, H, std=0.1)
        self.wr = torch.randn(H, En, generator=g, device="cuda") / math.sqrt(H)
        self.dw, self.dl = torch.randn(T, k, generator=g, device="cuda"), torch.tensor([0.3], device="cuda")
        self.rng = torch.tensor([0x123456789ABCDEF, 7], dtype=torch.int64, device="cuda")
        self.z, self.h, self.dx, self.dy = (torch.empty_like(self.x) for _ in range(4))
        self.idx, self.w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
        self.counts, self.n = torch.empty(En, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
        self.loss, self.dlog = torch.empty(1, device="cuda"), torch.empty(T, En, device="cuda")
        self.dgam, self.dbet = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
        self.logits = torch.empty(T, En, device="cuda")
        self.sigmoid = sigmoid
        self.ws = E.alloc_workspace(max(E.et_layer_norm_workspace_bytes(T, H), E.et_router_groups_workspace_bytes(T, En, k)))

    def run(self):
        E = self.E
        norm = dict(gamma=self.gam, eps=EPS, p=0.2, d_rng=self.rng, workspace=self.ws)
        how = dict(score=E.ET_SCORE_SIGMOID if self.sigmoid else E.ET_SCORE_SOFTMAX, renorm=True, scale=2.5, workspace=self.ws)
        E.et_layer_norm(self.x, self.y, self.z, self.h, beta=self.bet, **norm)
        torch.matmul(self.h.float(), self.wr, out=self.logits)
        E.et_router_groups(self.logits, self.idx, self.w, n_groups=4, k_groups=2, expert_counts=self.counts, n_routed=self.n, loss=self.loss, **how)
        E.et_router_groups_bwd(self.logits, self.idx, self.w, self.counts, self.n, self.dlog, d_loss=self.dl, d_topk_w=self.dw, **how)
        dh = torch.matmul(self.dlog, self.wr.t()).to(BF)
        E.et_layer_norm_bwd(self.x, self.y, self.dz, dh, self.dx, self.dy, d_gamma=self.dgam, d_beta=self.dbet, **norm)

    def outputs(self):
        return [self.z, self.h, self.idx, self.w, self.loss, self.dlog, self.dx, self.dy, self.dgam, self.dbet]


@pytest.mark.parametrize("sigmoid", [True, False])
def test_training_step(cuda_lib, sigmoid):
    s = Step(cuda_lib, sigmoid)
    s.run()
    torch.cuda.synchronize()
    # the whole step in 64 bits, by automatic differentiation, with the kernel's choice
    a = [t.double().cpu().requires_grad_(True) for t in (s.x, s.y, s.gam, s.bet)]
    kept, mul = ref.keep(*s.y.shape, 0.2, 0x123456789ABCDEF, 7)
    z = a[0] + torch.where(kept, a[1] * mul, torch.zeros_like(a[1]))
    hat = (z - z.mean(-1, keepdim=True)) / torch.sqrt(z.var(-1, unbiased=False, keepdim=True) + EPS) * a[2] + a[3]
    # the logits are taken from the rounded x_hat: the rounding is a constant to the gradient
    logits = (hat + (s.h.double().cpu() - hat).detach()) @ s.wr.double().cpu()
    r = ref.router_groups(s.logits.cpu(), s.k, 4, 2, sigmoid=sigmoid, scale=2.5)
    assert torch.equal(s.idx.cpu().long(), r["idx"])
    r = ref.router_groups(logits, s.k, 4, 2, sigmoid=sigmoid, scale=2.5, idx=r["idx"])
    total = (r["loss"] * s.dl.double().cpu()).sum() + (r["w"] * s.dw.double().cpu()).sum() + (z * s.dz.double().cpu()).sum()
    grads = torch.autograd.grad(total, a)
    for got, want, what in zip((s.dx, s.dy, s.dgam, s.dbet), grads, ("dx", "dy", "d_gamma", "d_beta")):
        # d_x_hat enters rounded to bf16: relative to the largest gradient of the tensor (sums over H or T of
        # independent roundings stay below 16 half steps of it)
        check(got, want, B * want.abs() + 16 * B * float(want.abs().max()), what)
        assert float((got.double().cpu() - want).norm() / want.norm()) < 2 * B
    assert (s.dy.cpu()[~kept] == 0).all()


def test_training_step_captured(cuda_lib):
    """One graph: every replay draws anew from the device's seed and offset, and gives the bits of an eager step."""
    s = Step(cuda_lib, True)
    s.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
        s.rng[1:].add_(1)
    seen = []
    s.rng[1:].fill_(100)
    for _ in range(4):
        g.replay()
        seen.append([t.clone() for t in s.outputs()])
    for i, want in enumerate(seen):
        s.rng[1:].fill_(100 + i)
        s.run()
        assert all(torch.equal(p, q) for p, q in zip(want, s.outputs()))
    assert not torch.equal(seen[0][0], seen[1][0])
    assert cuda_lib.et_status(s.ws) == (0, 0)


def test_back_to_back_calls_see_each_other(cuda_lib):
    """Each call reads what the one before it in the stream wrote, with nothing waited for in between."""
    E = cuda_lib
    g = _gen(31)
    for T, H, N in ((3, 256, 512), (200, 264 * 2, 384), (600, 512, 1024)):
        w = [_rn(g, N, H, std=1 / math.sqrt(H)), _rn(g, H, N, std=1 / math.sqrt(N))]
        packed = []
        ws = E.alloc_workspace(max(E.et_i8_gemm_workspace_bytes(T, N, H), E.et_i8_gemm_workspace_bytes(T, H, N),
                                   E.et_layer_norm_workspace_bytes(T, max(H, N))))
        x0 = _rn(g, T, H)
        first = None
        for step in range(20):
            x = x0.clone()
            seen = []
            for layer in range(3):
                packed = []
                for m in w:
                    packed.append((torch.empty(m.shape, dtype=torch.int8, device="cuda"), torch.empty(m.shape[0], device="cuda")))
                    E.et_i8_quantize(m, *packed[-1], workspace=ws)
                h, y = torch.empty(T, N, dtype=BF, device="cuda"), torch.empty(T, H, dtype=BF, device="cuda")
                n = torch.empty_like(x)
                E.et_layer_norm(x, None, None, n, eps=EPS, workspace=ws)
                for inp, out, (wq, sw) in ((n, h, packed[0]), (h, y, packed[1])):
                    xq, sx = torch.empty(inp.shape, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
                    E.et_i8_quantize(inp, xq, sx, workspace=ws)
                    E.et_i8_gemm(xq, sx, wq, sw, out, workspace=ws)
                    seen.append((inp, out, wq, sw))
                E.et_dropout(x, y, x, p=0.1, seed=5, offset=layer, workspace=ws)
            if step == 0:
                torch.cuda.synchronize()
                for inp, out, wq, sw in seen:
                    xq, sx = ref.i8_quantize(inp.cpu())
                    Y, e = ref.i8_gemm(xq, sx, wq.cpu(), sw.cpu())
                    check(out, Y, ref.bf16_bound(Y, e), "product")
                first = x
            else:  # nothing waited for: the same bits
                assert torch.equal(x, first)
        assert E.et_status(ws) == (0, 0)


@pytest.mark.parametrize("M,N,K", [(4096, 3000, 528), (3000, 14336, 272), (512, 14336, 1040), (300, 20000, 784), (20, 40000, 144), (8192 + 300, 512, 528)])
def test_many_tiles_stay_the_same(cuda_lib, M, N, K):
    """Products of several tiles a CTA, run again and again: exact sums, so every run gives the same bits."""
    g = _gen(M + N)
    xq = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    wq = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sx, sw = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
    ws = cuda_lib.alloc_workspace(cuda_lib.et_i8_gemm_workspace_bytes(M, N, K))
    # an exact product: |sums| < 2^24, 127 * 127 * K < 2^24 for K up to 1040, in fp32 without a rounding
    want = ((xq.float() @ wq.float().t()) * (sx[:, None] * sw)).to(BF)
    for _ in range(12):
        Y = torch.empty(M, N, dtype=BF, device="cuda")
        cuda_lib.et_i8_gemm(xq, sx, wq, sw, Y, workspace=ws)
        assert torch.equal(Y, want)


CAPTURE_FIRST = """
import sys
sys.path.insert(0, sys.argv[1])
import torch
from moe_task_scheduling_gb300 import etmoe as E
bf, dev = torch.bfloat16, "cuda"
torch.cuda.init()
outs, calls = [], []
wsp = E.alloc_workspace(1 << 26)
def new(*s, dtype=bf):
    t = torch.zeros(*s, dtype=dtype, device=dev)
    outs.append(t)
    return t
for T, H, En, k, G in ((4, 1024, 64, 4, 8), (1000, 250, 24, 3, 4), (300, 4096, 256, 8, 8)):
    x, y, g = torch.randn(T, H, device=dev).to(bf), torch.randn(T, H, device=dev).to(bf), torch.ones(H, device=dev, dtype=bf)
    L = torch.randn(T, En, device=dev)
    a = [new(T, H) for _ in range(5)]
    dg, db, ls, mp = new(H, dtype=torch.float32), new(H, dtype=torch.float32), new(1, dtype=torch.float32), new(En, dtype=torch.float32)
    idx, w, cnt, n, dL = new(T, k, dtype=torch.int32), new(T, k, dtype=torch.float32), new(En, dtype=torch.int32), new(1, dtype=torch.int32), new(T, En, dtype=torch.float32)
    def call(x=x, y=y, g=g, L=L, a=a, dg=dg, db=db, ls=ls, mp=mp, idx=idx, w=w, cnt=cnt, n=n, dL=dL, G=G):
        kw = dict(gamma=g, eps=1e-5, p=0.1, seed=3, workspace=wsp)
        E.et_dropout(x, y, a[0], p=0.1, workspace=wsp)
        E.et_layer_norm(x, y, a[1], a[2], beta=g, **kw)
        E.et_layer_norm_bwd(x, y, a[1], a[2], a[3], a[4], d_gamma=dg, d_beta=db, **kw)
        for sc in (E.ET_SCORE_SIGMOID, E.ET_SCORE_SOFTMAX):
            E.et_router_groups(L, idx, w, score=sc, n_groups=G, k_groups=2, expert_counts=cnt, n_routed=n, loss=ls, mean_prob=mp, workspace=wsp)
            E.et_router_groups_bwd(L, idx, w, cnt, n, dL, score=sc, d_loss=ls, d_topk_w=w, workspace=wsp)
    calls.append(call)
for M, N, K in ((1, 500, 1024), (12, 500, 1024), (64, 300, 528), (500, 2000, 1024), (2000, 4096, 512)):
    x, m = torch.randn(M, K, device=dev).to(bf), torch.randn(N, K, device=dev).to(bf)
    xq, sx, wq, sw, Y = new(M, K, dtype=torch.int8), new(M, dtype=torch.float32), new(N, K, dtype=torch.int8), new(N, dtype=torch.float32), new(M, N)
    def call(x=x, m=m, xq=xq, sx=sx, wq=wq, sw=sw, Y=Y):
        E.et_i8_quantize(x, xq, sx, workspace=wsp)
        E.et_i8_quantize(m, wq, sw, workspace=wsp)
        E.et_i8_gemm(xq, sx, wq, sw, Y, workspace=wsp)
    calls.append(call)
gr = torch.cuda.CUDAGraph()
with torch.cuda.graph(gr):
    for c in calls:
        c()
gr.replay()
torch.cuda.synchronize()
got = [t.clone() for t in outs]
for t in outs:
    t.zero_()
for c in calls:
    c()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, outs)) and all(float(t.float().abs().sum()) > 0 for t in outs)
assert E.et_status(wsp) == (0, 0)
print("captured first")
"""


def test_first_calls_inside_a_capture(cuda_lib):
    """A process whose first call of everything is captured into a graph."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CAPTURE_FIRST, root], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout + r.stderr[-2000:]
