"""The router, norm and 4-bit weight calls run together, as a block of a model uses them: decoding with 4-bit
experts (one captured graph for every token count), the same experts through et_moe_layer after expansion, and
the training direction of the router and the norms."""
import math
import os
import subprocess
import sys

import pytest
import torch

from tests import ref_ops as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
U, B = ref.F32_HALF, ref.BF16_HALF
EPS = 1e-5


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rn(g, *s, std=1.0, mean=0.0, dtype=BF):
    return (mean + std * torch.randn(s, generator=g, device="cuda")).to(dtype)


class Block:
    """x += gate * RMSNorm(experts(RMSNorm(x))): norm, router, 4-bit experts, norm with gate and residual."""

    def __init__(self, E, T, H, F, En, k, group, seed):
        g = _gen(seed)
        self.E, self.dims = E, (T, H, F, En, k, group)
        self.g_in, self.g_post = _rn(g, H, std=0.1, mean=1.0), _rn(g, H, std=0.1, mean=1.0)
        self.gate = _rn(g, H, std=0.2, mean=0.5)
        self.wr = torch.randn(H, En, generator=g, device="cuda") / math.sqrt(H)
        self.w = [_rn(g, En, N, K, std=1 / math.sqrt(K)) for N, K in ((F, H), (F, H), (H, F))]
        self.q = []
        for w in self.w:
            q = torch.empty(*w.shape[:2], w.shape[2] // 2, dtype=torch.uint8, device="cuda")
            s = torch.empty(En, w.shape[2] // group, w.shape[1], dtype=BF, device="cuda")
            E.et_w4_quantize(w, q, s)
            self.q += [q, s]
        self.x = torch.zeros(T, H, dtype=BF, device="cuda")
        self.xhat, self.y, self.out = (torch.full((T, H), 7.0, dtype=BF, device="cuda") for _ in range(3))
        self.logits = torch.zeros(T, En, device="cuda")
        self.idx, self.gw = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
        self.counts, self.n = torch.zeros(En, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        self.losses = torch.zeros(2, device="cuda")
        self.dT = torch.full((1,), T, dtype=torch.int32, device="cuda")
        self.wsn = E.alloc_workspace(E.et_block_norm_workspace_bytes(T, H))
        self.wsr = E.alloc_workspace(E.et_router_topk_workspace_bytes(T, En, k))
        self.wse = E.alloc_workspace(E.et_w4_experts_workspace_bytes(T, H, F, En, k, group))

    def run(self):
        E = self.E
        E.et_block_norm(self.x, None, None, self.xhat, gamma_pre=self.g_in, eps=EPS, d_T=self.dT, workspace=self.wsn)
        torch.matmul(self.xhat.float(), self.wr, out=self.logits)
        E.et_router_topk(self.logits, self.idx, self.gw, expert_counts=self.counts, n_routed=self.n, losses=self.losses,
                         d_T=self.dT, workspace=self.wsr)
        E.et_w4_experts(self.xhat, self.idx, self.gw, *self.q, self.y, d_T=self.dT, workspace=self.wse)
        E.et_block_norm(self.x, self.y, self.out, None, gamma_post=self.g_post, gate=self.gate, eps=EPS, d_T=self.dT,
                        workspace=self.wsn)

    def check(self, T):
        """Every stage against its 64-bit definition on the inputs it was given."""
        xh = self.xhat[:T].cpu()
        z, hat = ref.block_norm(self.x[:T].double().cpu(), gamma_pre=self.g_in.double().cpu(), eps=EPS)
        ref.check(xh, hat, (B + 64 * U) * hat.abs(), "x_hat")
        r = ref.router(self.logits[:T].cpu(), self.dims[4])
        assert torch.equal(self.idx[:T].cpu(), r["idx"].to(torch.int32))
        assert torch.equal(self.counts.cpu(), r["counts"].to(torch.int32)) and int(self.n) == T
        q = [t.cpu() for t in self.q]
        want, mag = ref.experts(xh, self.idx[:T].cpu(), self.gw[:T].cpu(), q[0:2], q[2:4], q[4:6])
        ref.check(self.y[:T], want, B * (want.abs() + mag) + mag, "experts")
        z, _ = ref.block_norm(self.x[:T].double().cpu(), self.y[:T].double().cpu(), self.g_post.double().cpu(),
                              self.gate.double().cpu(), 1.0, None, EPS)
        ref.check(self.out[:T], z, B * z.abs() + 64 * U * (self.x[:T].double().cpu().abs() + z.abs() + 4), "out")
        for t in (self.xhat, self.y, self.out):
            assert (t[T:] == 7).all()
        for ws in (self.wsn, self.wsr, self.wse):
            assert self.E.et_status(ws) == (0, 0)


def test_decoding_block(cuda_lib):
    """Eager, then one captured graph replayed for other inputs and token counts."""
    b = Block(cuda_lib, 12, 256, 384, 16, 4, 64, 1)
    b.x.copy_(_rn(_gen(2), 12, 256))
    b.run()
    torch.cuda.synchronize()
    b.check(12)
    eager = b.out.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(b.out, eager)
    for seed, T in ((3, 1), (4, 7), (5, 12)):
        b.x.copy_(_rn(_gen(seed), 12, 256))
        b.dT.fill_(T)
        for t in (b.xhat, b.y, b.out):
            t.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        b.check(T)


def test_one_workspace_for_all(cuda_lib):
    """The router, norm and 4-bit calls may share one workspace, one call after the other."""
    E = cuda_lib
    b = Block(E, 12, 256, 384, 16, 4, 64, 1)
    b.x.copy_(_rn(_gen(2), 12, 256))
    T, H, En, k = 3000, 520, 64, 4
    g = _gen(6)
    x, y, dz, dh = (_rn(g, T, H) for _ in range(4))
    gam = _rn(g, H, mean=1.0, std=0.1)
    L = torch.randn(T, En, generator=g, device="cuda")
    sizes = (E.et_block_norm_workspace_bytes(T, H), E.et_router_topk_workspace_bytes(T, En, k), b.wse.numel())

    def step(wsn, wsr):
        dx, dy = torch.empty_like(x), torch.empty_like(x)
        dg = torch.empty(H, device="cuda")
        idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
        losses = torch.empty(2, device="cuda")
        b.run()
        E.et_router_topk(L, idx, w, losses=losses, workspace=wsr)
        b.run()
        E.et_block_norm_bwd(x, y, dz, dh, dx, dy, gamma_post=gam, gamma_pre=gam, eps=EPS, d_gamma_pre=dg, workspace=wsn)
        E.et_router_topk(L, idx, w, losses=losses, workspace=wsr)
        return b.out.clone(), b.y.clone(), b.losses.clone(), dx, dy, dg, idx, w, losses

    want = step(E.alloc_workspace(sizes[0]), E.alloc_workspace(sizes[1]))
    one = E.alloc_workspace(max(sizes))
    b.wsn = b.wsr = b.wse = one
    for _ in range(3):
        assert all(torch.equal(a, c) for a, c in zip(step(one, one), want))
    assert E.et_status(one) == (0, 0)


def test_two_blocks_on_two_streams(cuda_lib):
    """Two blocks at once, each with its own workspaces, give what they give alone."""
    bs = [Block(cuda_lib, 5, 128, 256, 8, 2, 32, s) for s in (11, 12)]
    want = []
    for i, b in enumerate(bs):
        b.x.copy_(_rn(_gen(20 + i), 5, 128))
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


def test_back_to_back_calls_see_each_other(cuda_lib):
    """Each call reads what the one before it in the stream wrote, with nothing waited for in between."""
    E = cuda_lib
    T, H = 3, 256
    g = _gen(31)
    w = [_rn(g, 512, H, std=1 / 16.0), _rn(g, H, 512, std=1 / 22.0)]
    ws = E.alloc_workspace(256)
    wsn = E.alloc_workspace(E.et_block_norm_workspace_bytes(T, H))
    gm = torch.ones(H, dtype=BF, device="cuda")
    x0 = _rn(g, T, H)
    first = None
    for step in range(30):
        x = x0.clone()
        for layer in range(4):  # quantise, multiply, multiply, normalise and add
            packed = []
            for m in w:
                q = torch.empty(m.shape[0], m.shape[1] // 2, dtype=torch.uint8, device="cuda")
                s = torch.empty(m.shape[1] // 64, m.shape[0], dtype=BF, device="cuda")
                E.et_w4_quantize(m, q, s)
                packed.append((q, s))
            h = torch.empty(T, 512, dtype=BF, device="cuda")
            y = torch.empty(T, H, dtype=BF, device="cuda")
            E.et_w4_gemv(x, *packed[0], h, workspace=ws)
            E.et_w4_gemv(h, *packed[1], y, workspace=ws)
            x_in = x.clone() if step == 0 else None
            E.et_block_norm(x, y, x, None, gamma_post=gm, scale=0.5, eps=EPS, workspace=wsn)
            if step == 0:
                # each call on the bits it was given
                torch.cuda.synchronize()
                pk = [ref.w4_pack(m.cpu(), 64) for m in w]
                for got, inp, (q, s) in ((h, x_in, pk[0]), (y, h, pk[1])):
                    want, mag = ref.gemv(inp.cpu(), q, s)
                    ref.check(got, want, B * want.abs() + (2 * inp.shape[1] + 16) * U * mag, "gemv")
                z, _ = ref.block_norm(x_in.double().cpu(), y.double().cpu(), gm.double().cpu(), None, 0.5, None, EPS)
                ref.check(x, z, B * z.abs() + 64 * U * (x_in.double().cpu().abs() + z.abs()), "x")
        if step == 0:
            first = x
        else:  # nothing waited for: the same bits
            assert torch.equal(x, first)


def test_expanded_experts_through_the_moe_layer(cuda_lib):
    """et_w4_dequantize feeds et_moe_layer, whose routing feeds et_w4_experts: the same layer twice."""
    E = cuda_lib
    T, H, F, En, k, group = 16, 256, 512, 8, 2, 128
    b = Block(E, T, H, F, En, k, group, 41)
    x = _rn(_gen(42), T, H)
    ws = [torch.empty_like(w) for w in b.w]
    for w, q, s in zip(ws, b.q[0::2], b.q[1::2]):
        E.et_w4_dequantize(q, s, w)
    out = torch.empty(T, H, dtype=BF, device="cuda")
    wsm = E.alloc_workspace(E.et_moe_workspace_bytes(T, H, F, En, k))
    E.et_moe_layer(x, b.wr.to(BF), None, *ws, out, k=k, topk_idx=b.idx, topk_w=b.gw, workspace=wsm)
    E.et_w4_experts(x, b.idx, b.gw, *b.q, b.y, workspace=b.wse)
    q = [t.cpu() for t in b.q]
    want, mag = ref.experts(x.cpu(), b.idx.cpu(), b.gw.cpu(), q[0:2], q[2:4], q[4:6])
    ref.check(b.y, want, B * (want.abs() + mag) + mag, "experts")
    # the layer's weights are rounded to bf16 once more (half a step each on gate, up and down), its y too: the
    # magnitudes that mag holds for the sums, times 2^-8, and |y| 2^-8
    w64 = [ref.w4_values(q[i], q[i + 1]) for i in (0, 2, 4)]
    extra = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        xt = x[t].double().cpu()
        for j in range(k):
            e, wt = int(b.idx[t, j]), float(b.gw[t, j])
            g, u = w64[0][e] @ xt, w64[1][e] @ xt
            dg, du = (B * (m[e].abs() @ xt.abs()) for m in w64[:2])
            h = (g * torch.sigmoid(g) * u).abs()
            dh = 1.1 * dg * u.abs() + (g * torch.sigmoid(g)).abs() * du + 1.1 * dg * du
            extra[t] += wt * (w64[2][e].abs() @ (dh + B * (h + dh)) + B * (w64[2][e] @ (g * torch.sigmoid(g) * u)).abs())
    ref.check(out, want, B * (want.abs() + mag + extra) + mag + 1.01 * extra, "et_moe_layer on expanded weights")


def test_training_step_of_router_and_norms(cuda_lib):
    """Two norms around a router: forward, then backward through the losses, the gate weights and both norms."""
    E = cuda_lib
    T, H, En, k = 96, 512, 24, 3
    g = _gen(51)
    x, y = _rn(g, T, H), _rn(g, T, H, std=2.0)
    gp, gr, gate = _rn(g, H, std=0.1, mean=1.0), _rn(g, H, std=0.1, mean=1.0), torch.rand(T, generator=g, device="cuda")
    wr = torch.randn(H, En, generator=g, device="cuda") / math.sqrt(H)
    dw, dl = torch.randn(T, k, generator=g, device="cuda"), torch.tensor([0.3, 0.1], device="cuda")
    wsn, wsr = E.alloc_workspace(E.et_block_norm_workspace_bytes(T, H)), E.alloc_workspace(E.et_router_topk_workspace_bytes(T, En, k))
    xo, xh, dx, dy = (torch.empty_like(x) for _ in range(4))
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    counts, n, ls = torch.empty(En, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty(2, device="cuda")
    dlog = torch.empty(T, En, device="cuda")
    dgp, dgr, dgate = torch.empty(H, device="cuda"), torch.empty(H, device="cuda"), torch.empty(T, device="cuda")
    kw = dict(gamma_post=gp, gate=gate, scale=0.5, gamma_pre=gr, eps=EPS, workspace=wsn)

    def step():
        E.et_block_norm(x, y, xo, xh, **kw)
        logits = xh.float() @ wr
        E.et_router_topk(logits, idx, w, expert_counts=counts, n_routed=n, losses=ls, workspace=wsr)
        E.et_router_topk_bwd(logits, idx, w, counts, n, dlog, d_losses=dl, d_topk_w=dw, workspace=wsr)
        dh = (dlog @ wr.t()).to(BF)
        E.et_block_norm_bwd(x, y, torch.zeros_like(x), dh, dx, dy, d_gamma_post=dgp, d_gamma_pre=dgr, d_gate=dgate, **kw)
    step()
    # the whole step in 64 bits, by automatic differentiation, with the kernel's selection
    a = [t.double().cpu().requires_grad_(True) for t in (x, y, gp, gr)] + [gate.double().cpu()[:, None].requires_grad_(True)]
    z, hat = ref.block_norm(a[0], a[1], a[2], a[4], 0.5, a[3], EPS)
    # the logits are taken from the rounded x_hat: the rounding is a constant to the gradient
    logits = (hat + (xh.double().cpu() - hat).detach()) @ wr.double().cpu()
    r = ref.router(logits, k)
    assert torch.equal(idx.cpu(), r["idx"].to(torch.int32))
    total = (r["losses"] * dl.double().cpu()).sum() + (r["w"] * dw.double().cpu()).sum()
    grads = torch.autograd.grad(total, a)
    for got, want, what in ((dx, grads[0], "dx"), (dy, grads[1], "dy"), (dgp, grads[2], "d_gamma_post"),
                            (dgr, grads[3], "d_gamma_pre"), (dgate, grads[4][:, 0], "d_gate")):
        # d_x_hat enters rounded to bf16: relative to the largest gradient of the tensor (sums over H or T of
        # independent roundings stay below 16 half steps of it)
        ref.check(got, want, B * want.abs() + 16 * B * float(want.abs().max()), what)
        assert float((got.double().cpu() - want).norm() / want.norm()) < 2 * B
    first = [t.clone() for t in (dx, dy, dgp, dgr, dgate, dlog)]
    step()
    assert all(torch.equal(p, q) for p, q in zip(first, (dx, dy, dgp, dgr, dgate, dlog)))


CAPTURE_FIRST = """
import sys
sys.path.insert(0, sys.argv[1])
import torch
from moe_task_scheduling_gb300 import etmoe as E
bf, dev = torch.bfloat16, "cuda"
torch.cuda.init()
T, H, F, En, k = 4, 1024, 256, 8, 2
x, y = torch.randn(T, H, device=dev).to(bf), torch.randn(T, H, device=dev).to(bf)
g = torch.ones(H, device=dev, dtype=bf)
xo, xh, dx, dy, out = (torch.zeros_like(x) for _ in range(5))
dg = torch.zeros(H, device=dev)
L, idx, w = torch.randn(T, En, device=dev), torch.zeros(T, k, device=dev, dtype=torch.int32), torch.zeros(T, k, device=dev)
cnt, n, ls, dL = torch.zeros(En, device=dev, dtype=torch.int32), torch.zeros(1, device=dev, dtype=torch.int32), torch.zeros(2, device=dev), torch.zeros_like(L)
ws = [torch.randn(En, N, K, device=dev).to(bf) for N, K in ((F, H), (F, H), (H, F))]
q = []
for a in ws:
    q += [torch.zeros(En, a.shape[1], a.shape[2] // 2, device=dev, dtype=torch.uint8), torch.zeros(En, a.shape[2] // 64, a.shape[1], device=dev, dtype=bf)]
yg = torch.zeros(T, F, device=dev, dtype=bf)
back = torch.zeros_like(ws[0])
wsp = E.alloc_workspace(1 << 24)
def step():
    E.et_block_norm(x, y, xo, xh, gamma_post=g, gamma_pre=g, eps=1e-5, workspace=wsp)
    E.et_block_norm_bwd(x, y, xo, xh, dx, dy, gamma_post=g, gamma_pre=g, d_gamma_post=dg, eps=1e-5, workspace=wsp)
    E.et_router_topk(L, idx, w, expert_counts=cnt, n_routed=n, losses=ls, workspace=wsp)
    E.et_router_topk_bwd(L, idx, w, cnt, n, dL, d_losses=ls, workspace=wsp)
    for i in range(3):
        E.et_w4_quantize(ws[i], q[2 * i], q[2 * i + 1])
    E.et_w4_dequantize(q[0], q[1], back)
    E.et_w4_gemv(xh, q[0][0], q[1][0], yg, workspace=wsp)
    E.et_w4_experts(xh, idx, w, *q, out, workspace=wsp)
gr = torch.cuda.CUDAGraph()
with torch.cuda.graph(gr):
    step()
gr.replay()
torch.cuda.synchronize()
outs = (xo, xh, dx, dy, dg, idx, w, cnt, n, ls, dL, back, yg, out)
got = [t.clone() for t in outs]
for t in outs:
    t.zero_()
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, outs)) and float(out.float().abs().sum()) > 0
print("captured first")
"""


def test_first_calls_inside_a_capture(cuda_lib):
    """A process whose first call of everything is captured into a graph."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CAPTURE_FIRST, root], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout + r.stderr[-2000:]
