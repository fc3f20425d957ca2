"""Plain 64-bit definitions of the grouped router, the layer norm with dropout and the int8 products, and the error
bounds that go with them.  Test infrastructure: shares no code with the CUDA path."""
import math

import numpy as np
import torch

from tests.ref_ops import BF16_HALF, F32_HALF

F64 = torch.float64
U = F32_HALF


# ------------------------------------------------------------------ grouped router

def router_groups(logits, k, G, kg, best=2, sigmoid=True, bias=None, renorm=True, scale=1.0, mask=None, idx=None):
    """The choice and the outputs in 64 bits; logits may require grad (fp64 then).  idx: a given choice."""
    L = logits.double()
    T, E = L.shape
    if sigmoid:
        s = torch.sigmoid(L)
    else:
        top = torch.where(L.detach().amax(-1, keepdim=True) > -math.inf, L.detach().amax(-1, keepdim=True), torch.zeros(T, 1, dtype=F64))
        ex = torch.exp(L - top)
        z = ex.sum(-1, keepdim=True)
        s = ex / torch.where(z > 0, z, torch.ones_like(z))
    if idx is None:
        c = (s if bias is None else s + bias.double()).detach()
        c = torch.where(L.detach() == -math.inf, torch.full_like(c, -math.inf), c)
        idx = torch.full((T, k), -1, dtype=torch.int64)
        for t in range(T):
            if mask is not None and not mask[t]:
                continue
            row = c[t].tolist()
            rank = lambda v: math.inf if math.isnan(v) else v  # noqa: E731
            scores = []
            for g in range(G):
                there = sorted((rank(v) for v in row[g * (E // G):(g + 1) * (E // G)] if v != -math.inf), reverse=True)[:best]
                scores.append(sum(there) if there else -math.inf)
            into = sorted(range(G), key=lambda g: (-scores[g], g))[:kg]
            cand = [e for e in range(E) if e // (E // G) in into and row[e] != -math.inf]
            for j, e in enumerate(sorted(cand, key=lambda e: (-rank(row[e]), e))[:k]):
                idx[t, j] = e
    on = idx >= 0
    live = on.any(-1)

    def shares(ls, there):  # s / sum s of scores given by their logarithms, however small; 0 where not there
        top = torch.where(there, ls.detach(), torch.full_like(ls, -math.inf)).amax(-1, keepdim=True)
        ex = torch.where(there, torch.exp(torch.where(there, ls - top, torch.zeros_like(ls))), torch.zeros_like(ls))
        z = ex.sum(-1, keepdim=True)
        return ex / torch.where(z > 0, z, torch.ones_like(z))
    ls = torch.nn.functional.logsigmoid(L) if sigmoid else L
    sel = torch.gather(s, 1, idx.clamp(min=0))
    w = shares(torch.gather(ls, 1, idx.clamp(min=0)), on) if renorm else torch.where(on, sel, torch.zeros_like(sel))
    w = scale * w
    counts = torch.zeros(E, dtype=F64).index_add_(0, idx[on], torch.ones(int(on.sum()), dtype=F64))
    n = int(live.sum())
    rows = max(n, 1)
    p = shares(ls, live[:, None] & (L.detach() > -math.inf))
    mean_prob = p.sum(0) / rows
    loss = (E * (counts / (rows * k) * mean_prob).sum()).reshape(1)
    return dict(idx=idx, w=w, counts=counts, n=n, mean_prob=mean_prob, loss=loss, p=p, s=s, live=live)


def router_groups_grad(logits, r, k, d_loss, d_w, **how):
    """d_logits by automatic differentiation with the choice r["idx"] held."""
    L = logits.double().clone().requires_grad_(True)
    q = router_groups(L, k, 1, 1, idx=r["idx"], **how)
    total = (q["loss"] * d_loss.double()).sum() + torch.where(r["idx"] >= 0, q["w"] * d_w.double(), torch.zeros_like(q["w"])).sum()
    (g,) = torch.autograd.grad(total, L)
    return torch.where(r["live"][:, None], g, torch.zeros_like(g))


# ------------------------------------------------------------------ dropout

def philox(counter, key):
    """Philox4x32-10 of four counter words and two key words (numpy arrays or numbers)."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(v) for v in key]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def keep(T, H, p, seed, offset):
    """(bool [T, H] of the kept elements, the factor of a kept one)."""
    thr = int(np.rint(np.float64(np.float32(p)) * 65536))
    out = np.zeros((T, H), dtype=bool)
    h = np.arange(H)
    t = np.repeat(np.arange(T)[:, None], H, 1)
    w = philox([np.broadcast_to(h // 8, (T, H)), t, np.full((T, H), offset & 0xFFFFFFFF), np.full((T, H), offset >> 32)],
               [seed & 0xFFFFFFFF, seed >> 32])
    for i in range(8):
        sel = h % 8 == i
        half = (w[i // 2] >> np.uint64(16 * (i % 2))) & np.uint64(65535)
        out[:, sel] = (half >= thr)[:, sel]
    return torch.from_numpy(out), 65536.0 / (65536 - thr)


def residual(x, y=None, p=0.0, seed=0, offset=0):
    """z = x + dropout(y) in 64 bits; x or y may be None."""
    z = 0.0 if x is None else x.double()
    if y is None:
        return z
    k, mul = keep(*y.shape, p, seed, offset)
    return z + torch.where(k, y.double() * mul, torch.zeros(y.shape, dtype=F64))


# ------------------------------------------------------------------ layer norm

def layer_norm(z, gamma=None, beta=None, eps=1e-5):
    """(x_hat, n, 1 / sqrt(var + eps)) of z, 64 bits."""
    d = z - z.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((d * d).mean(-1, keepdim=True) + eps)
    n = d * r
    hat = n if gamma is None else n * gamma.double()
    return (hat if beta is None else hat + beta.double()), n, r


def norm_error(x, y, mul, z, n, r):
    """How far the kernel's n may be off, and its r in relation to r.

    z: two roundings (the kept y times its factor, the sum).  The mean: sixteen columns a thread, then warps and
    CTA, at most 32 roundings of sums of |z|.  d = z - mean: one more.  The sum of squares: as the mean's; its
    terms are off by 2 |d| e_d.  rsqrt: 2 ulp.
    """
    mag = x.double().abs() + (0.0 if y is None else y.double().abs() * mul)
    d = n / r
    e_d = 2 * U * mag + 40 * U * mag.mean(-1, keepdim=True) + 2 * U * d.abs()
    var = (d * d).mean(-1, keepdim=True)
    rel_r = (d.abs() * e_d).mean(-1, keepdim=True) * r * r + 20 * U * var * r * r + 8 * U
    return e_d * r + n.abs() * (rel_r + 2 * U), rel_r


def layer_norm_grad(z, n, r, gamma, d_x_out, d_x_hat):
    """(D, d_gamma, d_beta) from the formula, 64 bits."""
    dh = d_x_hat.double()
    a = dh if gamma is None else dh * gamma.double()
    D = r * (a - a.mean(-1, keepdim=True) - n * (a * n).mean(-1, keepdim=True))
    if d_x_out is not None:
        D = D + d_x_out.double()
    return D, (dh * n).sum(0), dh.sum(0)


def layer_norm_grad_bounds(n, r, e_n, rel_r, gamma, d_x_out, d_x_hat):
    """Bounds of the three before an output's own rounding."""
    dh = d_x_hat.double().abs()
    a = dh if gamma is None else dh * gamma.double().abs()
    an, na = (a * n.abs()).mean(-1, keepdim=True), n.abs()
    inner = a + a.mean(-1, keepdim=True) + na * an
    e = r * (inner * (rel_r + 48 * U) + e_n * an + na * (a * e_n).mean(-1, keepdim=True) + e_n * (a * e_n).mean(-1, keepdim=True))
    if d_x_out is not None:
        e = e + 4 * U * d_x_out.double().abs()
    T = n.shape[0]
    adds = (min(T, 256) + 64) * U
    return e, (dh * e_n).sum(0) + adds * (dh * (na + e_n)).sum(0), adds * dh.sum(0)


# ------------------------------------------------------------------ int8

def i8_quantize(x):
    """(q int8, scale fp32) by the written definition: both quotients fp32, ties to even."""
    f = x.float()
    top = f.abs().amax(-1)
    bad = ~torch.isfinite(f).all(-1)
    s = torch.where(bad, torch.full_like(top, math.nan), top / torch.full_like(top, 127.0))
    safe = torch.where((s > 0) & ~bad, s, torch.ones_like(s))[:, None]
    q = torch.where(((s > 0) & ~bad)[:, None], torch.round(f / safe).clamp(-127, 127), torch.zeros_like(f))
    return q.to(torch.int8), s


def i8_gemm(xq, sx, wq, sw):
    """(y, bound) in 64 bits: the bound before the rounding to bf16.

    Products are exact; a sum within 2^24 too.  Beyond, each MMA of 16 k cuts the fp32 sum to 24 bits, which takes less
    than 2^-23 of a sum of at most sum |x w|, and there are K / 16 of them: K 2^-27 sum |x w|.
    """
    x, w = xq.double(), wq.double()
    s = sx.double()[:, None] * sw.double()
    y = (x @ w.t()) * s
    mag = (x.abs() @ w.abs().t()) * s.abs()
    return y, 4 * U * y.abs() + (xq.shape[1] * 2.0 ** -27 * mag if xq.shape[1] > 1024 else 0.0) + 2.0 ** -133


def bf16_bound(want, e):
    """A value off by e before one rounding to bf16."""
    return e + BF16_HALF * (want.abs() + e) + 2.0 ** -134
