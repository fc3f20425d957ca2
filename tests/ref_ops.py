"""Plain 64-bit definitions of the router, norm and 4-bit weight operators, and the error bounds that go
with them.  Test infrastructure: shares no code with the CUDA path.

A rounding to bf16 is off by at most half a step, 2^-8 of the value; to fp32, 2^-24.  Every bound here is
(one rounding of the output) + (number of fp32 roundings on the way to it) * 2^-24 * (sum of the magnitudes
that were added), the latter returned beside each value.
"""
import math

import torch

BF16_HALF = 2.0 ** -8
F32_HALF = 2.0 ** -24
F64 = torch.float64


# ------------------------------------------------------------------ router

def router(logits, k, mask=None):
    """Selection and losses in 64 bits; logits may require grad (fp64 then)."""
    L = logits.double()
    T, E = L.shape
    live = (L > -math.inf).any(-1) | torch.isnan(L).any(-1)
    if mask is not None:
        live &= mask.bool()
    # order by (logit desc, index asc): a stable sort of the negated values
    order = torch.argsort(-L.detach(), dim=-1, stable=True)[:, :k]
    val = torch.gather(L, 1, order)
    on = live[:, None] & (val.detach() > -math.inf)
    idx = torch.where(on, order, -1)
    # a row with nothing to choose takes part as zeros that carry no gradient
    safe = torch.where(on, val, torch.full_like(val, -math.inf))
    top = torch.where(on[:, :1], val[:, :1].detach(), torch.zeros_like(val[:, :1]))
    ex = torch.where(on, torch.exp(safe - top), torch.zeros_like(safe))
    z = ex.sum(-1, keepdim=True)
    w = ex / torch.where(z > 0, z, torch.ones_like(z))
    counts = torch.zeros(E, dtype=F64).index_add_(0, idx[on], torch.ones(int(on.sum()), dtype=F64))
    n = int(live.sum())
    rows = max(n, 1)
    Ls = torch.where(live[:, None], L, torch.zeros_like(L))
    p = torch.where(live[:, None], torch.softmax(Ls, -1), torch.zeros_like(L))
    lse = torch.where(live, torch.logsumexp(Ls, -1), torch.zeros(T, dtype=F64))
    mean_prob = p.sum(0) / rows
    losses = torch.stack((E * (counts / (rows * k) * mean_prob).sum(), (lse ** 2).sum() / rows))
    return dict(idx=idx, w=w, counts=counts, n=n, mean_prob=mean_prob, losses=losses, p=p, lse=lse, live=live)


def router_grad(logits, k, d_losses, d_w, mask=None):
    """d_logits by automatic differentiation of router(), 64 bits."""
    L = logits.double().clone().requires_grad_(True)
    r = router(L, k, mask)
    total = (r["losses"] * d_losses.double()).sum()
    if d_w is not None:
        total = total + torch.where(r["idx"] >= 0, r["w"] * d_w.double(), torch.zeros_like(r["w"])).sum()
    (g,) = torch.autograd.grad(total, L)
    return torch.where(torch.isnan(g) & ~torch.isfinite(logits.double()), torch.zeros_like(g), g)


# ------------------------------------------------------------------ norms

def block_norm(x, y=None, gamma_post=None, gate=None, scale=1.0, gamma_pre=None, eps=1e-5):
    """z and x_hat in 64 bits (gate already broadcastable)."""
    z = x
    if y is not None:
        n = y
        if gamma_post is not None:
            n = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * gamma_post
        z = x + scale * (n if gate is None else gate * n)
    hat = None
    if gamma_pre is not None:
        hat = z / torch.sqrt((z * z).mean(-1, keepdim=True) + eps) * gamma_pre
    return z, hat


# ------------------------------------------------------------------ 4-bit weights

def w4_pack(w, group):
    """bf16 [.., N, K] -> q uint8 [.., N, K/2], scale bf16 [.., K/group, N], by the written definition."""
    f = w.float()
    lead, (N, K) = w.shape[:-2], w.shape[-2:]
    g = f.reshape(*lead, N, K // group, group)
    s = (g.abs().amax(-1) / 7).to(torch.bfloat16)
    bad = ~torch.isfinite(g).all(-1)
    s = torch.where(bad, torch.full_like(s, math.nan), s)
    sf = s.float()[..., None]
    v = torch.where(sf > 0, torch.round(g / sf).clamp(-8, 7), torch.zeros_like(g))
    v = (v + 8).to(torch.uint8).reshape(*lead, N, K)
    return v[..., 0::2] | (v[..., 1::2] << 4), s.transpose(-1, -2).contiguous()


def w4_values(q, scale, dtype=F64):
    """The values of a 4-bit weight [.., N, K], exact in 64 bits."""
    K = 2 * q.shape[-1]
    n = torch.empty(*q.shape[:-1], K, dtype=dtype)
    n[..., 0::2] = (q & 15).to(dtype)
    n[..., 1::2] = (q >> 4).to(dtype)
    return (n - 8) * scale.to(dtype).transpose(-1, -2).repeat_interleave(K // scale.shape[-2], -1)


def gemv(x, q, scale):
    """(x w^T, sum |x| |w|^T), 64 bits."""
    w = w4_values(q, scale)
    return x.double() @ w.t(), x.double().abs() @ w.abs().t()


def experts(x, idx, w, gate, up, down):
    """(out, bound) of the routed experts with h NOT rounded: 64 bits.

    h is stored as bf16, so the computed h is off by 2^-8 |h| plus what the fp32 sums of g and u add; the
    bound carries that through the down product."""
    T, H = x.shape
    F = gate[0].shape[1]
    out = torch.zeros(T, H, dtype=F64)
    mag = torch.zeros(T, H, dtype=F64)   # bound without the output's own rounding
    for e in sorted(set(idx.reshape(-1).tolist()) - {-1}):
        wg, wu, wd = (w4_values(a[0][e], a[1][e]) for a in (gate, up, down))
        for t, j in torch.nonzero(idx == e).tolist():
            xt = x[t].double()
            g, u = wg @ xt, wu @ xt
            eg, eu = (2 * H * F32_HALF * (m.abs() @ xt.abs()) for m in (wg, wu))
            sig = torch.sigmoid(g)
            h = g * sig * u
            # |silu'| <= 1.1; exp, the division and two products: 8 roundings
            dh = 1.1 * eg * u.abs() + (g * sig).abs() * eu + 1.1 * eg * eu + 8 * F32_HALF * h.abs()
            dh = dh + BF16_HALF * (h.abs() + dh)
            wt = abs(float(w[t, j]))
            out[t] += float(w[t, j]) * (wd @ h)
            mag[t] += wt * (wd.abs() @ dh + 2 * (F + 16) * F32_HALF * (wd.abs() @ (h.abs() + dh)))
    return out, mag


# ------------------------------------------------------------------ comparison

def check(got, want, bound, what):
    """|got - want| <= bound everywhere; non-finite values have to match."""
    g, w = got.detach().double().cpu(), want.detach().double().cpu()
    b = bound.detach().double().cpu() if isinstance(bound, torch.Tensor) else torch.full_like(w, bound)
    assert g.shape == w.shape, f"{what}: shape {tuple(g.shape)} != {tuple(w.shape)}"
    fin = torch.isfinite(w)
    assert torch.equal(torch.isfinite(g), fin), f"{what}: finite values in other places"
    bad = fin & ((g - w).abs() > b.expand_as(w))
    if bad.any():
        at = torch.nonzero(bad)[0].tolist()
        i = tuple(at)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {at}: {g[i]} vs {w[i]} "
                             f"(bound {b.expand_as(w)[i]})")
