"""Routed 4-bit experts on inputs whose gate and up products are exact, with a bound that shows a lost row or group.

x are integers up to 4 and scales powers of two, so every sum of gate and up is a multiple of the smallest scale
below 2^24 of it and fp32 holds it exactly.  What is left: silu(g) u in fp32, its rounding to bf16, the sums of the
down product and the output's rounding."""
import math

import torch

from tests.ref_ops import BF16_HALF, F32_HALF, F64, w4_values

BF = torch.bfloat16

# every form of the two products: clusters, units in turn, passes of 4, 8 and 16 rows, a warp a unit alone in one
# product or both, CTAs of eight warps
SIZES = [(1, 64, 32, 1, 1, 32), (1, 256, 512, 8, 2, 128), (16, 256, 512, 8, 2, 64), (5, 96, 160, 4, 4, 32), (3, 640, 128, 200, 8, 128),
         (64, 128, 128, 16, 8, 64), (33, 192, 320, 3, 2, 64), (64, 64, 64, 2, 2, 32), (7, 2048, 768, 16, 8, 128), (20, 160, 1120, 5, 1, 32),
         (64, 256, 256, 256, 8, 128), (64, 416, 288, 256, 8, 32), (64, 64, 1568, 200, 8, 32), (50, 128, 3200, 60, 8, 128),
         (33, 4096, 320, 6, 2, 64), (64, 4128, 96, 2, 2, 32)]


def inputs(T, H, F, En, k, group, seed):
    """x, idx, w, gate, up, down as the library takes them; g and u of order 2."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-4, 5, (T, H), generator=g).to(BF)

    def weight(N, K, size):
        q = torch.randint(0, 256, (En, N, K // 2), generator=g).to(torch.uint8)
        e = round(math.log2(2 / (12 * math.sqrt(K) * size)))
        return q, (2.0 ** (e - torch.randint(0, 2, (En, K // group, N), generator=g))).to(BF)
    gate, up, down = weight(F, H, 1), weight(F, H, 1), weight(H, F, 0.5)
    val, idx = torch.topk(torch.randn(T, En, generator=g), k, -1)
    return x, idx.to(torch.int32), torch.softmax(val, -1), gate, up, down


def experts(x, idx, w, gate, up, down, drop=None):
    """(out, bound without the output's rounding) in 64 bits.  drop: what a faulty kernel would lose -- "row" the
    last expert of the last token, "up" or "down" 32 inputs of that product for that expert's rows."""
    T, H = x.shape
    F = gate[0].shape[1]
    out, bound = torch.zeros(T, H, dtype=F64), torch.zeros(T, H, dtype=F64)
    last = int(idx[T - 1, -1])
    for e in sorted(set(idx.reshape(-1).tolist()) - {-1}):
        wg, wu, wd = (w4_values(a[0][e], a[1][e]) for a in (gate, up, down))
        if e == last and drop == "up":
            wu[:, H - 32:] = 0
        if e == last and drop == "down":
            wd[:, F - 32:] = 0
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if e == last and drop == "row":
            keep = ~((t == T - 1) & (j == idx.shape[1] - 1))
            t, j = t[keep], j[keep]
        g, u = x[t].double() @ wg.t(), x[t].double() @ wu.t()
        h = g * torch.sigmoid(g) * u
        h16 = h.to(BF).double()
        # exp (2 ulp), a sum, a division and a product: 8 roundings; where they can lead to another bf16 value, the step
        dh = ((h * (1 + 8 * F32_HALF)).to(BF).double() - (h * (1 - 8 * F32_HALF)).to(BF).double()).abs()
        wt = w[t, j].double()[:, None]
        out.index_add_(0, t, wt * (h16 @ wd.t()))
        # products are exact; F additions and one a group (truncated at worst: two half steps), the splits', the experts'
        bound.index_add_(0, t, wt * ((dh + 2 * (F + F / 32 + 64) * F32_HALF * h16.abs()) @ wd.abs().t()))
    return out, bound


def tolerance(want, bound):
    return BF16_HALF * (want.abs() + bound) + bound + 1e-38
