"""Measured cases of the operators around a routed block: the router's top-k with its balance loss, the norms
before and after a block, and products with 4-bit weights.

Each operator has a plain form (elementary torch operations in 32 bits) and, with `own` set, the framework's call.

  router       logits [T, E] -> top-k experts and gate weights, per-expert counts, balance and z loss; their gradients
  block_norm   x + scale * gate * RMSNorm(y), and the RMSNorm of that sum for the next block; their gradients
  w4_quantize  bf16 weights -> 4 bits with one bf16 scale per group of inputs, and back to bf16
  w4_gemv      y = x W^T for a few rows of x, W in 4 bits
  w4_experts   the routed SwiGLU experts of a few tokens, W in 4 bits

A 4-bit weight is w[n, k] = scale[k // group, n] * (q[n, k] - 8); q[n, 2i] is the low and q[n, 2i + 1] the high half of
byte i of row n.
"""
import math

import torch

own = False

EPS = 1e-5
SCALE = 0.5  # the residual scale of the norm cases

_workspaces = {}


def listed():
    return [
        # The split-K configuration's weight (the Mixtral-shaped down projection), one token: decoding.
        {"name": "gemv_m1_n4096_k14336", "op": "w4_gemv", "M": 1, "N": 4096, "K": 14336, "group": 128},
        # The size of the split-K smoke test, three tokens: what a call costs when it has little to do.
        {"name": "gemv_m3_n256_k1024", "op": "w4_gemv", "M": 3, "N": 256, "K": 1024, "group": 32},
        # The MLP configuration's gate or up projection for a batch of 16 sequences.
        {"name": "gemv_m16_n14336_k4096", "op": "w4_gemv", "M": 16, "N": 14336, "K": 4096, "group": 64},
        # The fine-grained configuration, one token: 8 of 128 small experts.
        {"name": "experts_fine_t1", "op": "w4_experts", "T": 1, "H": 2048, "F": 768, "E": 128, "k": 8, "group": 128},
        # The same with 32 tokens: most experts are touched by one to three rows.
        {"name": "experts_fine_t32", "op": "w4_experts", "T": 32, "H": 2048, "F": 768, "E": 128, "k": 8, "group": 64},
        # The Mixtral-shaped configuration with 4 tokens: few large experts.
        {"name": "experts_mixtral_t4", "op": "w4_experts", "T": 4, "H": 4096, "F": 14336, "E": 8, "k": 2, "group": 128},
        # The tiny configuration's router at its largest batch, as in decoding.
        {"name": "router_decode_t16", "op": "router", "T": 16, "E": 8, "k": 2, "masked": False, "backward": False},
        # A training batch of the fine-grained router, with padded tokens: forward and backward.
        {"name": "router_train_t16384", "op": "router", "T": 16384, "E": 128, "k": 8, "masked": True, "backward": True},
        # Between two blocks while decoding one token, with a per-channel gate.
        {"name": "norm_decode_h4096", "op": "block_norm", "T": 1, "H": 4096, "gate": "channel", "post": True, "backward": False},
        # A training batch with a full gate: forward and backward.
        {"name": "norm_train_t4096_h4096", "op": "block_norm", "T": 4096, "H": 4096, "gate": "full", "post": True, "backward": True},
        # One small ragged weight.
        {"name": "quantize_n1000_k2048", "op": "w4_quantize", "E": 1, "N": 1000, "K": 2048, "group": 32},
        # The gate projections of all Mixtral-shaped experts, laid out when a model is loaded.
        {"name": "quantize_e8_n14336_k4096", "op": "w4_quantize", "E": 8, "N": 14336, "K": 4096, "group": 128},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _multiple(rng, lo, hi, of):
    return max(1, _log(rng, lo, hi) // of) * of


def draw(rng):
    op = rng.choice(["w4_gemv", "w4_experts", "router", "block_norm", "w4_quantize"])
    group = rng.choice([32, 64, 128])
    if op == "w4_gemv":
        return {"op": op, "M": _log(rng, 1, 64), "N": _multiple(rng, 8, 16384, 8), "K": _multiple(rng, 128, 16384, group), "group": group}
    if op == "w4_experts":
        E = _log(rng, 1, 256)
        H, F = _multiple(rng, 128, 4096, group), _multiple(rng, 128, 14336, group)
        while E * H * F > 8 * 4096 * 14336:
            E = max(1, E // 2)
        return {"op": op, "T": _log(rng, 1, 64), "H": H, "F": F, "E": E, "k": rng.randint(1, min(8, E)), "group": group}
    if op == "router":
        E = _log(rng, 2, 256)
        return {"op": op, "T": _log(rng, 1, 65536), "E": E, "k": rng.randint(1, min(8, E)), "masked": rng.random() < 0.5, "backward": rng.random() < 0.6}
    if op == "block_norm":
        T = _log(rng, 1, 8192)
        H = min(_log(rng, 32, 8192), 4096 * 4096 // T)
        H = H if rng.random() < 0.3 else max(8, H // 8 * 8)
        return {"op": op, "T": T, "H": H, "gate": rng.choice(["none", "channel", "token", "full"]), "post": rng.random() < 0.7, "backward": rng.random() < 0.6}
    E = _log(rng, 1, 16)
    N, K = _multiple(rng, 8, 16384, 8), _multiple(rng, 128, 16384, group)
    while E * N * K > 8 * 14336 * 4096:
        E, N = max(1, E // 2), max(8, N // 16 * 8)
    return {"op": op, "E": E, "N": N, "K": K, "group": group}


def work(case):
    c = case
    if c["op"] == "w4_gemv":
        M, N, K, G = c["M"], c["N"], c["K"], c["group"]
        return {"bytes": N * K / 2 + K // G * N * 2 + M * K * 2 + M * N * 2, "flops": 2.0 * M * N * K}
    if c["op"] == "w4_experts":
        T, H, F, E, k, G = (c[n] for n in ("T", "H", "F", "E", "k", "group"))
        touched = E * (1 - (1 - k / E) ** T)
        return {"bytes": touched * 3 * H * F * (0.5 + 2 / G) + 2 * T * H * 2 + T * k * 8, "flops": 2.0 * T * k * 3 * H * F}
    if c["op"] == "w4_quantize":
        n = c["E"] * c["N"] * c["K"]
        return {"bytes": 2 * n * (2 + 0.5 + 2 / c["group"]), "flops": 4.0 * n}
    if c["op"] == "router":
        T, E, k = c["T"], c["E"], c["k"]
        n = 4 * T * E + 8 * T * k + (T if c["masked"] else 0) + 8 * E
        return {"bytes": n + (4 * T * E + 4 * T * k if c["backward"] else 0), "flops": (14.0 if c["backward"] else 6.0) * T * E}
    T, H = c["T"], c["H"]
    full = 1 if c["gate"] == "full" else 0
    n = 2 * T * H * (4 + full + (4 + full if c["backward"] else 0))
    n += 2 * H * 2 + (3 * 4 * H if c["backward"] else 0) + (8 * T if c["gate"] == "token" else 0)
    return {"bytes": n, "flops": (40.0 if c["backward"] else 10.0) * T * H}


# ---------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _w4_weight(g, E, N, K, group, std):
    """A 4-bit weight of [E, N, K] drawn N(0, std^2): bytes [E, N, K / 2] and scales [E, K / group, N]."""
    q = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.empty((E, K // group, N), dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        w = (_randn(g, N, K) * std).reshape(N, K // group, group)
        se = (w.abs().amax(-1) / 7).to(torch.bfloat16)
        v = (torch.round(w / se.float()[..., None]).clamp(-8, 7) + 8).to(torch.uint8).reshape(N, K)
        q[e] = v[:, 0::2] | (v[:, 1::2] << 4)
        s[e] = se.t()
    return q, s


def prepare(case, seed):
    c, g = case, _gen(seed)
    bf = torch.bfloat16
    st = {"case": c}
    if c["op"] == "w4_gemv":
        M, N, K = c["M"], c["N"], c["K"]
        st["x"] = _randn(g, M, K).to(bf)
        q, s = _w4_weight(g, 1, N, K, c["group"], 1 / math.sqrt(K))
        st["q"], st["s"] = q[0], s[0]
        st["y"] = torch.empty((M, N), dtype=bf, device="cuda")
    elif c["op"] == "w4_experts":
        T, H, F, E, k, G = (c[n] for n in ("T", "H", "F", "E", "k", "group"))
        st["x"] = _randn(g, T, H).to(bf)
        logits = _randn(g, T, E)
        val, idx = torch.sort(logits, dim=-1, descending=True, stable=True)
        st["idx"] = idx[:, :k].to(torch.int32).contiguous()
        st["w"] = torch.softmax(val[:, :k], -1)
        st["gate"] = _w4_weight(g, E, F, H, G, 1 / math.sqrt(H))
        st["up"] = _w4_weight(g, E, F, H, G, 1 / math.sqrt(H))
        st["down"] = _w4_weight(g, E, H, F, G, 1 / math.sqrt(F))
        st["out"] = torch.empty((T, H), dtype=bf, device="cuda")
    elif c["op"] == "w4_quantize":
        E, N, K, G = (c[n] for n in ("E", "N", "K", "group"))
        st["w"] = torch.empty((E, N, K), dtype=bf, device="cuda")
        for e in range(E):
            st["w"][e] = (_randn(g, N, K) * 0.02).to(bf)
        st["q"] = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
        st["s"] = torch.empty((E, K // G, N), dtype=bf, device="cuda")
        st["back"] = torch.empty((E, N, K), dtype=bf, device="cuda")
    elif c["op"] == "router":
        T, E, k = c["T"], c["E"], c["k"]
        st["logits"] = _randn(g, T, E) + 0.7 * _randn(g, E)  # some experts are hot
        st["mask"] = None
        if c["masked"]:  # right-padded sequences: about a tenth of the tokens are padding
            st["mask"] = (torch.rand((T,), generator=g, device="cuda") > 0.1).to(torch.uint8)
        st["d_losses"] = torch.tensor([1e-2, 1e-3], device="cuda")
        st["d_w"] = _randn(g, T, k) / T
        st["idx"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        st["w"] = torch.empty((T, k), device="cuda")
        st["counts"] = torch.empty((E,), dtype=torch.int32, device="cuda")
        st["n"] = torch.empty((1,), dtype=torch.int32, device="cuda")
        st["mean_prob"] = torch.empty((E,), device="cuda")
        st["losses"] = torch.empty((2,), device="cuda")
        st["d_logits"] = torch.empty((T, E), device="cuda")
    else:
        T, H = c["T"], c["H"]
        st["x"], st["y"] = _randn(g, T, H).to(bf), (2 * _randn(g, T, H)).to(bf)
        st["gpost"] = (1 + 0.1 * _randn(g, H)).to(bf) if c["post"] else None
        st["gpre"] = (1 + 0.1 * _randn(g, H)).to(bf)
        st["gate"] = {"none": lambda: None, "channel": lambda: (0.5 + 0.2 * _randn(g, H)).to(bf),
                      "token": lambda: torch.sigmoid(_randn(g, T)),
                      "full": lambda: torch.sigmoid(_randn(g, T, H)).to(bf)}[c["gate"]]()
        st["dz"], st["dhat"] = _randn(g, T, H).to(bf), _randn(g, T, H).to(bf)
        st["x_out"], st["x_hat"] = torch.empty_like(st["x"]), torch.empty_like(st["x"])
        st["dx"], st["dy"] = torch.empty_like(st["x"]), torch.empty_like(st["x"])
        st["dgpost"] = torch.empty((H,), device="cuda") if c["post"] else None
        st["dgpre"] = torch.empty((H,), device="cuda")
        st["dgate"] = {"none": lambda: None, "channel": lambda: torch.empty((H,), device="cuda"),
                       "token": lambda: torch.empty((T,), device="cuda"),
                       "full": lambda: torch.empty_like(st["x"])}[c["gate"]]()
    return st


# ---------------------------------------------------------------------------------------------- plain forms

def _expand(q, s, group):
    """The values of a 4-bit weight, fp32 [..., N, K]."""
    v = torch.stack((q & 15, q >> 4), dim=-1).flatten(-2).float() - 8
    return v * s.float().transpose(-1, -2).repeat_interleave(group, dim=-1)


def _plain_gemv(st):
    return (st["x"].float() @ _expand(st["q"], st["s"], st["case"]["group"]).t()).to(torch.bfloat16)


def _silu(v):
    return v / (1 + torch.exp(-v))


def _plain_experts(st):
    c = st["case"]
    G, T, E, k = c["group"], c["T"], c["E"], c["k"]
    x, idx = st["x"].float(), st["idx"].long()
    if T * k <= E:  # the weights of each routed row
        e = idx.reshape(-1)
        rows = x.repeat_interleave(k, 0)[:, :, None]
        g = _expand(st["gate"][0][e], st["gate"][1][e], G) @ rows
        u = _expand(st["up"][0][e], st["up"][1][e], G) @ rows
        h = (_silu(g) * u).to(torch.bfloat16).float()  # h is held in 16 bits by definition
        y = (_expand(st["down"][0][e], st["down"][1][e], G) @ h).reshape(T, k, -1)
        return (st["w"][:, :, None] * y).sum(1).to(torch.bfloat16)
    g = torch.matmul(x, _expand(*st["gate"], G).transpose(-1, -2))  # every expert on every token
    u = torch.matmul(x, _expand(*st["up"], G).transpose(-1, -2))
    h = (_silu(g) * u).to(torch.bfloat16).float()
    y = torch.matmul(h, _expand(*st["down"], G).transpose(-1, -2))
    share = torch.zeros((T, E), device="cuda").scatter_(1, idx, st["w"])
    return (share.t()[:, :, None] * y).sum(0).to(torch.bfloat16)


def _plain_quantize(st):
    c = st["case"]
    E, N, K, G = (c[n] for n in ("E", "N", "K", "group"))
    w = st["w"].float().reshape(E, N, K // G, G)
    s = (w.abs().amax(-1) / 7).to(torch.bfloat16)
    f = s.float()[..., None]
    v = torch.where(f > 0, torch.round(w / f).clamp(-8, 7), torch.zeros_like(w))
    return (v * f).reshape(E, N, K).to(torch.bfloat16), s.transpose(-1, -2).contiguous()


def _plain_router(st):
    c = st["case"]
    E, k = c["E"], c["k"]
    L = st["logits"]
    top = L.amax(-1, keepdim=True)
    live = top[:, 0] > -math.inf
    if st["mask"] is not None:
        live = live & (st["mask"] != 0)
    val, order = torch.sort(L, dim=-1, descending=True, stable=True)
    val = val[:, :k]
    on = live[:, None] & (val > -math.inf)
    idx = torch.where(on, order[:, :k], -1).to(torch.int32)
    ex = torch.where(on, torch.exp(val - val[:, :1]), 0.0)
    w = torch.where(on, ex / ex.sum(-1, keepdim=True), 0.0)
    counts = torch.bincount((idx + 1).reshape(-1), minlength=E + 1)[1:].to(torch.int32)
    n = live.sum().to(torch.int32).reshape(1)
    rows = n.clamp(min=1).float()
    ex = torch.exp(L - top)
    z = ex.sum(-1, keepdim=True)
    p = torch.where(live[:, None], ex / z, 0.0)
    lse = torch.where(live[:, None], top + torch.log(z), 0.0)
    mean_prob = p.double().sum(0).float() / rows
    f = counts.float() / (rows * k)
    losses = torch.stack((E * (f * mean_prob).sum(), (lse.double() ** 2).sum().float() / rows[0]))
    out = {"idx": idx, "w": w, "counts": counts, "n": n, "mean_prob": mean_prob, "losses": losses}
    if c["backward"]:
        db, dz = st["d_losses"][0], st["d_losses"][1]
        cost = E * f / rows
        d = db * p * (cost - (p * cost).sum(-1, keepdim=True)) + dz * 2 / rows * lse * p
        dw = torch.where(on, st["d_w"], 0.0)
        dsel = w * (dw - (w * dw).sum(-1, keepdim=True))
        out["d_logits"] = d.scatter_add_(1, idx.long().clamp(min=0), torch.where(on, dsel, 0.0))
    return out


def _plain_norm(st):
    c = st["case"]
    H = c["H"]
    x, y = st["x"].float(), st["y"].float()
    one = torch.ones((), device="cuda")
    gpost = st["gpost"].float() if c["post"] else one
    gpre = st["gpre"].float()
    gate = one if st["gate"] is None else st["gate"].float()[:, None] if c["gate"] == "token" else st["gate"].float()
    ry = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) if c["post"] else one
    n = y * ry * gpost
    z = x + SCALE * gate * n
    rz = torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS)
    out = {"x_out": z.to(torch.bfloat16), "x_hat": (z * rz * gpre).to(torch.bfloat16)}
    if not c["backward"]:
        return out
    dhat = st["dhat"].float()
    a = dhat * gpre
    dz = st["dz"].float() + rz * a - z * rz ** 3 * ((a * z).sum(-1, keepdim=True) / H)
    dn = SCALE * gate * dz
    dy = dn
    if c["post"]:
        b = dn * gpost
        dy = ry * b - y * ry ** 3 * ((b * y).sum(-1, keepdim=True) / H)
        out["d_gamma_post"] = (dn * y * ry).sum(0)
    out.update(dx=dz.to(torch.bfloat16), dy=dy.to(torch.bfloat16), d_gamma_pre=(dhat * z * rz).sum(0))
    dg = SCALE * n * dz
    if c["gate"] == "channel":
        out["d_gate"] = dg.sum(0)
    elif c["gate"] == "token":
        out["d_gate"] = dg.sum(-1)
    elif c["gate"] == "full":
        out["d_gate"] = dg.to(torch.bfloat16)
    return out


# ---------------------------------------------------------------------------------------------- the framework's calls

def _workspace(op, nbytes):
    """One zeroed workspace an operator, kept and grown as a program on one stream keeps it."""
    ws = _workspaces.get(op)
    if ws is None or ws.numel() < nbytes:
        from moe_task_scheduling_gb300 import etmoe
        ws = _workspaces[op] = etmoe.alloc_workspace(nbytes)
    return ws


def _own(st):
    from moe_task_scheduling_gb300 import etmoe as et
    c = st["case"]
    if c["op"] == "w4_gemv":
        ws = _workspace("gemv", et.et_w4_gemv_workspace_bytes(c["M"], c["N"], c["K"], c["group"]))
        et.et_w4_gemv(st["x"], st["q"], st["s"], st["y"], workspace=ws)
        return st["y"]
    if c["op"] == "w4_experts":
        ws = _workspace("experts", et.et_w4_experts_workspace_bytes(c["T"], c["H"], c["F"], c["E"], c["k"], c["group"]))
        et.et_w4_experts(st["x"], st["idx"], st["w"], *st["gate"], *st["up"], *st["down"], st["out"], workspace=ws)
        return st["out"]
    if c["op"] == "w4_quantize":
        et.et_w4_quantize(st["w"], st["q"], st["s"])
        et.et_w4_dequantize(st["q"], st["s"], st["back"])
        return st["back"], st["s"]
    if c["op"] == "router":
        ws = _workspace("router", et.et_router_topk_workspace_bytes(c["T"], c["E"], c["k"]))
        et.et_router_topk(st["logits"], st["idx"], st["w"], token_mask=st["mask"], expert_counts=st["counts"],
                          n_routed=st["n"], mean_prob=st["mean_prob"], losses=st["losses"], workspace=ws)
        out = {"idx": st["idx"], "w": st["w"], "counts": st["counts"], "n": st["n"], "mean_prob": st["mean_prob"],
               "losses": st["losses"]}
        if c["backward"]:
            et.et_router_topk_bwd(st["logits"], st["idx"], st["w"], st["counts"], st["n"], st["d_logits"],
                                  token_mask=st["mask"], d_losses=st["d_losses"], d_topk_w=st["d_w"], workspace=ws)
            out["d_logits"] = st["d_logits"]
        return out
    ws = _workspace("norm", et.et_block_norm_workspace_bytes(c["T"], c["H"]))
    args = dict(gamma_post=st["gpost"], gate=st["gate"], scale=SCALE, gamma_pre=st["gpre"], eps=EPS, workspace=ws)
    et.et_block_norm(st["x"], st["y"], st["x_out"], st["x_hat"], **args)
    out = {"x_out": st["x_out"], "x_hat": st["x_hat"]}
    if c["backward"]:
        et.et_block_norm_bwd(st["x"], st["y"], st["dz"], st["dhat"], st["dx"], st["dy"], d_gamma_post=st["dgpost"],
                             d_gamma_pre=st["dgpre"], d_gate=st["dgate"], **args)
        out.update(dx=st["dx"], dy=st["dy"], d_gamma_pre=st["dgpre"])
        if c["post"]:
            out["d_gamma_post"] = st["dgpost"]
        if c["gate"] != "none":
            out["d_gate"] = st["dgate"]
    return out


_PLAIN = {"w4_gemv": _plain_gemv, "w4_experts": _plain_experts, "w4_quantize": _plain_quantize,
          "router": _plain_router, "block_norm": _plain_norm}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------- 64 bits

def _weight64(q, s):
    """fp64 [N, K] of one 4-bit weight, from the definition w[n, k] = scale[k // group, n] * (q - 8)."""
    N, K = q.shape[0], 2 * q.shape[1]
    k = torch.arange(K, device=q.device)
    nib = (q.to(torch.int16)[:, k // 2] >> (4 * (k % 2)).to(torch.int16)) & 15
    return s.double()[k // (K // s.shape[0])].t() * (nib - 8).double()


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    if c["op"] == "w4_gemv":
        return torch.einsum("nk,mk->mn", _weight64(st["q"], st["s"]), st["x"].double())
    if c["op"] == "w4_experts":
        out = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device="cuda")
        idx = st["idx"].cpu()
        for e in sorted(set(idx.reshape(-1).tolist())):
            t, j = (v.cuda() for v in torch.nonzero(idx == e, as_tuple=True))
            x = st["x"].double()[t]
            g, u = (torch.einsum("fh,rh->rf", _weight64(st[n][0][e], st[n][1][e]), x) for n in ("gate", "up"))
            h = (g * torch.sigmoid(g) * u).to(torch.bfloat16).double()
            y = torch.einsum("hf,rf->rh", _weight64(st["down"][0][e], st["down"][1][e]), h)
            out.index_add_(0, t, st["w"].double()[t, j][:, None] * y)
        return out
    if c["op"] == "w4_quantize":
        w = st["w"]
        E, N, K = w.shape
        back = torch.empty((E, N, K), dtype=torch.float64, device="cuda")
        scales = torch.empty((E, K // c["group"], N), dtype=torch.float64, device="cuda")
        for e in range(E):
            v = w[e].double().unflatten(1, (-1, c["group"]))
            s = (v.abs().max(-1).values / 7).float().to(torch.bfloat16).double()  # the stored scale is 16 bits by definition
            r = torch.where(s[..., None] > 0, v / s[..., None], 0.0).float().double()  # and the quotient 32 bits before it is rounded
            back[e] = (torch.clamp(torch.round(r), -8, 7) * s[..., None]).flatten(1)
            scales[e] = s.t()
        return back, scales
    if c["op"] == "router":
        T, E, k = c["T"], c["E"], c["k"]
        L = st["logits"].double()
        keep = torch.ones((T,), dtype=torch.bool, device="cuda") if st["mask"] is None else st["mask"].bool()
        Tn = max(1, int(keep.sum()))
        p = torch.softmax(L, -1) * keep[:, None]
        lse = torch.logsumexp(L, -1) * keep
        sel = torch.argsort(-L, dim=-1, stable=True)[:, :k]
        wt = torch.softmax(torch.gather(L, 1, sel), -1) * keep[:, None]
        picked = torch.zeros((T, E), dtype=torch.float64, device="cuda").scatter_(1, sel, 1.0) * keep[:, None]
        f = picked.sum(0) / (Tn * k)
        P = p.sum(0) / Tn
        res = {"idx": None, "w": wt, "counts": None, "n": None, "mean_prob": P,
               "losses": torch.stack((E * torch.dot(f, P), torch.dot(lse, lse) / Tn))}
        if c["backward"]:
            b, z = st["d_losses"].double().tolist()
            grad_p = b * E * f[None, :] / Tn
            d = p * (grad_p - torch.einsum("te,e->t", p, grad_p[0])[:, None]) + z * 2 * lse[:, None] / Tn * p
            dw = st["d_w"].double()
            d += torch.zeros_like(d).scatter_(1, sel, wt * (dw - torch.einsum("tk,tk->t", wt, dw)[:, None]))
            res["d_logits"] = d
        return res
    H = c["H"]
    x, y, gpre = st["x"].double(), st["y"].double(), st["gpre"].double()
    gpost = st["gpost"].double() if c["post"] else torch.ones((H,), dtype=torch.float64, device="cuda")
    gate = torch.ones((1, 1), dtype=torch.float64, device="cuda") if st["gate"] is None else st["gate"].double()
    gate = gate.reshape({"none": (1, 1), "channel": (1, H), "token": (-1, 1), "full": (-1, H)}[c["gate"]])
    uy = y / torch.sqrt(y.square().mean(-1, keepdim=True) + EPS) if c["post"] else y
    z = x + SCALE * gate * (uy * gpost)
    sz = torch.sqrt(z.square().mean(-1, keepdim=True) + EPS)
    res = {"x_out": z, "x_hat": z / sz * gpre}
    if not c["backward"]:
        return res
    dhat = st["dhat"].double()
    uz = z / sz
    du = dhat * gpre
    d = st["dz"].double() + (du - uz * (du * uz).mean(-1, keepdim=True)) / sz
    dn = SCALE * gate * d
    res["dx"], res["d_gamma_pre"] = d, torch.einsum("th,th->h", dhat, uz)
    if c["post"]:
        sy = torch.sqrt(y.square().mean(-1, keepdim=True) + EPS)
        dv = dn * gpost
        res["dy"] = (dv - uy * (dv * uy).mean(-1, keepdim=True)) / sy
        res["d_gamma_post"] = torch.einsum("th,th->h", dn, uy)
    else:
        res["dy"] = dn
    dg = SCALE * (uy * gpost) * d
    if c["gate"] != "none":
        res["d_gate"] = {"channel": lambda: dg.sum(0), "token": lambda: dg.sum(1), "full": lambda: dg}[c["gate"]]()
    return res
