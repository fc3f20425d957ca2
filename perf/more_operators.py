"""Measured cases of further operators around a routed block: the grouped router, the layer norm with residual and
dropout, dropout by itself, and products of 8-bit integers.

Each operator has a plain form (elementary torch operations in 32 bits, in 64 where a choice or a random number hangs
on it) and, with `own` set, the framework's call.

  router_groups  logits [T, E] -> experts chosen by score + bias within the best groups, gate weights, counts, mean
                 scores, balance loss; their gradients
  layer_norm     z = x + dropout(y), and LayerNorm(z); their gradients
  dropout        out = x + dropout(y), and the gradient of y
  i8_linear      x quantised to int8 with a scale per token, times an int8 weight with a scale per channel

The random number of element (t, h) is 16 bits of Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers:
as easy as 1, 2, 3", 2011) with the key `seed` and the counter (h // 8, t, offset): element h % 8 takes the low or
high half of word h % 8 // 2. It is kept if its number is at least round(p * 2^16).
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5

_workspaces = {}


def listed():
    return [
        # Decoding with the fine-grained configuration's experts: 16 tokens, four of eight groups.
        {"name": "router_groups_decode_t16", "op": "router_groups", "T": 16, "E": 128, "k": 8, "G": 8, "kg": 4, "best": 2,
         "score": "sigmoid", "bias": True, "renorm": True, "masked": False, "backward": False},
        # A training batch with as many experts as the router takes and padded tokens: forward and backward.
        {"name": "router_groups_train_t16384", "op": "router_groups", "T": 16384, "E": 256, "k": 8, "G": 8, "kg": 4, "best": 2,
         "score": "sigmoid", "bias": True, "renorm": True, "masked": True, "backward": True},
        # The fine-grained configuration's largest batch: softmax scores, groups ranked by their best expert, weights as they are.
        {"name": "router_groups_softmax_t4096", "op": "router_groups", "T": 4096, "E": 128, "k": 8, "G": 16, "kg": 6, "best": 1,
         "score": "softmax", "bias": False, "renorm": False, "masked": False, "backward": True},
        # Between two blocks while decoding one token: residual and norm.
        {"name": "layer_norm_decode_h4096", "op": "layer_norm", "T": 1, "H": 4096, "y": True, "p": 0.0, "backward": False},
        # A training batch: residual with dropout and norm, forward and backward.
        {"name": "layer_norm_train_t4096_h4096", "op": "layer_norm", "T": 4096, "H": 4096, "y": True, "p": 0.1, "backward": True},
        # A plain norm of an odd width, forward and backward.
        {"name": "layer_norm_t1000_h1001", "op": "layer_norm", "T": 1000, "H": 1001, "y": False, "p": 0.0, "backward": True},
        # Few tokens of the fine-grained configuration: what a call costs when it has little to do.
        {"name": "dropout_t16_h2048", "op": "dropout", "T": 16, "H": 2048, "x": False, "p": 0.5, "backward": False},
        # The last block's residual in a large training batch, forward and backward.
        {"name": "dropout_t8192_h4096", "op": "dropout", "T": 8192, "H": 4096, "x": True, "p": 0.1, "backward": True},
        # The split-K configuration's weight, one token: decoding.
        {"name": "i8_m1_n4096_k14336", "op": "i8_linear", "M": 1, "N": 4096, "K": 14336},
        # The MLP configuration's gate or up projection for a batch of 16 sequences.
        {"name": "i8_m16_n14336_k4096", "op": "i8_linear", "M": 16, "N": 14336, "K": 4096},
        # A ragged one: a prompt of 200 tokens through a narrow projection.
        {"name": "i8_m200_n1000_k2064", "op": "i8_linear", "M": 200, "N": 1000, "K": 2064},
        # The MLP configuration's projection for a large batch of prompts.
        {"name": "i8_m4096_n14336_k4096", "op": "i8_linear", "M": 4096, "N": 14336, "K": 4096},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["router_groups", "layer_norm", "dropout", "i8_linear", "i8_linear"])
    if op == "router_groups":
        G = rng.choice([1, 2, 4, 5, 8, 16])
        E = G * _log(rng, 2, 256 // G)
        kg = rng.randint(1, G)
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(8, E // G * kg)), "G": G, "kg": kg,
                "best": rng.choice([1, 2]), "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.6,
                "renorm": rng.random() < 0.6, "masked": rng.random() < 0.5, "backward": rng.random() < 0.6}
    if op == "layer_norm":
        T = _log(rng, 1, 8192)
        H = min(_log(rng, 32, 8192), 4096 * 4096 // T)
        H = H if rng.random() < 0.3 else max(8, H // 8 * 8)
        y = rng.random() < 0.7
        return {"op": op, "T": T, "H": H, "y": y, "p": rng.choice([0.0, 0.1, 0.25, 0.5]) if y else 0.0, "backward": rng.random() < 0.6}
    if op == "dropout":
        T = _log(rng, 1, 8192)
        H = _log(rng, 32, 8192)
        H = H if rng.random() < 0.3 else max(8, H // 8 * 8)
        return {"op": op, "T": min(T, 8192 * 4096 // H), "H": H, "x": rng.random() < 0.6, "p": rng.choice([0.1, 0.3, 0.5]),
                "backward": rng.random() < 0.5}
    M, N, K = _log(rng, 1, 8192), _log(rng, 8, 16384), _log(rng, 128, 16384) // 16 * 16
    while M * N * K > 4096 * 14336 * 4096:
        M //= 2
    return {"op": op, "M": max(1, M), "N": N, "K": K}


def work(case):
    c = case
    if c["op"] == "router_groups":
        T, E, k = c["T"], c["E"], c["k"]
        n = 4 * T * E + 8 * T * k + (T if c["masked"] else 0) + 8 * E + (4 * E if c["bias"] else 0)
        return {"bytes": n + (4 * T * E + 4 * T * k if c["backward"] else 0), "flops": (16.0 if c["backward"] else 8.0) * T * E}
    if c["op"] == "layer_norm":
        T, H = c["T"], c["H"]
        n = 2 * T * H * ((4 if c["y"] else 2) + ((4 if c["y"] else 2) if c["backward"] else 0))
        return {"bytes": n + 4 * H + (8 * H if c["backward"] else 0), "flops": (30.0 if c["backward"] else 10.0) * T * H}
    if c["op"] == "dropout":
        T, H = c["T"], c["H"]
        return {"bytes": 2 * T * H * ((3 if c["x"] else 2) + (2 if c["backward"] else 0)), "flops": (4.0 if c["backward"] else 2.0) * T * H}
    M, N, K = c["M"], c["N"], c["K"]
    return {"bytes": 2 * M * K + N * K + 4 * N + 2 * M * N + 4 * M, "flops": 2.0 * M * N * K}


# ---------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def prepare(case, seed):
    c, g = case, _gen(seed)
    bf = torch.bfloat16
    st = {"case": c, "seed": 1000003 * seed + 17, "offset": (5 << 32) + seed}
    if c["op"] == "router_groups":
        T, E, k = c["T"], c["E"], c["k"]
        st["logits"] = _randn(g, T, E) + 0.7 * _randn(g, E)  # some experts are hot
        st["bias"] = 0.05 * _randn(g, E) if c["bias"] else None
        st["mask"] = None
        if c["masked"]:  # right-padded sequences: about a tenth of the tokens are padding
            st["mask"] = (torch.rand((T,), generator=g, device="cuda") > 0.1).to(torch.uint8)
        st["d_loss"] = torch.tensor([1e-2], device="cuda")
        st["d_w"] = _randn(g, T, k) / T
        st["idx"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        st["w"] = torch.empty((T, k), device="cuda")
        st["counts"] = torch.empty((E,), dtype=torch.int32, device="cuda")
        st["n"] = torch.empty((1,), dtype=torch.int32, device="cuda")
        st["mean_prob"] = torch.empty((E,), device="cuda")
        st["loss"] = torch.empty((1,), device="cuda")
        st["d_logits"] = torch.empty((T, E), device="cuda")
    elif c["op"] == "layer_norm":
        T, H = c["T"], c["H"]
        st["x"] = _randn(g, T, H).to(bf)
        st["y"] = (2 * _randn(g, T, H)).to(bf) if c["y"] else None
        st["gamma"], st["beta"] = (1 + 0.1 * _randn(g, H)).to(bf), (0.1 * _randn(g, H)).to(bf)
        st["dz"] = _randn(g, T, H).to(bf) if c["y"] else None
        st["dhat"] = _randn(g, T, H).to(bf)
        st["x_out"] = torch.empty_like(st["x"]) if c["y"] else None
        st["x_hat"], st["dx"] = torch.empty_like(st["x"]), torch.empty_like(st["x"])
        st["dy"] = torch.empty_like(st["x"]) if c["y"] else None
        st["dgamma"], st["dbeta"] = torch.empty((H,), device="cuda"), torch.empty((H,), device="cuda")
    elif c["op"] == "dropout":
        T, H = c["T"], c["H"]
        st["y"] = _randn(g, T, H).to(bf)
        st["x"] = _randn(g, T, H).to(bf) if c["x"] else None
        st["d_out"] = _randn(g, T, H).to(bf)
        st["out"], st["dy"] = torch.empty_like(st["y"]), torch.empty_like(st["y"])
    else:
        M, N, K = c["M"], c["N"], c["K"]
        st["x"] = _randn(g, M, K).to(bf)
        w = _randn(g, N, K) / math.sqrt(K)
        st["sw"] = w.abs().amax(-1) / 127
        st["wq"] = torch.round(w / st["sw"][:, None]).clamp(-127, 127).to(torch.int8)
        st["xq"] = torch.empty((M, K), dtype=torch.int8, device="cuda")
        st["sx"] = torch.empty((M,), device="cuda")
        st["out"] = torch.empty((M, N), dtype=bf, device="cuda")
    return st


# ---------------------------------------------------------------------------------------------- plain forms

def _plain_keep(T, H, p, seed, offset):
    """The kept elements, bool [T, H], and what they are multiplied by."""
    thr = int(round(p * 65536))
    m32 = 0xFFFFFFFF
    c0 = torch.arange((H + 7) // 8, device="cuda")[None, :].expand(T, -1)
    c1 = torch.arange(T, device="cuda")[:, None].expand_as(c0)
    c2, c3 = torch.full_like(c0, offset & m32), torch.full_like(c0, offset >> 32)
    k0, k1 = seed & m32, seed >> 32 & m32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # the low 64 bits of each product are right, whatever the sign says
        c0, c1, c2, c3 = (b >> 32 & m32) ^ c1 ^ k0, b & m32, (a >> 32 & m32) ^ c3 ^ k1, a & m32
        k0, k1 = k0 + 0x9E3779B9 & m32, k1 + 0xBB67AE85 & m32
    u = torch.stack((c0 & 65535, c0 >> 16, c1 & 65535, c1 >> 16, c2 & 65535, c2 >> 16, c3 & 65535, c3 >> 16), -1)
    return u.reshape(T, -1)[:, :H] >= thr, 65536.0 / (65536 - thr)


def _plain_dropout(st):
    c = st["case"]
    keep, mul = _plain_keep(c["T"], c["H"], c["p"], st["seed"], st["offset"])
    z = torch.where(keep, st["y"].float() * mul, 0.0)
    if c["x"]:
        z = st["x"].float() + z
    out = {"out": z.to(torch.bfloat16)}
    if c["backward"]:
        out["dy"] = torch.where(keep, st["d_out"].float() * mul, 0.0).to(torch.bfloat16)
    return out


def _plain_norm(st):
    c = st["case"]
    T, H = c["T"], c["H"]
    z = st["x"].float()
    keep, mul = None, 1.0
    if c["p"] > 0:
        keep, mul = _plain_keep(T, H, c["p"], st["seed"], st["offset"])
    if c["y"]:
        y = st["y"].float()
        z = z + (y if keep is None else torch.where(keep, y * mul, 0.0))
    d = z - z.mean(-1, keepdim=True)
    r = torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS)
    n = d * r
    gamma = st["gamma"].float()
    out = {"x_hat": (n * gamma + st["beta"].float()).to(torch.bfloat16)}
    if c["y"]:
        out["x_out"] = z.to(torch.bfloat16)
    if not c["backward"]:
        return out
    dhat = st["dhat"].float()
    a = dhat * gamma
    dz = r * (a - a.mean(-1, keepdim=True) - n * (a * n).mean(-1, keepdim=True))
    if c["y"]:
        dz = st["dz"].float() + dz
        out["dy"] = (dz if keep is None else torch.where(keep, dz * mul, 0.0)).to(torch.bfloat16)
    out.update(dx=dz.to(torch.bfloat16), d_gamma=(dhat * n).sum(0), d_beta=dhat.sum(0))
    return out


def _plain_router(st):
    c = st["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["G"]
    sig = c["score"] == "sigmoid"

    def scores(L):
        if sig:
            return 1 / (1 + torch.exp(-L))
        e = torch.exp(L - L.amax(-1, keepdim=True))
        return e / e.sum(-1, keepdim=True)

    # the choice, in 64 bits: scores and biases next to one another
    L = st["logits"]
    chance = scores(L.double())
    if st["bias"] is not None:
        chance = chance + st["bias"].double()
    best, _ = torch.sort(chance.reshape(T, G, E // G), dim=-1, descending=True)
    _, groups = torch.sort(best[..., :c["best"]].sum(-1), dim=-1, descending=True, stable=True)
    rank = torch.empty_like(groups).scatter_(1, groups, torch.arange(G, device="cuda").expand(T, G).contiguous())
    chance = torch.where((rank < c["kg"]).repeat_interleave(E // G, 1), chance, -math.inf)
    _, order = torch.sort(chance, dim=-1, descending=True, stable=True)
    live = torch.ones((T,), dtype=torch.bool, device="cuda") if st["mask"] is None else st["mask"] != 0
    on = live[:, None]
    sel = order[:, :k]
    idx = torch.where(on, sel, -1).to(torch.int32)
    s = scores(L)
    w = torch.gather(s, 1, sel)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    w = torch.where(on, 2.5 * w, 0.0)
    counts = torch.bincount((idx + 1).reshape(-1), minlength=E + 1)[1:].to(torch.int32)
    n = live.sum().to(torch.int32).reshape(1)
    rows = n.clamp(min=1).float()
    p = torch.where(on, s / s.sum(-1, keepdim=True), 0.0)
    mean_prob = p.double().sum(0).float() / rows
    f = counts.float() / (rows * k)
    out = {"idx": idx, "w": w, "counts": counts, "n": n, "mean_prob": mean_prob, "loss": (E * (f * mean_prob).sum()).reshape(1)}
    if c["backward"]:
        slope = 1 / (1 + torch.exp(L)) if sig else torch.ones((), device="cuda")  # 1 - s, or 1
        cost = E * f / rows
        d = st["d_loss"] * p * (cost - (p * cost).sum(-1, keepdim=True)) * slope
        wd = torch.where(on, w * st["d_w"], 0.0)
        if c["renorm"]:
            wd = wd - w / 2.5 * wd.sum(-1, keepdim=True)
        dsel = torch.zeros_like(L).scatter_add_(1, sel, wd)
        d = d + dsel * slope
        if not c["renorm"] and not sig:
            d = d - p * wd.sum(-1, keepdim=True)
        out["d_logits"] = torch.where(on, d, 0.0)
    return out


def _plain_i8(st):
    x = st["x"].float()
    sx = x.abs().amax(-1) / torch.full((), 127.0, device="cuda")  # a quotient, not a product with 1 / 127
    q = torch.where(sx[:, None] > 0, torch.round(x / sx[:, None]).clamp(-127, 127), 0.0)
    y = (q @ st["wq"].float().t()) * sx[:, None] * st["sw"]
    return {"out": y.to(torch.bfloat16), "sx": sx}


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
    if c["op"] == "router_groups":
        ws = _workspace("router", et.et_router_groups_workspace_bytes(c["T"], c["E"], c["k"]))
        score = et.ET_SCORE_SIGMOID if c["score"] == "sigmoid" else et.ET_SCORE_SOFTMAX
        et.et_router_groups(st["logits"], st["idx"], st["w"], score=score, bias=st["bias"], n_groups=c["G"], k_groups=c["kg"],
                            group_best=c["best"], renorm=c["renorm"], scale=2.5, token_mask=st["mask"],
                            expert_counts=st["counts"], n_routed=st["n"], mean_prob=st["mean_prob"], loss=st["loss"], workspace=ws)
        out = {n: st[n] for n in ("idx", "w", "counts", "n", "mean_prob", "loss")}
        if c["backward"]:
            et.et_router_groups_bwd(st["logits"], st["idx"], st["w"], st["counts"], st["n"], st["d_logits"], score=score,
                                    renorm=c["renorm"], scale=2.5, token_mask=st["mask"], d_loss=st["d_loss"], d_topk_w=st["d_w"],
                                    workspace=ws)
            out["d_logits"] = st["d_logits"]
        return out
    if c["op"] == "layer_norm":
        ws = _workspace("norm", et.et_layer_norm_workspace_bytes(c["T"], c["H"]))
        args = dict(gamma=st["gamma"], eps=EPS, p=c["p"], seed=st["seed"], offset=st["offset"], workspace=ws)
        et.et_layer_norm(st["x"], st["y"], st["x_out"], st["x_hat"], beta=st["beta"], **args)
        out = {"x_hat": st["x_hat"]}
        if c["y"]:
            out["x_out"] = st["x_out"]
        if c["backward"]:
            et.et_layer_norm_bwd(st["x"], st["y"], st["dz"], st["dhat"], st["dx"], st["dy"], d_gamma=st["dgamma"],
                                 d_beta=st["dbeta"], **args)
            out.update(dx=st["dx"], d_gamma=st["dgamma"], d_beta=st["dbeta"])
            if c["y"]:
                out["dy"] = st["dy"]
        return out
    if c["op"] == "dropout":
        ws = _workspace("dropout", et.et_dropout_workspace_bytes(c["T"], c["H"]))
        args = dict(p=c["p"], seed=st["seed"], offset=st["offset"], workspace=ws)
        et.et_dropout(st["x"], st["y"], st["out"], **args)
        out = {"out": st["out"]}
        if c["backward"]:
            et.et_dropout(None, st["d_out"], st["dy"], **args)
            out["dy"] = st["dy"]
        return out
    ws = _workspace("i8", et.et_i8_gemm_workspace_bytes(c["M"], c["N"], c["K"]))
    et.et_i8_quantize(st["x"], st["xq"], st["sx"], workspace=ws)
    et.et_i8_gemm(st["xq"], st["sx"], st["wq"], st["sw"], st["out"], workspace=ws)
    return {"out": st["out"], "sx": st["sx"]}


_PLAIN = {"router_groups": _plain_router, "layer_norm": _plain_norm, "dropout": _plain_dropout, "i8_linear": _plain_i8}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------- 64 bits

def _philox(counter, key):
    """Philox4x32-10 of uint64 arrays that hold 32-bit words, on the host."""
    low = np.uint64(0xFFFFFFFF)
    x = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(v) for v in key]
    for _ in range(10):
        left, right = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(right >> np.uint64(32)) ^ x[1] ^ np.uint64(k[0]), right & low, (left >> np.uint64(32)) ^ x[3] ^ np.uint64(k[1]), left & low]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return x


def _factor(case, st):
    """fp64 [T, H]: 0 where an element is dropped, 1 / (1 - p) elsewhere."""
    T, H, t16 = case["T"], case["H"], round(case["p"] * 2 ** 16)
    h8 = -(-H // 8)
    rows, cols = np.divmod(np.arange(T * h8, dtype=np.uint64), np.uint64(h8))
    o = st["offset"]
    words = _philox([cols, rows, np.full_like(rows, o % 2 ** 32), np.full_like(rows, o // 2 ** 32)],
                    [st["seed"] % 2 ** 32, st["seed"] // 2 ** 32 % 2 ** 32])
    kept = np.empty((T * h8, 8), dtype=bool)
    for i in range(8):
        kept[:, i] = (words[i // 2] >> np.uint64(16 * (i % 2))) % np.uint64(65536) >= t16
    return torch.from_numpy(kept.reshape(T, h8 * 8)[:, :H].copy()).cuda().double() / (1 - t16 / 2 ** 16)


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    if c["op"] == "i8_linear":
        x = st["x"].double()
        s = (x.abs().max(-1).values / 127).float().double()  # the stored scale is 32 bits by definition
        r = torch.where(s[:, None] > 0, x / s[:, None], 0.0).float().double()  # and the quotient before it is rounded
        q = torch.clamp(torch.round(r), -127, 127)
        return {"out": torch.einsum("mk,nk->mn", q * s[:, None], st["wq"].double() * st["sw"].double()[:, None]), "sx": s}
    if c["op"] == "dropout":
        f = _factor(c, st)
        res = {"out": f * st["y"].double() + (st["x"].double() if c["x"] else 0.0)}
        if c["backward"]:
            res["dy"] = f * st["d_out"].double()
        return res
    if c["op"] == "layer_norm":
        z = st["x"].double()
        f = _factor(c, st) if c["p"] > 0 else 1.0
        if c["y"]:
            z = z + f * st["y"].double()
        sd = torch.sqrt(z.var(-1, unbiased=False, keepdim=True) + EPS)
        u = (z - z.mean(-1, keepdim=True)) / sd
        gamma = st["gamma"].double()
        res = {"x_hat": torch.addcmul(st["beta"].double(), u, gamma)}
        if c["y"]:
            res["x_out"] = z
        if c["backward"]:
            dhat = st["dhat"].double()
            du = dhat * gamma
            d = (du - du.mean(-1, keepdim=True) - u * (du * u).mean(-1, keepdim=True)) / sd
            if c["y"]:
                d = d + st["dz"].double()
                res["dy"] = f * d
            res.update(dx=d, d_gamma=torch.einsum("th,th->h", dhat, u), d_beta=dhat.sum(0))
        return res
    T, E, k, G = c["T"], c["E"], c["k"], c["G"]
    L = st["logits"].double()
    keep = torch.ones((T,), dtype=torch.bool, device="cuda") if st["mask"] is None else st["mask"].bool()
    Tn = max(1, int(keep.sum()))
    sig = c["score"] == "sigmoid"
    s = torch.sigmoid(L) if sig else torch.softmax(L, -1)
    v = (s if st["bias"] is None else s + st["bias"].double()).unflatten(1, (G, -1))
    rank = torch.argsort(torch.argsort(-v.topk(min(c["best"], E // G), -1).values.sum(-1), dim=-1, stable=True), dim=-1)
    sel = torch.argsort(-torch.where((rank < c["kg"])[..., None], v, -math.inf).flatten(1), dim=-1, stable=True)[:, :k]
    chosen = torch.gather(s, 1, sel)
    wt = 2.5 * (chosen / chosen.sum(-1, keepdim=True) if c["renorm"] else chosen) * keep[:, None]
    f = torch.zeros((T, E), dtype=torch.float64, device="cuda").scatter_(1, sel, 1.0)[keep].sum(0) / (Tn * k)
    p = s / s.sum(-1, keepdim=True) * keep[:, None]
    P = p.sum(0) / Tn
    res = {"idx": None, "w": wt, "counts": None, "n": None, "mean_prob": P, "loss": (E * torch.dot(f, P)).reshape(1)}
    if c["backward"]:
        # through the scores: d s of the weights, d s of the loss, then d L
        dw = 2.5 * st["d_w"].double() * keep[:, None]
        if c["renorm"]:
            S = chosen.sum(-1, keepdim=True)
            dw = (dw - (dw * chosen).sum(-1, keepdim=True) / S) / S
        ds = torch.zeros_like(s).scatter_(1, sel, dw)
        dp = st["d_loss"].double() * E * f / Tn * keep[:, None]
        Z = s.sum(-1, keepdim=True)
        ds += (dp - (dp * s).sum(-1, keepdim=True) / Z) / Z
        res["d_logits"] = ds * s * torch.sigmoid(-L) if sig else s * (ds - (ds * s).sum(-1, keepdim=True))
    return res
