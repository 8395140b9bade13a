"""Cases of the router's and the 4-bit experts' operators: routing by softmax or
sigmoid scores with a balance bias and expert groups, its training step with the
gradient of the logits, the gradient of the weighted combine, the INT4 group
quantiser with its inverse, and products of few rows with INT4 weights.

The sizes are those of the 256-expert layer in workloads/ (hidden 6144, expert
width 256, top-8 of 256) from one token to a 16384-token prefill, and its dense
8192 product.
"""
import math

import numpy as np
import torch

own = False

F = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# route: softmax or sigmoid scores, `groups` of which `keep` stay; router_step: the same with all scores kept for a
# balance loss, and the logits' gradient.  combine_grad: gradients of the weighted sum of each token's k rows.
# quantize: [E, N, K] weights to 4 bits and back.  gemv: T tokens' rows on [E, N, K] 4-bit weights (gated: act(g) * u of N/2).
LISTED = [
    # one token of a serving loop through a sigmoid router with balance bias and groups: latency counts
    dict(name="route_token", kind="route", T=1, E=256, k=8, score="sigmoid", bias=True, groups=8, keep=4, top=2, renorm=True, scale=2.5, dtype="f32"),
    # the router of a prefill
    dict(name="route_prefill", kind="route", T=16384, E=256, k=8, score="sigmoid", bias=True, groups=8, keep=4, top=2, renorm=True, scale=2.5, dtype="f32"),
    # a training step of a softmax router on an odd number of tokens, bf16 logits, weights not renormalised
    dict(name="router_step_softmax", kind="router_step", T=2051, E=256, k=8, score="softmax", bias=False, groups=1, keep=1, top=1, renorm=False, scale=1.0, dtype="bf16"),
    # the training step of the grouped sigmoid router at prefill size
    dict(name="router_step_prefill", kind="router_step", T=16384, E=256, k=8, score="sigmoid", bias=True, groups=8, keep=4, top=2, renorm=True, scale=2.5, dtype="f32"),
    # the combine's gradients of a small training batch
    dict(name="combine_grad_small", kind="combine_grad", T=255, E=256, k=8, H=6144, dtype="bf16"),
    # and of a batch of prefill size: rows in, rows out
    dict(name="combine_grad_prefill", kind="combine_grad", T=16384, E=256, k=8, H=6144, dtype="bf16"),
    # one expert's gate_up weights to 4 bits and back (a fine-tuning step with quantised weights), with zero points
    dict(name="quantize_expert", kind="quantize", E=1, N=512, K=6144, group=64, zeros=True, dtype="f32"),
    # all experts' gate_up weights on the way into a 4-bit layer
    dict(name="quantize_layer", kind="quantize", E=256, N=512, K=6144, group=128, zeros=False, dtype="bf16"),
    # gate_up of one token through its 8 experts: 13 MB of weights, latency counts
    dict(name="gemv_token", kind="gemv", T=1, E=256, k=8, N=512, K=6144, group=128, zeros=False, act="silu", dtype="bf16"),
    # gate_up of a decode batch, 2 rows an expert: the whole 400 MB of weights streams through
    dict(name="gemv_decode", kind="gemv", T=64, E=256, k=8, N=512, K=6144, group=128, zeros=False, act="silu", dtype="bf16"),
    # down projection of a larger decode batch, 8 rows an expert, a short reduction
    dict(name="gemv_down", kind="gemv", T=256, E=256, k=8, N=6144, K=256, group=64, zeros=False, act="", dtype="bf16"),
    # a dense layer on three sequences in fp16, small groups with zero points
    dict(name="gemv_dense", kind="gemv", T=3, E=1, k=1, N=8192, K=8192, group=32, zeros=True, act="", dtype="f16"),
]


def listed():
    return [dict(c) for c in LISTED]


def _cost(c):
    w = work(c)
    return w["flops"] / 2.5e15 + w["bytes"] / 8e12


def draw(rng):
    """One more case: kinds, types and options freely, sizes spread over their logarithm, at most the largest listed cost."""
    most = max(_cost(c) for c in LISTED)

    def log(lo, hi, step=1):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
        return max(lo, min(hi, int(v) // step * step))

    while True:
        kind = rng.choice(["route", "router_step", "combine_grad", "quantize", "gemv", "gemv"])
        if kind in ("route", "router_step"):
            groups = rng.choice([1, 1, 2, 4, 8, 16])
            E = groups * log(2, 512 // groups)
            keep = rng.randint(1, groups)
            c = dict(kind=kind, T=log(1, 16384), E=E, k=rng.randint(1, min(16, E // groups * keep)), score=rng.choice(["softmax", "sigmoid"]),
                     bias=rng.random() < 0.5, groups=groups, keep=keep, top=rng.choice([1, 2]), renorm=rng.random() < 0.5,
                     scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "bf16", "f16"]))
        elif kind == "combine_grad":
            E = log(8, 256)
            c = dict(kind=kind, T=log(1, 16384), E=E, k=rng.randint(1, 8), H=log(64, 8192, 8), dtype=rng.choice(["bf16", "f32"]))
        elif kind == "quantize":
            group = rng.choice([32, 64, 128])
            c = dict(kind=kind, E=log(1, 256), N=log(8, 8192), K=log(group, 8192, group), group=group, zeros=rng.random() < 0.5, dtype=rng.choice(["bf16", "f16", "f32"]))
        else:
            group, E = rng.choice([32, 64, 128]), rng.choice([1, log(2, 256), 256])
            act = rng.choice(["", "silu", "gelu"])
            c = dict(kind=kind, T=log(1, 64 if E == 1 else 256), E=E, k=rng.randint(1, min(8, E)), N=log(16, 8192, 2 if act else 1),
                     K=log(group, 8192, group), group=group, zeros=rng.random() < 0.5, act=act, dtype=rng.choice(["bf16", "f16"]))
            if E * c["N"] * c["K"] > 1 << 30:
                continue
        if _cost(c) <= most:
            return c


def work(c):
    """What one pass has to read, write and compute: each input and output once, weights of the experts that get rows."""
    if c["kind"] in ("route", "router_step"):
        T, E, M = c["T"], c["E"], c["T"] * c["k"]
        eb = 4 if c["dtype"] == "f32" else 2
        b = T * E * eb + 24 * M + 8 * E + (4 * E if c["bias"] else 0)
        if c["kind"] == "route":
            return {"bytes": b, "flops": 8 * T * E}
        # all scores and the logits' gradient out, the weights' and the scores' gradient in
        return {"bytes": b + T * E * (4 + eb) + 4 * M + 4 * E, "flops": 16 * T * E}
    if c["kind"] == "combine_grad":
        n = 2 if c["dtype"] == "bf16" else 4
        T, M, H = c["T"], c["T"] * c["k"], c["H"]
        return {"bytes": (T + 2 * M) * H * n + 12 * M, "flops": 3 * M * H}
    W = c["N"] * c["K"]
    packed = W / 2 + W / c["group"] * (3 if c["zeros"] else 2)
    if c["kind"] == "quantize":
        return {"bytes": int(c["E"] * (W * (4 if c["dtype"] == "f32" else 2) + packed * 2 + W * 2)), "flops": 8 * c["E"] * W}
    M = c["T"] * c["k"]
    cols = c["N"] // 2 if c["act"] else c["N"]
    return {"bytes": int(min(c["E"], M) * packed + c["T"] * (c["K"] if c["act"] else c["k"] * c["K"]) * 2 + M * cols * 2), "flops": 2 * M * W}


def _rows(c, seed):
    """Top-k routing drawn on the host: the token of each row in expert order (stable), the experts' offsets, and each assignment's row."""
    T, E, k = c["T"], c["E"], c["k"]
    r = np.random.default_rng([seed, T, E, k])
    lg = r.standard_normal((T, E), dtype=np.float32)
    ids = np.sort(np.argpartition(-lg, min(k, E) - 1, axis=1)[:, :k], axis=1).reshape(-1)
    order = np.argsort(ids, kind="stable")
    row_of = np.empty(T * k, np.int64)
    row_of[order] = np.arange(T * k)
    return order // k, np.concatenate([[0], np.cumsum(np.bincount(ids, minlength=E))]), row_of


def _encode(x, group, zeros, dtype):
    """float32 [..., K] -> 4-bit codes in bytes [..., K/2], scales and zero points [..., K/group]."""
    v = x.reshape(*x.shape[:-1], -1, group)
    if zeros:
        lo, hi = v.amin(-1).clamp(max=0), v.amax(-1).clamp(min=0)
        s = ((hi - lo) / 15).to(dtype)
    else:
        s = (v.abs().amax(-1) / 7).to(dtype)
    s = torch.where(s == 0, torch.ones_like(s), s)
    f = s.float().unsqueeze(-1)
    z = torch.round(-lo / s.float()).clamp(0, 15).to(torch.uint8) if zeros else None
    shift = z.float().unsqueeze(-1) if zeros else 8.0
    q = (torch.round(v / f) + shift).clamp(0, 15).to(torch.uint8).reshape(x.shape)
    return q[..., 0::2] | (q[..., 1::2] << 4), s, z


def _decode(codes, s, z, group):
    """The values that codes stand for, float32."""
    q = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1, group).float()
    q -= 8.0 if z is None else z.float().unsqueeze(-1)
    q *= s.float().unsqueeze(-1)
    return q.reshape(*codes.shape[:-1], -1)


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(shape, dtype=torch.float32, std=1.0):
        out = torch.empty(shape, dtype=dtype, device=dev)
        flat = out.view(-1, shape[-1])
        step = max(1, (1 << 28) // shape[-1])
        for i in range(0, flat.shape[0], step):
            part = flat[i:i + step]
            part.copy_(torch.randn(part.shape, generator=g, device=dev).mul_(std))
        return out

    s = {"case": c}
    if own:
        import block_scaled_fp4_permute_amd as m
        s["m"] = m
    kind = c["kind"]
    if kind in ("route", "router_step"):
        T, E, k = c["T"], c["E"], c["k"]
        s["logits"] = normal((T, E), F[c["dtype"]])
        s["bias"] = normal((E,), std=0.05) if c["bias"] else None
        if kind == "router_step":
            # the weights' gradient from the combine, and that of a balance loss on the mean scores (one value an expert)
            s["dw"], s["dscores"] = normal((T, k)), normal((E,), std=0.01)
        return s
    if kind == "quantize":
        s["w"] = normal((c["E"], c["N"], c["K"]), F[c["dtype"]], 0.02)
        return s
    src, off, row_of = _rows(c, seed)
    M = c["T"] * c["k"]
    s["M"] = M
    if kind == "combine_grad":
        dt = F[c["dtype"]]
        s["dout"], s["y"] = normal((c["T"], c["H"]), dt), normal((M, c["H"]), dt)
        s["perm"] = torch.from_numpy(row_of.astype(np.int32)).to(dev)
        w = torch.rand((c["T"], c["k"]), generator=g, device=dev) + 0.05
        s["w"] = w / w.sum(1, keepdim=True)
        return s
    E, N, K, group = c["E"], c["N"], c["K"], c["group"]
    dt = F[c["dtype"]]
    s["offsets"], s["host_offsets"] = torch.from_numpy(off.astype(np.int32)).to(dev), off.tolist()
    # rows of gate_up are gathered by token; the others are in expert order
    gathered = bool(c["act"]) and E > 1
    s["rows"] = torch.from_numpy(src.astype(np.int32)).to(dev) if gathered else None
    s["token"] = torch.from_numpy(src).to(dev) if gathered else None
    s["x"] = normal((c["T"] if gathered else M, K), dt)
    codes = torch.empty((E, N, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((E, N, K // group), dtype=dt, device=dev)
    zeros = torch.empty((E, N, K // group), dtype=torch.uint8, device=dev) if c["zeros"] else None
    step = max(1, (1 << 26) // (N * K))
    for e in range(0, E, step):
        q, sc, z = _encode(normal((min(step, E - e), N, K), std=0.02), group, c["zeros"], dt)
        codes[e:e + step], scales[e:e + step] = q, sc
        if zeros is not None:
            zeros[e:e + step] = z
    s["b"] = (codes, scales, zeros)
    # the same routing as a padded table of rows per expert that has any (-1: no row)
    n = np.diff(off)
    active = np.flatnonzero(n)
    table = np.arange(n.max())[None, :]
    table = np.where(table < n[active][:, None], off[active][:, None] + table, -1)
    s["active"], s["table"] = torch.from_numpy(active).to(dev), torch.from_numpy(table).to(dev)
    if own:
        s["b4"] = m.INT4Tensor(codes, scales, zeros, group)
    return s


# ------------------------------------------------------------------ plain forms
def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    t = torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t)


def _plain_route(s):
    """Scores and choice in float64: the order of near-equal keys decides whole numbers."""
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    l = s["logits"].double()
    if c["score"] == "softmax":
        p = torch.exp(l - l.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-l))
    key = p + s["bias"].double() if c["bias"] else p
    order = key if c["bias"] else l
    if G > 1:
        best = key.view(T, G, E // G).sort(dim=2, descending=True).values[..., :c["top"]].sum(2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        open_ = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        order = torch.where(open_.repeat_interleave(E // G, 1), order, -math.inf)
    ids = order.sort(dim=1, descending=True, stable=True).indices[:, :k]
    u = p.gather(1, ids)
    if c["renorm"]:
        u = u / u.sum(1, keepdim=True)
    w = (u * c["scale"]).float()
    flat = ids.reshape(-1)
    counts = torch.zeros(E, dtype=torch.int64, device=l.device).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    by_expert = flat.sort(stable=True).indices
    row_of = torch.empty_like(flat)
    row_of[by_expert] = torch.arange(T * k, device=l.device)
    i32 = torch.int32
    out = {"ids": ids.to(i32), "w": w, "counts": counts.to(i32), "offsets": offsets.to(i32), "src": (by_expert // k).to(i32),
           "row_of": row_of.to(i32), "row_w": w.reshape(-1)[by_expert]}
    return out, p, u


def _plain_router_step(s):
    c = s["case"]
    out, p, u = _plain_route(s)
    ids, g = out["ids"].long(), s["dw"].double()
    part = u * (g - (g * u).sum(1, keepdim=True)) if c["renorm"] else u * g
    chosen = torch.zeros_like(p).scatter_(1, ids, part * c["scale"])
    q = s["dscores"].double()
    if c["score"] == "softmax":
        d = chosen - p * chosen.sum(1, keepdim=True) + p * (q - (p * q).sum(1, keepdim=True))
    else:
        d = (1 - p) * (chosen + p * q)
    out["scores"], out["dlogits"] = p.float(), d.to(s["logits"].dtype)
    return out


def _plain_combine_grad(s):
    dout, rows = s["dout"].float(), s["perm"].long().view(s["w"].shape)
    dy = torch.empty_like(s["y"])
    dy[rows.reshape(-1)] = (dout.unsqueeze(1) * s["w"].unsqueeze(-1)).to(dy.dtype).view(-1, dy.shape[1])
    return dy, (dout.unsqueeze(1) * s["y"][rows].float()).sum(-1)


def _kept(c):
    """The type of scales and values: the weights' own, bf16 for float32 ones."""
    return torch.bfloat16 if c["dtype"] == "f32" else F[c["dtype"]]


def _plain_quantize(s):
    c = s["case"]
    dt = _kept(c)
    codes, scales, zeros = _encode(s["w"].float(), c["group"], c["zeros"], dt)
    return _decode(codes, scales, zeros, c["group"]).to(dt), scales, zeros


def _plain_gemv(s):
    c, t = s["case"], s["table"]
    codes, scales, zeros = s["b"]
    a = s["active"]
    b = _decode(codes[a], scales[a], None if zeros is None else zeros[a], c["group"])
    rows = s["x"] if s["token"] is None else s["x"][s["token"]]
    x = rows[t.clamp(min=0)].float() * (t >= 0).unsqueeze(-1)
    y = torch.bmm(x, b.transpose(1, 2))
    if c["act"]:
        I = c["N"] // 2
        y = _act(y[..., :I], c["act"]) * y[..., I:]
    out = torch.empty((s["M"], y.shape[-1]), dtype=rows.dtype, device=y.device)
    out[t[t >= 0]] = y[t >= 0].to(rows.dtype)
    return out


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    kind = c["kind"]
    if not own:
        if kind == "route":
            return _plain_route(s)[0]
        return {"router_step": _plain_router_step, "combine_grad": _plain_combine_grad, "quantize": _plain_quantize, "gemv": _plain_gemv}[kind](s)
    m = s["m"]
    if kind in ("route", "router_step"):
        how = dict(score=m.SCORE_SIGMOID if c["score"] == "sigmoid" else m.SCORE_SOFTMAX, renormalize=c["renorm"], scale=c["scale"])
        choice = dict(bias=s["bias"], n_group=c["groups"], topk_group=c["keep"], group_top=min(c["top"], c["E"] // c["groups"]))
        if kind == "route":
            r, more = m.moe_route_scored(s["logits"], c["k"], **how, **choice), {}
        else:
            r, scores = m.moe_route_scored(s["logits"], c["k"], **how, **choice, save_scores=True)
            more = {"scores": scores, "dlogits": m.moe_route_scored_backward(s["dw"], s["logits"], r.topk_ids, **how, d_scores=s["dscores"])}
        return {"ids": r.topk_ids, "w": r.topk_w, "counts": r.counts, "offsets": r.offsets, "src": r.perm_src_token, "row_of": r.perm_of_assignment,
                "row_w": r.perm_weight, **more}
    if kind == "combine_grad":
        return m.moe_unpermute_combine_backward(s["dout"], s["y"], s["perm"], s["w"])
    if kind == "quantize":
        q = m.int4_quantize(s["w"], group=c["group"], zeros=c["zeros"])
        return m.int4_dequantize(q), q.scales, q.zeros
    if c["act"]:
        return m.int4_grouped_gemv(s["x"], s["b4"], s["offsets"], m_total=s["M"], a_rows=s["rows"], gated=True,
                                   activation=m.ACT_SILU if c["act"] == "silu" else m.ACT_GELU)
    return m.int4_grouped_gemv(s["x"], s["b4"], s["offsets"], m_total=s["M"], a_rows=s["rows"])


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    """Token by token, expert by expert or group by group in float64."""
    c, s = case, prepare(case, seed)
    D, kind = torch.float64, case["kind"]
    if kind in ("route", "router_step"):
        return _exact_route(c, s)
    if kind == "combine_grad":
        if c["T"] * c["k"] * c["H"] > 1 << 31:
            return None
        dy = torch.empty(s["y"].shape, dtype=D, device=s["y"].device)
        dw = torch.empty(s["w"].shape, dtype=D, device=s["y"].device)
        at = s["perm"].long().view(c["T"], c["k"])
        for j in range(c["k"]):
            dy[at[:, j]] = s["w"][:, j:j + 1].to(D) * s["dout"].to(D)
            dw[:, j] = torch.einsum("th,th->t", s["dout"].to(D), s["y"][at[:, j]].to(D))
        return dy, dw
    if kind == "quantize":
        x = s["w"]
        if x.numel() > 1 << 31:
            return None
        v = x.to(D).unflatten(-1, (-1, c["group"]))
        dt = _kept(c)
        if c["zeros"]:
            lo, hi = v.min(-1).values.clamp(max=0), v.max(-1).values.clamp(min=0)
            # scale, quotients and zero points are decided in float32, the scale then in the type that holds it
            sc = ((hi.float() - lo.float()) / 15).to(dt).to(D)
        else:
            sc = (v.abs().max(-1).values.float() / 7).to(dt).to(D)
        sc[sc == 0] = 1
        k = torch.round((v / sc[..., None]).float()).to(D)
        if not c["zeros"]:
            return (k.clamp(-8, 7) * sc[..., None]).flatten(-2), sc, None
        z = torch.round((-lo / sc).float()).to(D).clamp(0, 15)
        return (((k + z[..., None]).clamp(0, 15) - z[..., None]) * sc[..., None]).flatten(-2), sc, z.to(torch.uint8)
    codes, scales, zeros = s["b"]
    cols = c["N"] // 2 if c["act"] else c["N"]
    out = torch.empty((s["M"], cols), dtype=D, device=codes.device)
    for e in range(c["E"]):
        lo, hi = s["host_offsets"][e:e + 2]
        if lo == hi:
            continue
        w = torch.empty((c["N"], c["K"]), dtype=D, device=codes.device)
        w[:, 0::2], w[:, 1::2] = (codes[e] % 16).to(D), (codes[e] // 16).to(D)
        w -= 8 if zeros is None else zeros[e].to(D).repeat_interleave(c["group"], 1)
        w *= scales[e].to(D).repeat_interleave(c["group"], 1)
        x = s["x"][lo:hi] if s["token"] is None else s["x"][s["token"][lo:hi]]
        y = x.to(D) @ w.T
        if c["act"]:
            g, u = y[:, :cols], y[:, cols:]
            if c["act"] == "gelu":
                z = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
                y = g * u / (1 + torch.exp(-2 * z))
            else:
                y = g * u / (1 + torch.exp(-g))
        out[lo:hi] = y
    return out


def _exact_route(c, s):
    """Expert after expert: the best that is left, k times."""
    D = torch.float64
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    l = s["logits"].to(D)
    p = torch.softmax(l, 1) if c["score"] == "softmax" else torch.sigmoid(l)
    key = p + s["bias"].to(D) if c["bias"] else p
    order = (key if c["bias"] else l).clone()
    t = torch.arange(T, device=l.device)
    if G > 1:
        left, value = key.clone().view(T, G, -1), 0
        for _ in range(min(c["top"], E // G)):
            top = left.max(2)
            value = value + top.values
            left.scatter_(2, top.indices[..., None], -math.inf)
        out_of = torch.ones((T, G), dtype=torch.bool, device=l.device)
        for _ in range(c["keep"]):
            b = (value == value.amax(1, keepdim=True)).int().argmax(1)
            out_of[t, b], value[t, b] = False, -math.inf
        order[out_of.repeat_interleave(E // G, 1)] = -math.inf
    ids = torch.empty((T, k), dtype=torch.int64, device=l.device)
    for j in range(k):
        ids[:, j] = (order == order.amax(1, keepdim=True)).int().argmax(1)
        order[t, ids[:, j]] = -math.inf
    u = p[t[:, None], ids]
    share = u / u.sum(1, keepdim=True) if c["renorm"] else u
    w = share * c["scale"]
    counts = torch.bincount(ids.view(-1), minlength=E)
    rows = torch.argsort(ids.view(-1) * (T * k) + torch.arange(T * k, device=l.device))
    row_of = torch.argsort(rows)
    i32 = torch.int32
    out = {"ids": ids.to(i32), "w": w, "counts": counts.to(i32), "offsets": torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(i32),
           "src": (rows // k).to(i32), "row_of": row_of.to(i32), "row_w": w.view(-1)[rows]}
    if c["kind"] == "route":
        return out
    # gradient of sum(w dw) + sum(scores dscores) by the chain rule over the scores
    g = s["dw"].to(D) * c["scale"]
    ds = s["dscores"].to(D).expand(T, E).clone()
    if c["renorm"]:
        total = u.sum(1, keepdim=True)
        ds.scatter_add_(1, ids, g / total - (g * u).sum(1, keepdim=True) / total ** 2)
    else:
        ds.scatter_add_(1, ids, g)
    if c["score"] == "softmax":
        d = p * ds - p * (p * ds).sum(1, keepdim=True)
    else:
        d = ds * p * (1 - p)
    out["scores"], out["dlogits"] = p, d
    return out
