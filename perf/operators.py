"""Cases of the experts' feed-forward operators in 16-bit types and in 8-bit
integers: the gated block with its gradients, the grouped product after it with
its gradients, the per-row INT8 quantiser and the INT8 grouped product.

The sizes are those of the 256-expert layer in workloads/ (hidden 6144, expert
width 256, top-8 of 256) from one token to a 16384-token prefill, of its dense
8192 product, and of a generic dense block (hidden 2048, width 8192).
"""
import math

import numpy as np
import torch

own = False

F = {"bf16": torch.bfloat16, "f16": torch.float16}

# H: reduction of the gated block / output columns of the product after it; I:
# expert width.  gated: h = act(x Wg^T) * (x Wu^T), rows gathered by token.
# product: y = a b^T on rows in expert order.  "train" adds the gradients.
LISTED = [
    # one token through its 8 experts: 50 MB of weights, latency counts
    dict(name="gated_token", kind="gated", T=1, H=6144, I=256, E=256, k=8, zipf=False, dtype="bf16", act="silu", train=False),
    # a decode batch, 8 rows an expert: the whole 1.6 GB of weights streams through
    dict(name="gated_decode", kind="gated", T=256, H=6144, I=256, E=256, k=8, zipf=False, dtype="bf16", act="silu", train=False),
    # fine-tuning on a small batch with skewed routing: experts of a few rows up to hundreds
    dict(name="gated_train_skewed", kind="gated", T=2048, H=6144, I=256, E=256, k=8, zipf=True, dtype="bf16", act="silu", train=True),
    # a training step's gated block at prefill size: 512 rows an expert, both gradients
    dict(name="gated_train_prefill", kind="gated", T=16384, H=6144, I=256, E=256, k=8, zipf=False, dtype="bf16", act="silu", train=True),
    # a dense (shared-expert) block with GELU in fp16 and an odd number of tokens
    dict(name="gated_train_dense", kind="gated", T=4099, H=2048, I=8192, E=1, k=1, zipf=False, dtype="f16", act="gelu", train=True),
    # the down projection of the decode batch
    dict(name="product_decode", kind="product", T=256, H=6144, I=256, E=256, k=8, zipf=False, dtype="bf16", act="", train=False),
    # the down projection of the skewed training batch with both gradients
    dict(name="product_train_skewed", kind="product", T=2048, H=6144, I=256, E=256, k=8, zipf=True, dtype="bf16", act="", train=True),
    # the activations of a few tokens on the way into an INT8 layer
    dict(name="quantize_tokens", kind="quantize", T=37, H=6144, I=0, E=1, k=1, zipf=False, dtype="bf16", act="", train=False),
    # the activations of a prefill
    dict(name="quantize_prefill", kind="quantize", T=16384, H=6144, I=0, E=1, k=1, zipf=False, dtype="bf16", act="", train=False),
    # INT8 gate_up with the SwiGLU in its epilogue, skewed decode batch
    dict(name="int8_gated_skewed", kind="int8_gated", T=2048, H=6144, I=256, E=256, k=8, zipf=True, dtype="bf16", act="silu", train=False),
    # INT8 down projection of the decode batch
    dict(name="int8_decode", kind="int8", T=256, H=6144, I=256, E=256, k=8, zipf=False, dtype="bf16", act="", train=False),
    # one large dense INT8 product
    dict(name="int8_dense", kind="int8", T=8192, H=8192, I=8192, E=1, k=1, zipf=False, dtype="bf16", act="", train=False),
]


def listed():
    return [dict(c) for c in LISTED]


def _cost(c):
    w = work(c)
    return w["flops"] / 2.5e15 + w["bytes"] / 8e12


def draw(rng):
    """One more case: kind, type and activation freely, sizes spread over their logarithm, at most the largest listed cost."""
    most = max(_cost(c) for c in LISTED)

    def log(lo, hi, step):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
        return max(lo, min(hi, int(v) // step * step))

    while True:
        kind = rng.choice(["gated", "gated", "product", "quantize", "int8_gated", "int8"])
        step = 16 if kind.startswith("int8") else 8
        E = rng.choice([1, log(2, 256, 1), 256]) if kind != "quantize" else 1
        big = 8192 if E == 1 else 1024
        c = dict(kind=kind, T=log(1, 16384, 1), H=log(64, 8192, step), I=log(32, big, step) if kind != "quantize" else 0, E=E,
                 k=rng.randint(1, min(8, E)), zipf=rng.random() < 0.5 and E > 1, dtype=rng.choice(["bf16", "f16"]),
                 act=rng.choice(["silu", "gelu"]) if kind == "gated" else "silu" if kind == "int8_gated" else "",
                 train=rng.random() < 0.5 and kind in ("gated", "product"))
        if kind.startswith("int8"):
            c["dtype"] = rng.choice(["bf16", "f32"]) if kind == "int8" else "bf16"
        if kind == "quantize":
            c["dtype"] = rng.choice(["bf16", "f32"])
        if _cost(c) <= most:
            return c


def work(c):
    """What one pass has to read, write and multiply: weights of the experts that get rows, each activation row once."""
    T, H, I, M = c["T"], c["H"], c["I"], c["T"] * c["k"]
    Ea = min(c["E"], M)
    if c["kind"] == "quantize":
        return {"bytes": T * (H * (4 if c["dtype"] == "f32" else 2) + H + 4), "flops": 3 * T * H}
    if c["kind"] == "gated":
        W, x, h = Ea * 2 * I * H * 2, T * H * 2, M * I * 2
        fl = 2 * M * 2 * I * H
        if not c["train"]:
            return {"bytes": W + x + h, "flops": fl}
        # and dh in, dx rows and dW out
        return {"bytes": W + x + 2 * h + M * H * 2 + c["E"] * 2 * I * H * 2, "flops": 3 * fl}
    if c["kind"] == "product":
        W, a, y = Ea * I * H * 2, M * I * 2, M * H * 2
        fl = 2 * M * I * H
        if not c["train"]:
            return {"bytes": W + a + y, "flops": fl}
        # and dy in, da and dW out
        return {"bytes": W + 2 * a + 2 * y + c["E"] * I * H * 2, "flops": 3 * fl}
    if c["kind"] == "int8_gated":
        return {"bytes": Ea * 2 * I * (H + 4) + T * (H + 4) + M * I * 2, "flops": 2 * M * 2 * I * H}
    return {"bytes": Ea * H * (I + 4) + M * (I + 4) + M * H * (4 if c["dtype"] == "f32" else 2), "flops": 2 * M * I * H}


def _routing(c, seed):
    """Top-k routing drawn on the host: rows in expert order (stable), the token of each, and the experts' offsets."""
    T, E, k = c["T"], c["E"], c["k"]
    if E == 1:
        return np.zeros(T, np.int64), np.array([0, T], np.int64)
    r = np.random.default_rng([seed, T, E, k])
    lg = r.standard_normal((T, E), dtype=np.float32)
    if c["zipf"]:
        lg -= (0.55 * 1.1) * np.log(np.maximum(r.permutation(E) + 1, 32 if E >= 64 else 1)).astype(np.float32)
    ids = np.sort(np.argpartition(-lg, k - 1, axis=1)[:, :k], axis=1).reshape(-1)
    order = np.argsort(ids, kind="stable")
    return order // k, np.concatenate([[0], np.cumsum(np.bincount(ids, minlength=E))])


def _row_quantized(x):
    """Codes and scales of a symmetric quantiser along the last axis."""
    s = x.abs().amax(-1, keepdim=True) / 127
    return torch.round(x / s).to(torch.int8), s[..., 0].contiguous()


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(shape, dtype, std=1.0):
        out = torch.empty(shape, dtype=dtype, device=dev)
        flat = out.view(-1, shape[-1])
        step = max(1, (1 << 28) // shape[-1])
        for i in range(0, flat.shape[0], step):
            part = flat[i:i + step]
            part.copy_(torch.randn(part.shape, generator=g, device=dev).mul_(std))
        return out

    T, H, I, E, k = (c[n] for n in ("T", "H", "I", "E", "k"))
    s = {"case": c, "M": T * k}
    if own:
        import block_scaled_fp4_permute_amd as m
        s["m"] = m
    if c["kind"] == "quantize":
        # activations with a few large channels, as after a norm
        x = normal((T, H), torch.float32)
        x[:, torch.randperm(H, generator=g, device=dev)[:max(1, H // 128)]] *= 20
        s["x"] = x.to(torch.float32 if c["dtype"] == "f32" else torch.bfloat16)
        return s
    src, off = _routing(c, seed)
    s["offsets"] = torch.from_numpy(off.astype(np.int32)).to(dev)
    s["host_offsets"] = off.tolist()
    gathered = c["kind"] in ("gated", "int8_gated") and E > 1
    s["rows"] = torch.from_numpy(src.astype(np.int32)).to(dev) if gathered else None
    # the same routing as a padded table of rows per expert that has any (-1: no row)
    n = np.diff(off)
    active = np.flatnonzero(n)
    table = np.arange(n.max())[None, :]
    table = np.where(table < n[active][:, None], off[active][:, None] + table, -1)
    s["active"], s["table"] = torch.from_numpy(active).to(dev), torch.from_numpy(table).to(dev)
    s["token"] = torch.from_numpy(src).to(dev) if gathered else None
    dt = F.get(c["dtype"])
    if c["kind"] == "gated":
        s["x"], s["w"] = normal((T, H), dt), normal((E, 2 * I, H), dt, 0.02)
        if c["train"]:
            s["dh"] = normal((T * k, I), dt)
    elif c["kind"] == "product":
        s["a"], s["b"] = normal((T * k, I), dt), normal((E, H, I), dt, 0.02)
        if c["train"]:
            s["dy"] = normal((T * k, H), dt)
    else:
        N, K, rows = (2 * I, H, T) if c["kind"] == "int8_gated" else (H, I, T * k)
        s["a"] = _row_quantized(normal((rows, K), torch.float32))
        b = torch.empty((E, N, K), dtype=torch.int8, device=dev)
        bs = torch.empty((E, N), dtype=torch.float32, device=dev)
        for e0 in range(0, E, 32):
            part = normal((min(32, E - e0), N, K), torch.float32, 0.02)
            b[e0:e0 + 32], bs[e0:e0 + 32] = _row_quantized(part)
        s["b"] = (b, bs)
    if own and c["kind"].startswith("int8"):
        s["a8"], s["b8"] = m.INT8Tensor(*s["a"]), m.INT8Tensor(*s["b"])
    return s


# ------------------------------------------------------------------ plain forms
def _gather(s, rows):
    """Rows [M, n] -> float32 [active experts, most rows, n], zero where there is no row."""
    t = s["table"]
    return rows[t.clamp(min=0)].float() * (t >= 0).unsqueeze(-1)


def _scatter(s, padded, dtype):
    t = s["table"]
    out = torch.empty((s["M"], padded.shape[-1]), dtype=dtype, device=padded.device)
    out[t[t >= 0]] = padded[t >= 0].to(dtype)
    return out


def _act(g, act):
    """The activation and its derivative."""
    if act == "silu":
        sg = 1 / (1 + torch.exp(-g))
        return g * sg, sg * (1 + g * (1 - sg))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _full(s, part, E, dtype):
    out = torch.zeros((E,) + part.shape[1:], dtype=dtype, device=part.device)
    out[s["active"]] = part.to(dtype)
    return out


def _plain_gated(s):
    c, x, w = s["case"], s["x"], s["w"]
    I = c["I"]
    xp = _gather(s, x if s["token"] is None else x[s["token"]])
    wa = w[s["active"]].float()
    y = torch.bmm(xp, wa.transpose(1, 2))
    g, u = y[..., :I], y[..., I:]
    a, da = _act(g, c["act"])
    h = _scatter(s, a * u, x.dtype)
    if not c["train"]:
        return h
    dh = _gather(s, s["dh"])
    dgu = torch.cat([dh * u * da, dh * a], -1)
    dx = _scatter(s, torch.bmm(dgu, wa), x.dtype)
    dw = _full(s, torch.bmm(dgu.transpose(1, 2), xp), c["E"], w.dtype)
    return h, dx, dw


def _plain_product(s):
    c, a, b = s["case"], s["a"], s["b"]
    ap, ba = _gather(s, a), b[s["active"]].float()
    y = _scatter(s, torch.bmm(ap, ba.transpose(1, 2)), a.dtype)
    if not c["train"]:
        return y
    dy = _gather(s, s["dy"])
    da = _scatter(s, torch.bmm(dy, ba), a.dtype)
    db = _full(s, torch.bmm(dy.transpose(1, 2), ap), c["E"], b.dtype)
    return y, da, db


def _plain_quantize(s):
    x = s["x"].float()
    top = x.abs().amax(-1)
    scale = torch.where(top > 0, top / 127, torch.ones_like(top))
    return torch.round(x / scale[:, None]).clamp(-127, 127).to(torch.int8), scale


def _plain_int8(s):
    c = s["case"]
    (a, sa), (b, sb) = s["a"], s["b"]
    if s["token"] is not None:
        a, sa = a[s["token"]], sa[s["token"]]
    acc = torch.bmm(_gather(s, a), b[s["active"]].float().transpose(1, 2))
    y = acc * _gather(s, sa[:, None]) * sb[s["active"]][:, None, :]
    if c["kind"] == "int8_gated":
        g, u = y[..., :c["I"]], y[..., c["I"]:]
        y = _act(g, "silu")[0] * u
    return _scatter(s, y, torch.float32 if c["dtype"] == "f32" else torch.bfloat16)


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    if not own:
        return {"gated": _plain_gated, "product": _plain_product, "quantize": _plain_quantize}.get(c["kind"], _plain_int8)(s)
    m = s["m"]
    if c["kind"] == "gated":
        act = m.ACT_SILU if c["act"] == "silu" else m.ACT_GELU
        if not c["train"]:
            return m.moe_gated_ffn(s["x"], s["w"], s["offsets"], m_total=s["M"], a_rows=s["rows"], activation=act)
        h, gu = m.moe_gated_ffn(s["x"], s["w"], s["offsets"], m_total=s["M"], a_rows=s["rows"], activation=act, save_gu=True)
        dx, dw = m.moe_gated_ffn_backward(s["dh"], gu, s["x"], s["w"], s["offsets"], a_rows=s["rows"], activation=act)
        return h, dx, dw
    if c["kind"] == "product":
        y = m.moe_grouped_gemm(s["a"], s["b"], s["offsets"], m_total=s["M"])
        if not c["train"]:
            return y
        da, db = m.moe_grouped_gemm_backward(s["dy"], s["a"], s["b"], s["offsets"])
        return y, da, db
    if c["kind"] == "quantize":
        q = m.int8_quantize(s["x"])
        return q.codes, q.scales
    epi = m.EPI_SWIGLU_BF16 if c["kind"] == "int8_gated" else m.EPI_F32 if c["dtype"] == "f32" else m.EPI_BF16
    return m.int8_grouped_gemm(s["a8"], s["b8"], s["offsets"], m_total=s["M"], a_rows=s["rows"], epilogue=epi)


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    """Expert by expert in float64."""
    c, s = case, prepare(case, seed)
    D = torch.float64
    if c["kind"] == "quantize":
        x = s["x"].to(D)
        top = x.abs().amax(1)
        scale = torch.where(top > 0, top / 127, torch.ones_like(top))
        # the quotient that decides is the float32 one
        q = (x / scale.float().to(D)[:, None]).float()
        return torch.round(q).clamp(-127, 127).to(torch.int8), scale
    off, M, E, H, I = s["host_offsets"], s["M"], c["E"], c["H"], c["I"]
    dev = s["offsets"].device
    train = c["train"]

    def act64(g):
        if c["act"] == "gelu":
            r = math.sqrt(2 / math.pi)
            z = r * (g + 0.044715 * g ** 3)
            th = 1 - 2 / (torch.exp(2 * z) + 1)
            return g * (1 + th) / 2, (1 + th) / 2 + g * (1 - th) * (1 + th) / 2 * r * (1 + 0.134145 * g ** 2)
        e = torch.exp(-g)
        return g / (1 + e), 1 / (1 + e) + g * e / (1 + e) ** 2

    width = I if c["kind"] in ("gated", "int8_gated") else H
    first = torch.empty((M, width), dtype=D, device=dev)
    if train:
        rows_grad = torch.empty((M, H if c["kind"] == "gated" else I), dtype=D, device=dev)
        weight_grad = torch.zeros(s["w" if c["kind"] == "gated" else "b"].shape, dtype=D, device=dev)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        at = slice(lo, hi) if s["token"] is None else s["token"][lo:hi]
        if c["kind"] == "gated":
            x, w = s["x"][at].to(D), s["w"][e].to(D)
            g, u = x @ w[:I].T, x @ w[I:].T
            a, slope = act64(g)
            first[lo:hi] = a * u
            if train:
                dh = s["dh"][lo:hi].to(D)
                dg, du = dh * u * slope, dh * a
                rows_grad[lo:hi] = dg @ w[:I] + du @ w[I:]
                weight_grad[e, :I], weight_grad[e, I:] = dg.T @ x, du.T @ x
        elif c["kind"] == "product":
            a, b = s["a"][lo:hi].to(D), s["b"][e].to(D)
            first[lo:hi] = a @ b.T
            if train:
                dy = s["dy"][lo:hi].to(D)
                rows_grad[lo:hi], weight_grad[e] = dy @ b, dy.T @ a
        else:
            a = s["a"][0][at].to(D) * s["a"][1][at].to(D)[:, None]
            b = s["b"][0][e].to(D) * s["b"][1][e].to(D)[:, None]
            y = a @ b.T
            if c["kind"] == "int8_gated":
                y = act64(y[:, :I])[0] * y[:, I:]
            first[lo:hi] = y
    return (first, rows_grad, weight_grad) if train else first
