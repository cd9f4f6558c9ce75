"""The cases of the INT8 operators: the norm that hands rows on in 8 bits, rows
and weights to 8-bit integers with a scale per row, the grouped product of such
rows and weights over the batching's group list, and the experts' SwiGLU network
with such weights.

Each case runs in two forms on the same inputs: a plain form (elementary torch
operations in 32 bits, a row's mean of squares in 64, rounded once at the end)
and the package's own entry points (`own` true). exact() gives the same outputs
from the definitions in 64 bits.

Definitions (T: the type of x):
  int8    a = max(max |v|, 2^-96) over a row, s = a / 127, q = round(v (127 / a)),
          to nearest even; s and 127 / a are each rounded to fp32
  norm    h = x + residual, rounded to T; r = 1 / sqrt(mean(h^2) + eps), rounded
          to fp32 once; y = (h r) w; the residual's successor is h, and y goes
          out in T, as int8 rows, or as e4m3 with a scale per 128 values (the
          smallest power of two s with max(amax, 2^-96) <= 448 s)
  matmul  y[r, n] = (sum_k x[r, k] w[e, n, k]) t[e, n] s[r], e the expert of row
          r; rows are int8 with scales s, or of 16 bits without
  ffn     h = silu(x W1^T) * (x W3^T), rounded to bf16, y = h W2^T, each product
          as in matmul
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -96
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "i8": torch.int8}
ELEM = {"bf16": 2, "f16": 2, "f32": 4, "i8": 1}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the rows of one decode step before the experts, handed on as INT8: launch latency
        dict(name="norm decode step", op="norm", rows=64, k=7168, dtype="bf16", residual=True, out="int8", y=False),
        # odd sizes, both outputs, no residual (the first norm of a network)
        dict(name="norm odd sizes", op="norm", rows=1003, k=1000, dtype="f16", residual=False, out="e4m3", y=True),
        # a prefill batch before a routed layer: 16 bits for the router, 8 for the experts
        dict(name="norm prefill", op="norm", rows=16384, k=7168, dtype="bf16", residual=True, out="e4m3", y=True),
        # the rows of a batched decode step (64 sessions x 9 slots) to INT8
        dict(name="quantize decode rows", op="quantize", rows=576, k=7168, dtype="bf16"),
        # 32 experts' matrices to INT8 with a scale per channel, as a loader makes them
        dict(name="quantize weights", op="quantize", rows=65536, k=4096, dtype="bf16"),
        # one token through one projection, as in the step of a single user: the smallest product
        dict(name="matmul one token", op="matmul", rows=1, experts=1, k=4096, n=2048, x="i8", out="bf16", skew=0.0),
        # odd sizes: ragged groups, a row length and a width that no tile divides, fp32 out
        dict(name="matmul odd sizes", op="matmul", rows=1003, experts=12, k=1000, n=1100, x="f16", out="f32", skew=0.5),
        # a batched decode step: 64 sessions x 9 slots over 64 experts, Zipf; weights from HBM
        dict(name="matmul decode batch", op="matmul", rows=576, experts=64, k=7168, n=4096, x="i8", out="bf16",
             skew=1.1),
        # a shared (dense) expert's projection over a prefill batch: bound by the tensor cores
        dict(name="matmul dense prefill", op="matmul", rows=16384, experts=1, k=7168, n=7168, x="i8", out="bf16",
             skew=0.0),
        # odd sizes through the whole expert network: ragged groups, tails in both products
        dict(name="ffn odd sizes", op="ffn", rows=515, experts=6, hidden=1080, inter=712, x="bf16", skew=0.8),
        # the experts of a batched decode step, rows as the batching's INT8 mode leaves them
        dict(name="ffn decode batch", op="ffn", rows=576, experts=64, hidden=7168, inter=1024, x="i8", skew=1.1),
        # the experts over the permuted rows of 4096 tokens x 8: the largest
        dict(name="ffn top-k rows", op="ffn", rows=32768, experts=64, hidden=4096, inter=2048, x="i8", skew=0.3),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["norm", "norm", "quantize", "matmul", "matmul", "ffn", "ffn"])
        if op == "norm":
            out = rng.choice(["int8", "e4m3", "none"])
            c = dict(op=op, rows=_log_int(rng, 1, 32768), k=_log_int(rng, 64, 8192),
                     dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), residual=rng.random() < 0.7, out=out,
                     y=out == "none" or rng.random() < 0.5)
        elif op == "quantize":
            c = dict(op=op, rows=_log_int(rng, 1, 65536), k=_log_int(rng, 64, 8192),
                     dtype=rng.choice(["bf16", "f16", "f32"]))
        elif op == "matmul":
            c = dict(op=op, rows=_log_int(rng, 1, 32768), experts=_log_int(rng, 1, 128), k=_log_int(rng, 64, 7168),
                     n=_log_int(rng, 64, 7168), x=rng.choice(["i8", "i8", "bf16", "f16"]),
                     out=rng.choice(["bf16", "f16", "f32"]), skew=rng.choice([0.0, 0.5, 1.1]))
        else:
            c = dict(op=op, rows=_log_int(rng, 1, 32768), experts=_log_int(rng, 1, 64),
                     hidden=_log_int(rng, 64, 7168), inter=_log_int(rng, 64, 2048),
                     x=rng.choice(["i8", "i8", "bf16", "f16"]), skew=rng.choice([0.0, 0.5, 1.1]))
        if _fits(c):
            return c


def _fits(c):
    """No drawn case costs more than the largest listed one, in work or in memory."""
    w = work(c)
    if w["flops"] > 1.6e12 or w["bytes"] > 2.4e9:
        return False
    if c["op"] in ("matmul", "ffn"):  # the plain form pads every group to the largest
        cap, width = max(_counts(c)), (c["n"] if c["op"] == "matmul" else 2 * c["inter"])
        return cap * c["experts"] * (c.get("k") or c["hidden"]) * width * 2 < 8e12
    return c["rows"] * c["k"] <= 65536 * 4096


def _counts(c):
    """Rows of each group, largest first: shares ~ 1 / rank^skew."""
    share = 1.0 / np.arange(1, c["experts"] + 1) ** c["skew"]
    edge = np.floor(np.cumsum(share / share.sum()) * c["rows"] + 0.5).astype(np.int64)
    edge[-1] = c["rows"]
    return [int(v) for v in np.diff(np.concatenate([[0], edge]))]


def _blocks(n):
    return -(-n // BLOCK)


def work(c):
    if c["op"] in ("norm", "quantize"):
        n, e = c["rows"] * c["k"], ELEM[c["dtype"]]
        if c["op"] == "quantize":
            return {"bytes": n * (e + 1) + 4 * c["rows"], "flops": 3 * n}
        b = n * e * (1 + 2 * c["residual"] + c["y"]) + c["k"] * e
        if c["out"] != "none":
            b += n + 4 * c["rows"] * (1 if c["out"] == "int8" else _blocks(c["k"]))
        return {"bytes": b, "flops": n * (5 + c["residual"] + 2 * (c["out"] != "none"))}
    active = sum(v > 0 for v in _counts(c))
    if c["op"] == "matmul":
        b = active * c["n"] * (c["k"] + 4) + c["rows"] * (c["k"] * ELEM[c["x"]] + 4 * (c["x"] == "i8"))
        b += c["rows"] * c["n"] * ELEM[c["out"]] + 16 * c["experts"]
        return {"bytes": b, "flops": 2 * c["rows"] * c["n"] * c["k"]}
    h, i = c["hidden"], c["inter"]
    b = active * (3 * h * i + 4 * (2 * i + h)) + c["rows"] * (h * ELEM[c["x"]] + 4 * (c["x"] == "i8"))
    b += 2 * c["rows"] * h + 16 * c["experts"]
    return {"bytes": b, "flops": 6 * c["rows"] * h * i}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _rows(rows, k, dtype, g):
    """Hidden states: N(0, 1), a few channels ten times larger, as such states have."""
    x = torch.randn(rows, k, device="cuda", generator=g)
    x[:, torch.randint(0, k, (max(1, k // 200),), device="cuda", generator=g)] *= 10.0
    return x.to(DTYPES[dtype])


def _padded(*shape, dtype):
    """Rows that start at multiples of 16 bytes, as a loader lays weights out."""
    unit = 16 // ELEM[dtype]
    wide = -(-shape[-1] // unit) * unit
    return torch.zeros(*shape[:-1], wide, device="cuda", dtype=DTYPES[dtype])[..., :shape[-1]]


def _weights8(lead, n, k, g):
    """int8 weights [*lead, n, k] as a quantizer with a scale per channel leaves normal ones, and their scales."""
    w = _padded(*lead, n, k, dtype="i8")
    flat = w.as_strided((math.prod(lead), n, k), (n * w.stride(-2), w.stride(-2), 1))
    for j in range(flat.shape[0]):
        v = torch.randn(n, k, device="cuda", generator=g) * 32.0
        flat[j].copy_(v.round_().clamp_(-127.0, 127.0).to(torch.int8))
    s = torch.randn(*lead, n, device="cuda", generator=g)
    return w, torch.exp(0.2 * s) / (32.0 * math.sqrt(k))


def _rows8(rows, k, g):
    """int8 rows as a quantizer leaves hidden states with outlying channels, and their scales."""
    x = _padded(rows, k, dtype="i8")
    v = torch.randn(rows, k, device="cuda", generator=g)
    v[:, torch.randint(0, k, (max(1, k // 200),), device="cuda", generator=g)] *= 10.0
    s = v.abs().amax(1, keepdim=True) / 127.0
    x.copy_((v / s).round_().clamp_(-127.0, 127.0).to(torch.int8))
    return x, s[:, 0] * torch.exp(0.3 * torch.randn(rows, device="cuda", generator=g))


def _group_list(c, g):
    """The batching's compacted list: (expert, rows) of the experts that have rows, in
    ascending order, then (0, 0). Which expert has which count is drawn."""
    counts = np.array(_counts(c), dtype=np.int64)
    order = torch.randperm(c["experts"], device="cuda", generator=g).cpu().numpy()
    counts = counts[order]
    out = np.zeros((c["experts"], 2), np.int64)
    present = np.nonzero(counts)[0]
    out[:len(present), 0], out[:len(present), 1] = present, counts[present]
    return torch.from_numpy(out).cuda()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] in ("norm", "quantize"):
        s["x"] = _rows(c["rows"], c["k"], c["dtype"], g)
        if c["op"] == "norm":
            s["residual"] = _rows(c["rows"], c["k"], c["dtype"], g) if c["residual"] else None
            s["w"] = (1.0 + 0.2 * torch.randn(c["k"], device="cuda", generator=g)).to(DTYPES[c["dtype"]])
        return s
    s["groups"] = _group_list(c, g)
    s["cap"] = max(_counts(c))
    k = c["k"] if c["op"] == "matmul" else c["hidden"]
    if c["x"] == "i8":
        s["x"], s["x_scales"] = _rows8(c["rows"], k, g)
    else:
        s["x"], s["x_scales"] = _padded(c["rows"], k, dtype=c["x"]), None
        s["x"].copy_(_rows(c["rows"], k, c["x"], g))
    if c["op"] == "matmul":
        s["w"], s["w_scales"] = _weights8((c["experts"],), c["n"], k, g)
    else:
        s["w13"], s["w13_scales"] = _weights8((c["experts"], 2), c["inter"], k, g)
        s["w2"], s["w2_scales"] = _weights8((c["experts"],), k, c["inter"], g)
    return s


# ---------------------------------------------------------------------------
# One pass: the package's entry points, or the plain form
# ---------------------------------------------------------------------------

def _out_dtype(c):
    return torch.bfloat16 if c["x"] == "i8" else DTYPES[c["x"]]


def run(state):
    s, c = state, state["case"]
    if own:
        import unpermute_stable_counting_gb300 as usc
        if c["op"] == "norm":
            r = usc.moe_add_rms_norm(s["x"], s["w"], s["residual"], eps=EPS, with_y=c["y"],
                                     quantize=None if c["out"] == "none" else c["out"])
            return {k: r[k] for k in _norm_outputs(c)}
        if c["op"] == "quantize":
            r = usc.moe_quantize_int8(s["x"])
            return {"values": r["values"], "scales": r["scales"]}
        if c["op"] == "matmul":
            return usc.moe_grouped_matmul_int8(s["x"], s["w"], s["w_scales"], s["groups"], x_scales=s["x_scales"],
                                               out_dtype=DTYPES[c["out"]])["y"]
        return usc.moe_expert_ffn_int8(s["x"], s["w13"], s["w13_scales"], s["w2"], s["w2_scales"], s["groups"],
                                       x_scales=s["x_scales"], out_dtype=_out_dtype(c))["y"]
    if c["op"] == "norm":
        h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(DTYPES[c["dtype"]])
        r = (1.0 / torch.sqrt(h.double().square().mean(-1, keepdim=True) + EPS)).float()
        y = (h.float() * r) * s["w"].float()
        o = {"residual": h, "y": y.to(DTYPES[c["dtype"]])}
        if c["out"] == "int8":
            o["values"], o["scales"] = _int8(y)
        elif c["out"] == "e4m3":
            o["values"], o["scales"] = _e4m3_blocks(y)
        return {k: o[k] for k in _norm_outputs(c)}
    if c["op"] == "quantize":
        q, sc = _int8(s["x"].float())
        return {"values": q, "scales": sc}
    xp, back = _by_group(s["x"].float(), s["groups"], s["cap"])
    scales = None if s["x_scales"] is None else _by_group(s["x_scales"][:, None], s["groups"], s["cap"])[0]
    ids = s["groups"][:, 0]
    if c["op"] == "matmul":
        return _product(xp, scales, s["w"][ids], s["w_scales"][ids])[back].to(DTYPES[c["out"]])
    w13, t13 = s["w13"][ids], s["w13_scales"][ids]
    a = _product(xp, scales, w13[:, 0], t13[:, 0])
    h = a / (1.0 + torch.exp(-a)) * _product(xp, scales, w13[:, 1], t13[:, 1])
    y = _product(h.to(torch.bfloat16).float(), None, s["w2"][ids], s["w2_scales"][ids])
    return y[back].to(_out_dtype(c))


def _norm_outputs(c):
    return ["residual"] * c["residual"] + ["y"] * c["y"] + (["values", "scales"] if c["out"] != "none" else [])


def _product(x, s, w, t):
    """[groups, rows, n] of rows [groups, rows, k] (their scales s, or None) and weights [groups, n, k]."""
    y = x @ w.float().transpose(1, 2) * t[:, None, :]
    return y if s is None else y * s


def _int8(v):
    a = v.abs().amax(-1, keepdim=True).clamp_min(AMAX_FLOOR)
    full = torch.full_like(a, 127.0)  # a tensor, so that each division is one rounding
    return torch.round(v * (full / a)).to(torch.int8), (a / full)[..., 0]


def _e4m3_blocks(x):
    """(e4m3 values, their scales) of fp32 rows [..., k]."""
    k = x.shape[-1]
    v = torch.nn.functional.pad(x, (0, -k % BLOCK)).unflatten(-1, (-1, BLOCK))
    m, e = torch.frexp(v.abs().amax(-1).clamp_min(AMAX_FLOOR))  # amax = m 2^e, m in [1/2, 1)
    s = torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875))    # 448 = 0.875 * 2^9
    return (v / s[..., None]).flatten(-2)[..., :k].to(torch.float8_e4m3fn), s


def _by_group(x, groups, cap):
    """Rows [groups, cap, k], zeros past a group's rows, and the index that takes them back."""
    counts = groups[:, 1]
    ends = counts.cumsum(0)
    at = torch.arange(cap, device=x.device)
    rows = ((ends - counts)[:, None] + at).clamp_max(x.shape[0] - 1)
    xp = x[rows] * (at < counts[:, None])[..., None]
    r = torch.arange(x.shape[0], device=x.device)
    group = (r[:, None] >= ends).sum(1)
    return xp, (group, r - (ends - counts)[group])


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_norm(c, s):
    h = s["x"].double()
    if c["residual"]:
        h = h + s["residual"].double()
    o = {"residual": h}
    if c["residual"]:  # what is normalised is the rounded sum
        h = h.to(DTYPES[c["dtype"]]).double()
    y = h * torch.rsqrt((h * h).sum(1, keepdim=True) / c["k"] + EPS) * s["w"].double()
    o["y"] = y
    if c["out"] == "int8":
        o["values"], o["scales"] = _exact_int8(y)
    elif c["out"] == "e4m3":
        o["values"], o["scales"] = _exact_e4m3(y)
    return {k: o[k] for k in _norm_outputs(c)}


def _exact_int8(v):
    s = v.abs().max(dim=1).values.clamp_min(AMAX_FLOOR) / 127.0
    return torch.round(v / s[:, None]).to(torch.int8), s


def _exact_e4m3(v):
    q, scales = torch.zeros_like(v), []
    for b in range(0, v.shape[1], BLOCK):
        part = v[:, b:b + BLOCK]
        need = part.abs().max(dim=1).values.clamp_min(AMAX_FLOOR) / E4M3_MAX
        s = torch.exp2(torch.ceil(torch.log2(need)))
        s = torch.where(s * 0.5 >= need, s * 0.5, torch.where(s < need, s * 2.0, s))
        part = part / s[:, None]
        _, e = torch.frexp(part)  # |part| in [2^(e-1), 2^e)
        step = torch.exp2((e - 1).clamp_min(-6).double() - 3)
        q[:, b:b + BLOCK] = torch.round(part / step) * step
        scales.append(s)
    return q, torch.stack(scales, 1)


def _exact_product(x, s, w, t):
    y = x @ w.double().T * t.double()
    return y if s is None else y * s.double()[:, None]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        return _exact_norm(c, s)
    if c["op"] == "quantize":
        q, sc = _exact_int8(s["x"].double())
        return {"values": q, "scales": sc}
    parts, at = [], 0
    for e, count in s["groups"].tolist():
        if count == 0:
            continue
        rows = s["x"][at:at + count].double()
        sc = None if s["x_scales"] is None else s["x_scales"][at:at + count]
        if c["op"] == "matmul":
            parts.append(_exact_product(rows, sc, s["w"][e], s["w_scales"][e]))
        else:
            a, b = (_exact_product(rows, sc, s["w13"][e, j], s["w13_scales"][e, j]) for j in (0, 1))
            h = (a * torch.sigmoid(a) * b).to(torch.bfloat16).double()
            parts.append(_exact_product(h, None, s["w2"][e], s["w2_scales"][e]))
        at += count
    return torch.cat(parts)
