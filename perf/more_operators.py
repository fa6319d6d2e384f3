"""Measured cases of further operators of the sparse transformer block: root-mean-square norm with the
residual's addition (and its output in 8 bits with scales), embedding lookup with its gradient, and
attention within a sliding window that keeps an item's first keys visible (sinks).

`own` selects what `run` computes: False the plain form (elementary torch operations in float32,
rounded once at the end), True the framework's calls.  `prepare` makes the same state for both.

Rows of all items are concatenated; item b holds rows offsets[b] .. offsets[b + 1] - 1.  Query i of an item
with nq queries and nk keys stands at key position i + nk - nq.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6
ALL = -1  # a window without an end


def listed():
    return [
        # The tiny 450-voxel shell's tokens through a block's norm while sampling, residual added: latency.
        {"name": "rms forward 450x768 f16", "op": "rms", "mode": "forward", "type": "f16", "n": 450, "c": 768, "residual": True, "group": 0},
        # The 135,826-voxel shell's tokens before a linear layer in 8 bits: residual, norm, a scale each 128 channels.
        {"name": "rms 8 bits 135826x1024 bf16", "op": "rms", "mode": "8 bits", "type": "bf16", "n": 135826, "c": 1024, "residual": True, "group": 128},
        # Gradients on a small set in float32, rows that no wide load divides.
        {"name": "rms backward 4099x675 f32", "op": "rms", "mode": "backward", "type": "f32", "n": 4099, "c": 675, "residual": False, "group": 0},
        # Gradients at full size: the input's (joined with the residual stream's) and the weight's.
        {"name": "rms backward 135826x1024 bf16", "op": "rms", "mode": "backward", "type": "bf16", "n": 135826, "c": 1024, "residual": True, "group": 0},
        # Codebook entries of a small set's tokens, scaled: one sampling step.
        {"name": "embed 450x768 f16 of 8192", "op": "embed", "mode": "forward", "type": "f16", "n": 450, "c": 768, "rows": 8192, "skew": 0.0, "absent": 0.0, "bits": 64},
        # Gradient of a codebook on a small set: a table about as long as the set, odd rows, float32.
        {"name": "embed backward 4099x675 f32 of 1021", "op": "embed", "mode": "backward", "type": "f32", "n": 4099, "c": 675, "rows": 1021, "skew": 0.0, "absent": 0.1, "bits": 32},
        # Gradient of a large table at full size: a few tokens are a large part of all, some are padding.
        {"name": "embed backward 135826x1024 bf16 of 65536", "op": "embed", "mode": "backward", "type": "bf16", "n": 135826, "c": 1024, "rows": 65536, "skew": 1.0, "absent": 0.05, "bits": 64},
        # One new token per sequence, grouped heads, a window of 4,096 keys and 4 sinks of long caches.
        {"name": "window one token 8x30k 16/4x128 bf16", "op": "window", "mode": "forward", "type": "bf16", "q_lens": "1,1,1,1,1,1,1,1", "k_lens": "32768,30011,28672,32001,17,32768,31999,20480",
         "heads": 16, "kv_heads": 4, "dim": 128, "left": 4095, "right": 0, "sinks": 4},
        # Serialised voxels of four items, each sees its neighbours both ways and the item's first 8 rows.
        {"name": "window both ways 9371 12x64 f16", "op": "window", "mode": "forward", "type": "f16", "q_lens": "4001,450,2799,2121", "k_lens": "", "heads": 12, "kv_heads": 12, "dim": 64,
         "left": 255, "right": 256, "sinks": 8},
        # A long prompt of two items, causal, 2,048 keys and 4 sinks: the largest forward pass.
        {"name": "window causal 24576 16x128 bf16", "op": "window", "mode": "forward", "type": "bf16", "q_lens": "13001,11575", "k_lens": "", "heads": 16, "kv_heads": 16, "dim": 128,
         "left": 2047, "right": 0, "sinks": 4},
        # Forward and backward of a fine-tuning step on ragged items, grouped heads, causal without an end.
        {"name": "causal train 7813 12/4x64 f16", "op": "window", "mode": "train", "type": "f16", "q_lens": "2048,1733,0,2971,1061", "k_lens": "", "heads": 12, "kv_heads": 4, "dim": 64,
         "left": ALL, "right": 0, "sinks": 0},
        # Forward and backward on two long items, a causal window of 1,024 keys and 4 sinks: the largest training pass.
        {"name": "window train 16384 16x128 bf16", "op": "window", "mode": "train", "type": "bf16", "q_lens": "9000,7384", "k_lens": "", "heads": 16, "kv_heads": 16, "dim": 128,
         "left": 1023, "right": 0, "sinks": 4},
    ]


# ------------------------------------------------------------------------------ drawn cases

def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _lens(rng, items, longest):
    """Lengths of some items, ragged within a factor of three of the longest."""
    return [max(1, round(longest * rng.uniform(0.34, 1.0))) for _ in range(items)]


def draw(rng):
    op = rng.choice(["rms", "rms", "embed", "window", "window", "window"])
    kind = rng.choice(["f16", "bf16", "bf16", "f32"])
    most = 135826 * 1024 * 2
    if op == "rms":
        c = rng.choice([_log(rng, 24, 2048), 8 * _log(rng, 4, 256)])
        n = _log(rng, 1, min(200000, most // (c * SIZE[kind])))
        return {"op": op, "mode": rng.choice(["forward", "8 bits", "backward"]), "type": kind, "n": n, "c": c, "residual": rng.random() < 0.7,
                "group": rng.choice([0, 32, 64, 128, 128])}
    if op == "embed":
        c = rng.choice([_log(rng, 24, 2048), 8 * _log(rng, 4, 256)])
        n = _log(rng, 1, min(135826, most // (c * SIZE[kind])))
        return {"op": op, "mode": rng.choice(["forward", "backward", "backward"]), "type": kind, "n": n, "c": c, "rows": _log(rng, 2, min(65536, most // (2 * c * SIZE[kind]))),
                "skew": rng.choice([0.0, 0.7, 1.0]), "absent": rng.choice([0.0, 0.05, 0.3]), "bits": rng.choice([32, 64])}
    heads = rng.choice([4, 6, 8, 12, 16])
    kv_heads = heads // rng.choice([d for d in (1, 1, 2, 4) if heads % d == 0])
    dim = rng.choice([32, 40, 64, 64, 80, 96, 128, 128])
    mode = rng.choice(["one token", "chunk", "self", "train", "train"])
    items = rng.choice([1, 2, 3, 4, 8])
    slow = 4 if kind == "f32" else 1
    k = []
    if mode == "one token":
        items = rng.choice([1, 3, 8, 17])
        q, k = [1] * items, _lens(rng, items, _log(rng, 1, 240000 // (items * slow)))
    elif mode == "chunk":  # new tokens of a prompt after those that the cache holds
        q = _lens(rng, items, _log(rng, 2, 2000 // slow))
        k = [n + m for n, m in zip(q, _lens(rng, items, _log(rng, 1, 8192 // (slow * items))))]
    elif mode == "self":
        q = _lens(rng, items, _log(rng, 2, 16384 // (items * slow)))
    else:  # gradients of sets of a few tokens are mostly rounding: none shorter than 48
        q = _lens(rng, items, _log(rng, 144, 9000 // (items * slow)))
    if len(q) > 1 and not k and rng.random() < 0.3:
        q[rng.randrange(len(q))] = 0
    left = rng.choice([ALL, _log(rng, 16, 4096), _log(rng, 16, 4096), _log(rng, 16, 4096)])
    right = 0 if k else rng.choice([0, 0, 0, _log(rng, 16, 1024), ALL if left != ALL else 0])
    return {"op": op, "mode": "train" if mode == "train" else "forward", "type": kind, "q_lens": ",".join(map(str, q)), "k_lens": ",".join(map(str, k)), "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "left": left, "right": right, "sinks": rng.choice([0, 1, 4, 4, _log(rng, 5, 64)])}


# ---------------------------------------------------------------------------------- inputs

def _lengths(case):
    q = [int(t) for t in case["q_lens"].split(",")]
    k = [int(t) for t in case["k_lens"].split(",")] if case["k_lens"] else q
    return q, k


def _offsets(lens):
    return torch.tensor([0, *lens], dtype=torch.int64).cumsum(0).to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    kind = TYPES[case["type"]]
    normal = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
    s = {"case": case}
    if case["op"] == "rms":
        n, c = case["n"], case["c"]
        x = normal(n, c) * (0.5 + torch.rand(n, 1, generator=g, device=DEV)) + 0.3 * normal(c)
        s["gamma"] = (1.0 + 0.2 * normal(c)).to(kind)
        if case["mode"] == "backward":  # what the forward pass kept: the sum that it normalised, 1 / root mean square
            s["total"] = x.to(kind)
            s["rstd"] = torch.rsqrt(s["total"].float().square().mean(1) + EPS)
            s["dy"] = (0.05 * normal(n, c)).to(kind)
            s["dtotal"] = (0.05 * normal(n, c)).to(kind) if case["residual"] else None
        else:
            s["residual"] = x.to(kind) if case["residual"] else None
            s["x"] = (0.3 * normal(n, c)).to(kind) if case["residual"] else x.to(kind)
    elif case["op"] == "embed":
        n, c, rows = case["n"], case["c"], case["rows"]
        # skew 0: every row as often; 1: row r about as often as 1 / (r + 1)
        u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64)
        even, zipf = u * rows, torch.exp(u * math.log(rows + 1)) - 1.0
        at = torch.where(torch.rand(n, generator=g, device=DEV) < case["skew"], zipf, even).long().clamp(0, rows - 1)
        at = torch.randperm(rows, generator=g, device=DEV)[at]
        at = torch.where(torch.rand(n, generator=g, device=DEV) < case["absent"], torch.full_like(at, -1), at)  # padding
        s["tokens"] = at.to(torch.int32) if case["bits"] == 32 else at
        s["scale"] = math.sqrt(c)
        if case["mode"] == "forward":
            s["table"] = (normal(rows, c) / math.sqrt(c)).to(kind)
        else:
            s["dout"] = (0.05 * normal(n, c)).to(kind)
    else:
        ql, kl = _lengths(case)
        h, kh, d = case["heads"], case["kv_heads"], case["dim"]
        s["q_off"], s["k_off"] = _offsets(ql), _offsets(kl)
        s["max_q"], s["max_k"] = max(ql), max(kl)
        if case["k_lens"]:
            s["q"] = normal(sum(ql), h, d).to(kind)
            s["kv"] = normal(sum(kl), 2 * kh, d).to(kind)
        else:
            s["qkv"] = normal(sum(ql), h + 2 * kh, d).to(kind)
        if case["mode"] == "train":
            s["dout"] = (0.05 * normal(sum(ql), h, d)).to(kind)
    return s


def _heads(s):
    """q, k, v as views of what the projections wrote."""
    h, kh = s["case"]["heads"], s["case"]["kv_heads"]
    if "qkv" in s:
        return s["qkv"][:, :h], s["qkv"][:, h:h + kh], s["qkv"][:, h + kh:]
    return s["q"], s["kv"][:, :kh], s["kv"][:, kh:]


# ------------------------------------------------------------------------------ plain forms

def _spread(scales, group, c):
    """The scale of every channel."""
    return scales.repeat_interleave(group, 1)[:, :c]


def _plain_rms(s):
    case, kind = s["case"], TYPES[s["case"]["type"]]
    gamma, c = s["gamma"].float(), case["c"]
    if case["mode"] == "backward":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        h = s["total"].float() * rstd
        a = dy * gamma
        dx = rstd * (a - h * (a * h).mean(1, keepdim=True))
        if case["residual"]:
            dx = dx + s["dtotal"].float()
        return {"dx": dx.to(kind), "dgamma": (dy * h).sum(0).to(kind)}
    x = s["x"].float()
    if case["residual"]:
        x = x + s["residual"].float()
    rstd = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    y = x * rstd * gamma
    got = {"total": x.to(kind)} if case["residual"] else {}
    if case["mode"] == "forward":
        return {"y": y.to(kind), "rstd": rstd[:, 0], **got}
    group = case["group"] or c
    blocks = torch.nn.functional.pad(y.abs(), (0, -c % group)).reshape(case["n"], -1, group)
    scales = (blocks.amax(2) / 448.0).clamp(min=2.0 ** -126)  # 448: the largest e4m3 number
    wide = _spread(scales, group, c)
    return {"q": (y / wide).to(torch.float8_e4m3fn), "scales": scales, **got}


def _plain_embed(s):
    case, kind = s["case"], TYPES[s["case"]["type"]]
    at = s["tokens"].long()
    there = (at >= 0)[:, None]
    if case["mode"] == "forward":
        return {"out": (s["table"].float()[at.clamp(min=0)] * s["scale"] * there).to(kind)}
    d = torch.zeros(case["rows"], case["c"], device=at.device)
    d.index_add_(0, at.clamp(min=0), s["dout"].float() * there)
    return {"dtable": (d * s["scale"]).to(kind)}


def _padded(x, off, longest):
    """Rows of all items [n, h, d] as [items, h, longest, d] in float32, zeros beyond an item's end; and which rows are there."""
    at = off[:-1, None] + torch.arange(longest, device=x.device)
    there = at < off[1:, None]
    rows = x.float()[at.clamp(max=x.shape[0] - 1)] * there[:, :, None, None]
    return rows.transpose(1, 2), there


def _rows(x, off, n):
    """The inverse: [items, h, longest, d] back to rows [n, h, d]."""
    row = torch.arange(n, device=x.device)
    item = (row[:, None] >= off[None, 1:]).sum(1)
    return x[item, :, row - off[item]]


def _plain_window(s):
    case = s["case"]
    q, k, v = _heads(s)
    kind, nq, nk, d = q.dtype, q.shape[0], k.shape[0], q.shape[2]
    items, kh, g = s["q_off"].shape[0] - 1, case["kv_heads"], case["heads"] // case["kv_heads"]
    scale = 1.0 / math.sqrt(d)
    qp, _ = _padded(q, s["q_off"], s["max_q"])
    qp = qp.reshape(items, kh, g * s["max_q"], d)  # the g query heads that share a key head: g times as many rows of it
    kp, there = _padded(k, s["k_off"], s["max_k"])
    vp, _ = _padded(v, s["k_off"], s["max_k"])
    # which keys a query sees
    key = torch.arange(s["max_k"], device=q.device)
    shift = (s["k_off"].diff() - s["q_off"].diff())[:, None, None]
    at = torch.arange(s["max_q"], device=q.device)[:, None] + shift
    seen = there[:, None, :].expand(items, s["max_q"], s["max_k"])
    if case["right"] != ALL:
        seen = seen & (key <= at + case["right"])
    if case["left"] != ALL:
        seen = seen & ((key >= at - case["left"]) | (key < case["sinks"]))
    seen = seen.repeat(1, g, 1)[:, None]
    score = torch.matmul(qp, kp.transpose(2, 3).contiguous())
    score *= scale
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = score.sub_(top).exp_()
    total = p.sum(3, keepdim=True)
    some = total > 0
    p *= torch.where(some, 1.0 / total, torch.zeros_like(total))
    out = torch.matmul(p, vp)
    lse = torch.where(some, top + torch.log(total), torch.full_like(top, -math.inf))
    split = lambda t: t.reshape(items, kh * g, s["max_q"], t.shape[3])  # noqa: E731
    got = {"out": _rows(split(out), s["q_off"], nq).to(kind), "lse": _rows(split(lse), s["q_off"], nq)[:, :, 0]}
    if case["mode"] == "forward":
        return got
    do, _ = _padded(s["dout"], s["q_off"], s["max_q"])
    do = do.reshape(items, kh, g * s["max_q"], d)
    delta = (do * out).sum(3, keepdim=True)
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = torch.matmul(do, vp.transpose(2, 3).contiguous()).sub_(delta).mul_(p).mul_(scale)
    dq = torch.matmul(ds, kp)
    dk = torch.matmul(ds.transpose(2, 3), qp)
    dq, dk, dv = _rows(split(dq), s["q_off"], nq), _rows(dk, s["k_off"], nk), _rows(dv, s["k_off"], nk)
    return {**got, "dqkv": torch.cat([dq, dk, dv], 1).to(kind)}


# ------------------------------------------------------------------------- the framework's

def _own_rms(s):
    import submanifold_sparse_convolution_amd as sc

    case = s["case"]
    if case["mode"] == "backward":
        dx, dgamma = sc.sparse_rms_norm_backward(s["dy"], s["total"], s["rstd"], s["gamma"], dtotal=s["dtotal"])
        return {"dx": dx, "dgamma": dgamma}
    if case["mode"] == "forward":
        y, total, rstd = sc.sparse_rms_norm_forward(s["x"], s["gamma"], s["residual"], EPS, stats=True)
        return {"y": y, "rstd": rstd, "total": total} if case["residual"] else {"y": y, "rstd": rstd}
    q, scales, total, _ = sc.sparse_rms_norm_quantize_forward(s["x"], s["gamma"], s["residual"], EPS, group=case["group"])
    return {"q": q, "scales": scales, "total": total} if case["residual"] else {"q": q, "scales": scales}


def _own_embed(s):
    import submanifold_sparse_convolution_amd as sc

    if s["case"]["mode"] == "forward":
        return {"out": sc.sparse_embedding_forward(s["table"], s["tokens"], s["scale"])}
    return {"dtable": sc.sparse_embedding_backward(s["dout"], s["tokens"], s["case"]["rows"], s["scale"])}


def _own_window(s):
    import submanifold_sparse_convolution_amd as sc

    case = s["case"]
    q, k, v = _heads(s)
    window = {"left": None if case["left"] == ALL else case["left"], "right": None if case["right"] == ALL else case["right"], "sinks": case["sinks"]}
    out, lse = sc.sparse_window_attention_forward(q, k, v, s["q_off"], s["k_off"], **window)
    got = {"out": out, "lse": lse}
    if case["mode"] == "forward":
        return got
    h, kh = case["heads"], case["kv_heads"]
    d = torch.empty_like(s["qkv"])  # the gradients go straight into the packed projection's gradient
    sc.sparse_window_attention_backward(s["dout"], q, k, v, out, lse, s["q_off"], s["k_off"], **window, dq=d[:, :h], dk=d[:, h:h + kh], dv=d[:, h + kh:])
    return {**got, "dqkv": d}


def run(state):
    forms = (_own_rms, _own_embed, _own_window) if own else (_plain_rms, _plain_embed, _plain_window)
    return forms[("rms", "embed", "window").index(state["case"]["op"])](state)


# ------------------------------------------------------------------------ bytes and operations

def _seen(case):
    """(query and key pairs that see each other, keys that some query sees), each head counted once."""
    ql, kl = _lengths(case)
    pairs = keys = 0
    for m, n in zip(ql, kl):
        if m == 0 or n == 0:
            continue
        at = torch.arange(m, dtype=torch.int64) + n - m
        last = torch.full_like(at, n - 1) if case["right"] == ALL else (at + case["right"]).clamp(max=n - 1)
        first = torch.zeros_like(at) if case["left"] == ALL else (at - case["left"]).clamp(min=0)
        near = (last - first + 1).clamp(min=0)
        sunk = torch.minimum(torch.full_like(at, case["sinks"]), torch.minimum(first, last + 1)).clamp(min=0)
        pairs += int((near + sunk).sum())
        low = max(0, int(first.min()))
        keys += max(0, int(last.max()) + 1 - low) + min(case["sinks"], low)
    return pairs, keys


def work(case):
    b = SIZE[case["type"]]
    if case["op"] == "rms":
        n, c = case["n"], case["c"]
        if case["mode"] == "backward":
            return {"bytes": (4 if case["residual"] else 3) * n * c * b + 4 * n + 2 * c * b, "flops": 9 * n * c}
        read = 2 * n * c * b if case["residual"] else n * c * b
        kept = n * c * b if case["residual"] else 0
        if case["mode"] == "forward":
            return {"bytes": read + kept + n * c * b + 4 * n + c * b, "flops": 5 * n * c}
        scales = n * -(-c // (case["group"] or c))
        return {"bytes": read + kept + n * c + 4 * scales + c * b, "flops": 7 * n * c}
    if case["op"] == "embed":
        n, c, rows = case["n"], case["c"], case["rows"]
        if case["mode"] == "forward":  # entries that several tokens name are read once
            distinct = round(rows * -math.expm1(-n / rows))
            return {"bytes": (distinct + n) * c * b + n * case["bits"] // 8, "flops": n * c}
        there = round(n * (1.0 - case["absent"]))  # rows of padding tokens need not be read
        return {"bytes": (there + rows) * c * b + n * case["bits"] // 8, "flops": there * c}
    ql, kl = _lengths(case)
    h, kh, d = case["heads"], case["kv_heads"], case["dim"]
    pairs, keys = _seen(case)
    qs, ks = sum(ql) * h * d * b, keys * kh * d * b
    products = pairs * h * d * 2
    if case["mode"] == "forward":  # reads q and the keys and values that are seen; writes out and the log sums
        return {"bytes": 2 * qs + 2 * ks + 4 * sum(ql) * h, "flops": 2 * products}
    # forward and backward: q, k, v and dout read once, out, the log sums and three gradients written once
    return {"bytes": 4 * qs + 4 * ks + 4 * sum(ql) * h, "flops": 7 * products}


# --------------------------------------------------------------------------- 64-bit definition

def _exact_rms(s):
    case = s["case"]
    w = s["gamma"].double()
    n, c = case["n"], case["c"]
    if case["mode"] == "backward":
        x, dy = s["total"].double(), s["dy"].double()
        r = (x.pow(2).sum(1, keepdim=True) / c + EPS).pow(-0.5)
        a = dy * w
        dx = r * a - x * r ** 3 * (a * x).sum(1, keepdim=True) / c
        if case["residual"]:
            dx += s["dtotal"].double()
        return {"dx": dx, "dgamma": (dy * x * r).sum(0)}
    x = s["x"].double()
    if case["residual"]:
        x = x + s["residual"].double()
    r = (x.pow(2).sum(1, keepdim=True) / c + EPS).pow(-0.5)
    y = x * r * w
    got = {"total": x} if case["residual"] else {}
    if case["mode"] == "forward":
        return {"y": y, "rstd": r[:, 0], **got}
    group = case["group"] or c
    q, scales = torch.empty_like(y), []
    for first in range(0, c, group):
        part = y[:, first:first + group]
        scale = (part.abs().max(1, keepdim=True).values / 448.0).clamp(min=2.0 ** -126)
        scales.append(scale)
        q[:, first:first + group] = (part / scale).to(torch.float8_e4m3fn).double()
    return {"q": q, "scales": torch.cat(scales, 1), **got}


def _exact_embed(s):
    case = s["case"]
    at = s["tokens"].long()
    if case["mode"] == "forward":
        out = torch.zeros(case["n"], case["c"], dtype=torch.float64, device=DEV)
        out[at >= 0] = s["table"].double()[at[at >= 0]] * s["scale"]
        return {"out": out}
    # sorted tokens: a row's sum is the difference of two running sums
    order = torch.argsort(at, stable=True)
    ends = torch.searchsorted(at[order], torch.arange(-1, case["rows"], device=DEV), right=True)
    run = torch.zeros(case["n"] + 1, case["c"], dtype=torch.float64, device=DEV)
    torch.cumsum(s["dout"][order].double(), 0, out=run[1:])
    return {"dtable": run[ends].diff(dim=0) * s["scale"]}


def _exact_window(s):
    case = s["case"]
    q, k, v = _heads(s)
    ql, kl = _lengths(case)
    h, kh, d = case["heads"], case["kv_heads"], case["dim"]
    train = case["mode"] == "train"
    wide = lambda t: t.transpose(0, 1).double().contiguous()  # noqa: E731  [heads, rows, d]
    q, k, v = wide(q), wide(k), wide(v)
    dout = wide(s["dout"]) if train else None
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    share = lambda t: t.repeat_interleave(h // kh, 0)  # noqa: E731  key heads for query heads
    join = lambda t: t.reshape(kh, h // kh, *t.shape[1:]).sum(1)  # noqa: E731  and back
    a = b = 0
    for m, n in zip(ql, kl):
        for first in range(0, m if n else 0, 1024):  # blocks of queries against the keys that one of them may see
            rows = torch.arange(first, min(first + 1024, m), device=DEV)
            at = (rows + n - m)[:, None]
            low = 0 if case["left"] == ALL else max(0, int(at[0]) - case["left"])
            keys = torch.cat([torch.arange(0, min(case["sinks"], low), device=DEV), torch.arange(low, n, device=DEV)])
            if case["right"] != ALL:
                keys = keys[keys <= int(at[-1]) + case["right"]]
            if not len(keys):
                continue
            hidden = torch.zeros(len(rows), len(keys), dtype=torch.bool, device=DEV)
            if case["right"] != ALL:
                hidden |= keys > at + case["right"]
            if case["left"] != ALL:
                hidden |= (keys < at - case["left"]) & (keys >= case["sinks"])
            ki, vi = share(k[:, b + keys]), share(v[:, b + keys])
            w = torch.bmm(q[:, a + rows], ki.transpose(1, 2).contiguous()) / math.sqrt(d)
            w[:, hidden] = -math.inf
            norm = torch.logsumexp(w, 2)
            lse[:, a + rows] = norm
            w = torch.exp(w - torch.where(norm == -math.inf, torch.zeros_like(norm), norm)[:, :, None])
            out[:, a + rows] = torch.bmm(w, vi)
            if train:
                gi = dout[:, a + rows]
                dv[:, b + keys] += join(torch.bmm(w.transpose(1, 2).contiguous(), gi))
                e = torch.bmm(gi, vi.transpose(1, 2).contiguous())
                e = w * (e - (e * w).sum(2, keepdim=True)) / math.sqrt(d)
                dq[:, a + rows] = torch.bmm(e, ki)
                dk[:, b + keys] += join(torch.bmm(e.transpose(1, 2).contiguous(), q[:, a + rows]))
        a, b = a + m, b + n
    got = {"out": out.transpose(0, 1), "lse": lse.t()}
    if train:
        got["dqkv"] = torch.cat([t.transpose(0, 1) for t in (dq, dk, dv)], 1)
    return got


def exact(case, seed):
    s = prepare(case, seed)
    return {"rms": _exact_rms, "embed": _exact_embed, "window": _exact_window}[case["op"]](s)
