"""Plain CPU reference for the operators of a sparse transformer block, float64 throughout: layer
norm, rotary positions and attention within the items of a ragged batch, with their gradients.

TEST INFRASTRUCTURE.  Only tests/ and __graft_entry__.smoke() may use this module; the HIP library
never does.

The pages name the operators without formulas (attention in full mode, rotary phases from voxel
coordinates, norms with and without affine weights: trellis_sparse_mrp_mlx commit log); the
reading is the usual one.  Written from the definitions, one item and one head at a time:

* layer norm: h = (x - mean) / sqrt(var + eps) over a row, biased variance; y = h g + b.
* rotary positions: pair i of a head, axis i // F, angle = position * frequency, rotated as the
  complex number u + j v; gradient: rotated back.
* attention: softmax(scale q k^T) v of the queries and keys of one item; query head h reads key
  head h // (heads / kv_heads); a query without keys gives 0 and log sum -inf.

Pins (tests/test_transformer_pins.py): torch's float64 autograd of the same definitions, central
differences, invariants, and planted mistakes that must fail.
"""
from __future__ import annotations

import numpy as np


def layer_norm(x, gamma=None, beta=None, eps: float = 1e-5):
    """(y, mean, rstd) of the rows of x [N, C]."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(axis=1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if gamma is not None:
        y = y * np.asarray(gamma, dtype=np.float64)
    if beta is not None:
        y = y + np.asarray(beta, dtype=np.float64)
    return y, mean, rstd


def layer_norm_grad(dy, x, gamma=None, eps: float = 1e-5):
    """(dx, dgamma, dbeta)."""
    dy = np.asarray(dy, dtype=np.float64)
    h, _, rstd = layer_norm(x, eps=eps)
    a = dy if gamma is None else dy * np.asarray(gamma, dtype=np.float64)
    dx = rstd[:, None] * (a - a.mean(axis=1, keepdims=True) - h * (a * h).mean(axis=1, keepdims=True))
    return dx, (dy * h).sum(axis=0), dy.sum(axis=0)


def rope(x, positions, freq, interleaved: bool, magnitude: float = 1.0, back: bool = False):
    """Rotary positions of x [N, heads, D]; positions [N, axes], freq [F]."""
    x = np.asarray(x, dtype=np.float64)
    positions = np.asarray(positions, dtype=np.float64)
    freq = np.asarray(freq, dtype=np.float64)
    pairs = positions.shape[1] * len(freq)
    y = x.copy()
    for i in range(pairs):
        u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        t = positions[:, i // len(freq)] * freq[i % len(freq)]
        z = (x[:, :, u] + 1j * x[:, :, v]) * (magnitude * np.exp((-1j if back else 1j) * t))[:, None]
        y[:, :, u], y[:, :, v] = z.real, z.imag
    return y


def _blocks(q, k, q_offsets, k_offsets):
    """(query rows, key rows, query head, key head) of every non-empty product."""
    heads, kv_heads = q.shape[1], k.shape[1]
    for b in range(len(q_offsets) - 1):
        rows, keys = slice(q_offsets[b], q_offsets[b + 1]), slice(k_offsets[b], k_offsets[b + 1])
        if rows.stop > rows.start and keys.stop > keys.start:
            for h in range(heads):
                yield rows, keys, h, h // (heads // kv_heads)


def _probabilities(qi, ki, scale):
    s = scale * (qi @ ki.T)
    top = s.max(axis=1, keepdims=True)
    lse = top + np.log(np.exp(s - top).sum(axis=1, keepdims=True))
    return np.exp(s - lse), lse[:, 0]


def attention(q, k, v, q_offsets, k_offsets, scale: float):
    """(out [Nq, heads, D], lse [Nq, heads])."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    out, lse = np.zeros_like(q), np.full(q.shape[:2], -np.inf)
    for rows, keys, h, j in _blocks(q, k, q_offsets, k_offsets):
        p, lse[rows, h] = _probabilities(q[rows, h], k[keys, j], scale)
        out[rows, h] = p @ v[keys, j]
    return out, lse


def attention_grad(dout, q, k, v, q_offsets, k_offsets, scale: float):
    """(dq, dk, dv)."""
    dout, q, k, v = (np.asarray(t, dtype=np.float64) for t in (dout, q, k, v))
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for rows, keys, h, j in _blocks(q, k, q_offsets, k_offsets):
        p, _ = _probabilities(q[rows, h], k[keys, j], scale)
        dp = dout[rows, h] @ v[keys, j].T
        ds = scale * p * (dp - (p * dp).sum(axis=1, keepdims=True))
        dq[rows, h] = ds @ k[keys, j]
        dk[keys, j] += ds.T @ q[rows, h]
        dv[keys, j] += p.T @ dout[rows, h]
    return dq, dk, dv


def attention_error_bounds(q, k, v, q_offsets, k_offsets, scale: float, u: float, tiny: float, u_p: float, dout=None):
    """Componentwise bounds of an evaluation with float32 accumulation and storage roundoff `u`.

    u_p: relative and `tiny` smallest absolute roundoff of the probabilities and of e = p (dp - d)
    where they are rounded for the matrix product (0 when they stay float32); `tiny` is that of
    the scaled numbers the library rounds (p times 2^15 or at most 1, e taken to the largest
    |dout|).  With f = 2^-23 (one float32 operation, any rounding mode):
      score      |ds|  <= (D + 2) f scale sum |q||k|
      p          rel   <= eta = 2 max_j |ds| + (keys + 64) f + 2^-20  (exponential, sum, 1 / l)
      out        |err| <= u |out| + (u_p + eta) sum p |v| + tiny sum |v|
      d          |err| <= sum |dout| err(out) + (D + 2) f sum |dout||out|
      dp         |err| <= (D + 2) f sum |dout||v|
      e          |err| <= (u_p + eta) |e| + p (err(dp) + err(d)) + tiny max|dout|
      dq, dk, dv       <= u |.| + the products of those with |k|, |q|, |dout|, (terms) f each
    Returns (out, lse) bounds, and with dout also (dq, dk, dv).
    """
    f = 2.0 ** -23
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    d = q.shape[2]
    ob, lb = np.zeros_like(q), np.zeros(q.shape[:2])
    grads = None
    if dout is not None:
        dout = np.asarray(dout, dtype=np.float64)
        grads = [np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)]
    for rows, keys, h, j in _blocks(q, k, q_offsets, k_offsets):
        qi, ki, vi = q[rows, h], k[keys, j], v[keys, j]
        m, n = len(qi), len(ki)
        p, lse = _probabilities(qi, ki, scale)
        ds = (d + 2) * f * abs(scale) * (np.abs(qi) @ np.abs(ki).T)
        eta = 2 * ds.max(axis=1, keepdims=True) + (n + 64) * f + 2.0 ** -20
        out = p @ vi
        ob[rows, h] = u * np.abs(out) + (u_p + eta) * (p @ np.abs(vi)) + tiny * np.abs(vi).sum(axis=0)
        lb[rows, h] = eta[:, 0] + 4 * f * np.abs(lse)
        if dout is None:
            continue
        g = dout[rows, h]
        dp = g @ vi.T
        e = p * (dp - (p * dp).sum(axis=1, keepdims=True))
        err_d = (np.abs(g) * ob[rows, h]).sum(axis=1, keepdims=True) + (d + 2) * f * (np.abs(g) * np.abs(out)).sum(axis=1, keepdims=True)
        err_e = (u_p + eta) * np.abs(e) + p * ((d + 2) * f * (np.abs(g) @ np.abs(vi).T) + err_d)
        peak_rows, peak = np.abs(g).max(axis=1, keepdims=True), np.abs(dout[rows]).max()
        dq = scale * (e @ ki)
        grads[0][rows, h] = u * np.abs(dq) + abs(scale) * ((err_e + tiny * peak_rows + (n + 2) * f * np.abs(e)) @ np.abs(ki))
        grads[1][keys, j] += abs(scale) * ((err_e + tiny * peak + (m + 2) * f * np.abs(e)).T @ np.abs(qi))
        grads[2][keys, j] += ((u_p + eta + (m + 2) * f) * p + tiny).T @ np.abs(g)
    if dout is None:
        return ob, lb
    _, dk, dv = attention_grad(dout, q, k, v, q_offsets, k_offsets, scale)
    grads[1] += u * np.abs(dk)
    grads[2] += u * np.abs(dv)
    return ob, lb, grads[0], grads[1], grads[2]


# --------------------------------------------------- root-mean-square norm, embedding, sliding windows
#
# * root-mean-square norm: t = x + residual; y = t g / sqrt(mean(t^2) + eps); in 8 bits: a scale s = max |y| /
#   448 a group of channels, q = y / s rounded to e4m3 (3 fraction bits, exponents from -6, no infinity).
# * embedding: scale * table[token], zeros for a token outside the table.
# * sliding window: query i of an item with nq queries and nk keys stands at p = i + nk - nq and sees key j
#   if j <= p + right and (j >= p - left or j < sinks).

def rms_norm(x, residual=None, gamma=None, eps: float = 1e-6):
    """(y, total, rstd) of the rows of x + residual [N, C]."""
    t = np.asarray(x, dtype=np.float64)
    if residual is not None:
        t = t + np.asarray(residual, dtype=np.float64)
    rstd = 1.0 / np.sqrt((t ** 2).mean(axis=1) + eps)
    y = t * rstd[:, None]
    return y if gamma is None else y * np.asarray(gamma, dtype=np.float64), t, rstd


def rms_norm_grad(dy, total, rstd, gamma=None, dtotal=None):
    """(dx, dgamma) where rstd is a function of total, given its value."""
    dy, t, r = np.asarray(dy, dtype=np.float64), np.asarray(total, dtype=np.float64), np.asarray(rstd, dtype=np.float64)[:, None]
    a = dy if gamma is None else dy * np.asarray(gamma, dtype=np.float64)
    h = t * r
    dx = r * (a - h * (a * h).mean(axis=1, keepdims=True))
    return dx if dtotal is None else dx + np.asarray(dtotal, dtype=np.float64), (dy * h).sum(axis=0)


def e4m3(v):
    """v rounded to the nearest e4m3 number, ties to even; |v| <= 448."""
    v = np.asarray(v, dtype=np.float64)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -20))), -6.0) - 3.0)
    return np.rint(v / step) * step


def group_scales(y, group: int):
    """max(max |y| / 448, 2^-126) of each group of channels, [N, groups]; group 0: the row."""
    y = np.abs(np.asarray(y, dtype=np.float64))
    group = group or y.shape[1]
    tops = [y[:, c:c + group].max(axis=1) for c in range(0, y.shape[1], group)]
    return np.maximum(np.stack(tops, axis=1) / 448.0, 2.0 ** -126)


def embedding(table, tokens, scale: float = 1.0):
    table, out = np.asarray(table, dtype=np.float64), np.zeros((len(tokens), np.shape(table)[1]))
    for i, t in enumerate(tokens):
        if 0 <= t < len(table):
            out[i] = scale * table[t]
    return out


def embedding_grad(dout, tokens, rows: int, scale: float = 1.0):
    d = np.zeros((rows, np.shape(dout)[1]))
    for t, g in zip(tokens, np.asarray(dout, dtype=np.float64)):
        if 0 <= t < rows:
            d[t] += scale * g
    return d


def window_mask(nq: int, nk: int, left=None, right=None, sinks: int = 0):
    """Which keys each query of an item sees, [nq, nk]; None: no end."""
    seen = np.ones((nq, nk), dtype=bool)
    for i in range(nq):
        p = i + nk - nq
        for j in range(nk):
            if right is not None and j > p + right:
                seen[i, j] = False
            if left is not None and j < p - left and j >= sinks:
                seen[i, j] = False
    return seen


def _window_blocks(q, k, q_offsets, k_offsets, window, k_lengths=None):
    """(query rows, key rows, query head, key head, mask) of every product."""
    heads, kv_heads, masks = q.shape[1], k.shape[1], {}
    for b in range(len(q_offsets) - 1):
        nq, nk = q_offsets[b + 1] - q_offsets[b], k_offsets[b + 1] - k_offsets[b]
        if k_lengths is not None:
            nk = min(nk, k_lengths[b])
        if nq <= 0 or nk <= 0:
            continue
        if (nq, nk) not in masks:  # the rows of window_mask, without its loops
            p, j = np.arange(nq)[:, None] + (nk - nq), np.arange(nk)[None, :]
            left, right, sinks = window
            seen = np.ones((nq, nk), dtype=bool)
            if right is not None:
                seen &= j <= p + right
            if left is not None:
                seen &= (j >= p - left) | (j < sinks)
            masks[nq, nk] = seen
        rows, keys = slice(q_offsets[b], q_offsets[b + 1]), slice(k_offsets[b], k_offsets[b] + nk)
        for h in range(heads):
            yield rows, keys, h, h // (heads // kv_heads), masks[nq, nk]


def _masked_probabilities(qi, ki, scale, seen):
    s = np.where(seen, scale * (qi @ ki.T), -np.inf)
    top = s.max(axis=1, keepdims=True)
    top = np.where(np.isneginf(top), 0.0, top)
    p = np.where(seen, np.exp(np.where(seen, s, 0.0) - top), 0.0)
    total = p.sum(axis=1, keepdims=True)
    some = seen.any(axis=1, keepdims=True)
    lse = np.where(some, top + np.log(np.where(some, total, 1.0)), -np.inf)
    return p / np.where(some, total, 1.0), lse[:, 0]


def window_attention(q, k, v, q_offsets, k_offsets, scale: float, left=None, right=None, sinks: int = 0, k_lengths=None):
    """(out [Nq, heads, D], lse [Nq, heads])."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    out, lse = np.zeros_like(q), np.full(q.shape[:2], -np.inf)
    for rows, keys, h, j, seen in _window_blocks(q, k, q_offsets, k_offsets, (left, right, sinks), k_lengths):
        p, lse[rows, h] = _masked_probabilities(q[rows, h], k[keys, j], scale, seen)
        out[rows, h] = p @ v[keys, j]
    return out, lse


def window_attention_grad(dout, q, k, v, q_offsets, k_offsets, scale: float, left=None, right=None, sinks: int = 0):
    """(dq, dk, dv)."""
    dout, q, k, v = (np.asarray(t, dtype=np.float64) for t in (dout, q, k, v))
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for rows, keys, h, j, seen in _window_blocks(q, k, q_offsets, k_offsets, (left, right, sinks)):
        p, _ = _masked_probabilities(q[rows, h], k[keys, j], scale, seen)
        dp = dout[rows, h] @ v[keys, j].T
        ds = scale * p * (dp - (p * dp).sum(axis=1, keepdims=True))
        dq[rows, h] = ds @ k[keys, j]
        dk[keys, j] += ds.T @ q[rows, h]
        dv[keys, j] += p.T @ dout[rows, h]
    return dq, dk, dv


def window_attention_error_bounds(q, k, v, q_offsets, k_offsets, scale: float, u: float, tiny: float, u_p: float, dout=None,
                                  left=None, right=None, sinks: int = 0, k_lengths=None):
    """attention_error_bounds with sums over the keys that a query sees (and the queries that see a key)."""
    f = 2.0 ** -23
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    d = q.shape[2]
    ob, lb = np.zeros_like(q), np.zeros(q.shape[:2])
    grads = None
    if dout is not None:
        dout = np.asarray(dout, dtype=np.float64)
        grads = [np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)]
    for rows, keys, h, j, seen in _window_blocks(q, k, q_offsets, k_offsets, (left, right, sinks), k_lengths):
        qi, ki, vi = q[rows, h], k[keys, j], v[keys, j]
        m, n = len(qi), len(ki)
        p, lse = _masked_probabilities(qi, ki, scale, seen)
        ds = np.where(seen, (d + 2) * f * abs(scale) * (np.abs(qi) @ np.abs(ki).T), 0.0)
        eta = 2 * ds.max(axis=1, keepdims=True) + (n + 64) * f + 2.0 ** -20
        out = p @ vi
        ob[rows, h] = u * np.abs(out) + (u_p + eta) * (p @ np.abs(vi)) + tiny * (seen @ np.abs(vi))
        lb[rows, h] = eta[:, 0] + 4 * f * np.where(np.isfinite(lse), np.abs(lse), 0.0)
        if dout is None:
            continue
        g = dout[rows, h]
        dp = g @ vi.T
        e = p * (dp - (p * dp).sum(axis=1, keepdims=True))
        err_d = (np.abs(g) * ob[rows, h]).sum(axis=1, keepdims=True) + (d + 2) * f * (np.abs(g) * np.abs(out)).sum(axis=1, keepdims=True)
        err_e = (u_p + eta) * np.abs(e) + p * ((d + 2) * f * (np.abs(g) @ np.abs(vi).T) + err_d)
        peak_rows, peak = np.abs(g).max(axis=1, keepdims=True), np.abs(dout[rows]).max()
        dq = scale * (e @ ki)
        of_dq = np.where(seen, err_e + tiny * peak_rows + (n + 2) * f * np.abs(e), 0.0)
        of_dk = np.where(seen, err_e + tiny * peak + (m + 2) * f * np.abs(e), 0.0)
        grads[0][rows, h] = u * np.abs(dq) + abs(scale) * (of_dq @ np.abs(ki))
        grads[1][keys, j] += abs(scale) * (of_dk.T @ np.abs(qi))
        grads[2][keys, j] += np.where(seen, (u_p + eta + (m + 2) * f) * p + tiny, 0.0).T @ np.abs(g)
    if dout is None:
        return ob, lb
    _, dk, dv = window_attention_grad(dout, q, k, v, q_offsets, k_offsets, scale, left, right, sinks)
    grads[1] += u * np.abs(dk)
    grads[2] += u * np.abs(dv)
    return ob, lb, grads[0], grads[1], grads[2]
