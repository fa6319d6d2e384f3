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
