"""What a row does not see leaves its window's results alone: rows without any key beside keys that are not
finite, and large finite hidden values, which scale nothing that does not see them.

Finite hidden values meet only zeros, so results of the rows (and gradients of the keys) that do not see them
have to be the same bits; those beside values that are not finite may be computed again in another order, within
the componentwise bounds of oracle.transformer_ref.window_attention_error_bounds."""
import functools

import numpy as np
import pytest
import torch

import submanifold_sparse_convolution_amd as sc
import synth
from oracle import transformer_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    sc.load_library()


def f64(t):
    return t.double().cpu().numpy()


def make(nq, nk, heads, kv_heads, d, dtype, seed, g_scale=0.1):
    rng = np.random.default_rng(seed)
    r = lambda n, h, s: synth.round_to(rng.standard_normal((n, h, d)) * s, dtype).to(DEV)  # noqa: E731
    return r(nq, heads, 1.0), r(nk, kv_heads, 1.0), r(nk, kv_heads, 1.0), r(nq, heads, g_scale)


def both(q, k, v, g, qo, ko, window, given=None):
    """out, lse (`given`, or computed) and the gradients."""
    out, lse = sc.sparse_window_attention_forward(q, k, v, qo, ko, *window) if given is None else given
    return (out, lse, *sc.sparse_window_attention_backward(g, q, k, v, out, lse, qo, ko, *window))


def kept(mask):
    return torch.from_numpy(mask).to(DEV)


# queries, keys, window, the key that is not finite: seen by later rows of the tile alone, behind the sinks, among them
NO_KEYS = [(127, 64, (None, 0, 0), 10), (127, 64, (20, 0, 3), 40), (300, 150, (40, 5, 0), 30), (300, 150, (20, 0, 8), 2),
           (900, 600, (None, 0, 0), 10), (900, 600, (400, 0, 4), 50)]  # (the last two in parts)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("nq,nk,window,at", NO_KEYS)
@pytest.mark.parametrize("heads,kv_heads,d", [(2, 2, 64), (6, 2, 128)])
def test_rows_without_keys_beside_values_that_are_not_finite(dtype, nq, nk, window, at, heads, kv_heads, d):
    q, k, v, g = make(nq, nk, heads, kv_heads, d, dtype, nq + d)
    qo, ko = (torch.tensor([0, n], device=DEV) for n in (nq, nk))
    seen = ref.window_mask(nq, nk, *window)
    none, sees = ~seen.any(1), seen[:, at]
    assert none.sum() >= nq - nk - 5 and sees.any()
    scale, u_p = d ** -0.5, 0.0 if dtype == "f32" else U[dtype]
    a = [f64(t) for t in (q, k, v)]
    o = ([0, nq], [0, nk], scale)
    want = ref.window_attention_grad(f64(g), *a, *o, *window)
    bounds = ref.window_attention_error_bounds(*a, *o, U[dtype], TINY[dtype], u_p, f64(g), *window)[2:]
    for x in (float("nan"), float("inf")):
        for odd_rows in (False, True):  # and gradients of those rows that are not finite either
            kb, gb = k.clone(), g.clone()
            kb[at, :, 3] = x
            if odd_rows:
                gb[kept(none), :, 5] = x
            out, lse, dq, dk, dv = both(q, kb, v, gb, qo, ko, window)
            assert (out[kept(none)] == 0).all() and torch.isneginf(lse[kept(none)]).all()
            assert (dq[kept(none)] == 0).all(), (x, odd_rows)
            away = ~seen[sees].any(0)  # keys that no row sees which sees it
            for got, w, b, keep, what in zip((dq, dk, dv), want, bounds, (~sees, away, away), ("dq", "dk", "dv")):
                error = np.abs(f64(got[kept(keep)]) - w[keep])
                assert (error <= b[keep] + TINY[dtype]).all(), (what, x, odd_rows)


WINDOWS = [(40, 0, 0), (40, 0, 4), (None, 0, 0), (30, 20, 10), (2, 3, 0), (0, 0, 1), (600, 0, 40), (300, 310, 0), (0, None, 0), (500, None, 128)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("window", WINDOWS)
@pytest.mark.parametrize("nq,nk,heads,kv_heads,d", [(1500, 1500, 2, 2, 64), (700, 1300, 6, 2, 128), (300, 300, 40, 1, 40), (1100, 900, 3, 1, 96)])
def test_large_hidden_values(dtype, window, nq, nk, heads, kv_heads, d):
    # 60,000 in every channel of a key's value, or of a row's gradient: the scale of a float16 product that took
    # them in would leave others' terms among the subnormals
    q, k, v, g = make(nq, nk, heads, kv_heads, d, dtype, nq + d, g_scale=2.0 ** -7)
    qo, ko = (torch.tensor([0, n], device=DEV) for n in (nq, nk))
    seen = ref.window_mask(nq, nk, *window)
    clean = both(q, k, v, g, qo, ko, window)
    for j in (0, 3, nk // 2 - 9, nk // 2, nk - 130, nk - 1):
        vb = v.clone()
        vb[j] = 60000.0 * torch.sign(vb[j])
        got = both(q, k, vb, g, qo, ko, window)
        rows, keys = kept(~seen[:, j]), kept(~seen[seen[:, j]].any(0))
        for i, what in enumerate(("out", "lse", "dq")):
            assert torch.equal(got[i][rows], clean[i][rows]), (j, what)
        for i, what in ((3, "dk"), (4, "dv")):
            assert torch.equal(got[i][keys], clean[i][keys]), (j, what)
    for i in (0, 5, nq // 2 - 7, nq // 2, nq - 140, nq - 1):
        gb = g.clone()
        gb[i] = 60000.0 * torch.sign(gb[i])
        _, _, dq, dk, dv = both(q, k, v, gb, qo, ko, window, clean[:2])
        rows, keys = torch.arange(nq, device=DEV) != i, kept(~seen[i])
        assert torch.equal(dq[rows], clean[2][rows]), i
        assert torch.equal(dk[keys], clean[3][keys]) and torch.equal(dv[keys], clean[4][keys]), i


@pytest.mark.parametrize("window", [(511, 0, 0), (511, 0, 4), (None, 0, 0)])
def test_float16_gradients_beside_large_hidden_values(window):
    # the same against float64, with every hidden value of the compared rows large: within the bounds of the clean inputs
    n, heads, d = 1200, 2, 128
    q, k, v, g = make(n, n, heads, heads, d, "f16", 21)
    o = torch.tensor([0, n], device=DEV)
    seen = ref.window_mask(n, n, *window)
    some = np.arange(600, 664)
    a = [f64(t) for t in (q, k, v)]
    want = ref.window_attention_grad(f64(g), *a, [0, n], [0, n], d ** -0.5, *window)[0]
    bound = ref.window_attention_error_bounds(*a, [0, n], [0, n], d ** -0.5, U["f16"], TINY["f16"], U["f16"], f64(g), *window)[2]
    hidden = kept(~seen[some].any(0))
    v[hidden] = 60000.0 * torch.sign(v[hidden])
    dq = both(q, k, v, g, o, o, window)[2]
    assert (np.abs(f64(dq)[some] - want[some]) <= bound[some] + TINY["f16"]).all()


@pytest.mark.parametrize("window", [(40, 0, 0), (None, 0, 0), (30, 20, 10), (300, 0, 4), (2, 3, 0), (0, None, 0), (200, 0, 128)])
@pytest.mark.parametrize("nq,nk,heads,kv_heads,d", [(500, 500, 1, 1, 128), (260, 390, 4, 2, 64), (90, 400, 9, 1, 32)])
def test_large_values_that_are_seen(window, nq, nk, heads, kv_heads, d):
    # float16, one key's value or one row's gradient far above the others, the key with about half of every softmax
    # that sees it: a scale that missed it would take p (dp - d) past 65,504.  Bounds: those of the inputs, and the
    # half subnormal 2^-25 of p (dp - d) scaled by at least 2^14 / (2 |dout| max |v|), times the sum of |k| or |q|.
    q, k, v, g = make(nq, nk, heads, kv_heads, d, "f16", nq + d, g_scale=2.0 ** -8)
    qo, ko = (torch.tensor([0, n], device=DEV) for n in (nq, nk))
    seen = ref.window_mask(nq, nk, *window)
    q[:, :, 0] = 4.0
    boost = np.log(max(seen.sum(1).max() - 1, 1)) * d ** 0.5 / 4
    group, scale = heads // kv_heads, d ** -0.5

    def compare(k, v, g, what):
        got = both(q, k, v, g, qo, ko, window)[2:]
        for h in range(kv_heads):
            a = [f64(t) for t in (q[:, h * group:(h + 1) * group], k[:, h:h + 1], v[:, h:h + 1])]
            gh = f64(g[:, h * group:(h + 1) * group])
            want = ref.window_attention_grad(gh, *a, [0, nq], [0, nk], scale, *window)
            bounds = ref.window_attention_error_bounds(*a, [0, nq], [0, nk], scale, U["f16"], TINY["f16"], U["f16"], gh, *window)[2:]
            longest = np.where(seen, np.linalg.norm(a[2][:, 0], axis=1), 0.0).max(1)  # of the values that a row sees
            least = 2.0 ** -38 * np.linalg.norm(gh, axis=2) * longest[:, None]  # [rows, heads of the group]
            of_keys = np.where(seen, least.max(1)[:, None], 0.0).max(0)
            extra = (scale * least[:, :, None] * (seen @ np.abs(a[1][:, 0]))[:, None], scale * (of_keys[:, None] * (seen.T @ np.abs(a[0]).sum(1)))[:, None], 0.0)
            at = (slice(h * group, (h + 1) * group), slice(h, h + 1), slice(h, h + 1))
            for i, name in enumerate(("dq", "dk", "dv")):
                error = np.abs(f64(got[i][:, at[i]]) - want[i])
                assert (error <= bounds[i] + extra[i] + TINY["f16"]).all(), (what, h, name)

    for j in (0, 1, 31, 32, nk // 2 - 15, nk // 2, nk - 40, nk - 2, nk - 1):
        kb, vb = k.clone(), v.clone()
        kb[j, :, 0] = boost
        vb[j] = 60000.0 * torch.sign(vb[j])
        compare(kb, vb, g, f"key {j}")
    for i in (0, 1, 31, 32, nq // 2 - 15, nq // 2, nq - 40, nq - 2, nq - 1):
        gb = g.clone()
        gb[i] = 200.0 * torch.sign(gb[i])
        compare(k, v, gb, f"row {i}")


@functools.lru_cache(maxsize=None)
def clean_case(dtype, window):
    """Inputs of 1,600 tokens, their gradients in 64 bits and the componentwise bounds."""
    n, heads, d = 1600, 2, 64
    t = make(n, n, heads, heads, d, dtype, 31, g_scale=1.0)
    a, o, scale = [f64(x) for x in t], [0, n], d ** -0.5
    want = (*ref.window_attention(*a[:3], o, o, scale, *window), *ref.window_attention_grad(a[3], *a[:3], o, o, scale, *window))
    bounds = ref.window_attention_error_bounds(*a[:3], o, o, scale, U[dtype], TINY[dtype], 0.0 if dtype == "f32" else U[dtype], a[3], *window)
    return t, want, bounds, ref.window_mask(n, n, *window)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("window", [(255, 0, 4), (None, 0, 0), (100, 100, 0), (300, 0, 40)])
@pytest.mark.parametrize("bad", ["q", "k", "v", "dout", "all"])
def test_what_is_computed_again_is_as_exact(dtype, window, bad):
    # tokens from 700 on, every 301st, are not finite: the rows that see none of them, many of which meet them in
    # their tiles and are computed again, are within the bounds of any evaluation, component by component
    t, want, bounds, seen = clean_case(dtype, window)
    n = len(seen)
    t, at = [x.clone() for x in t], np.zeros(n, dtype=bool)
    at[700::301] = True
    for i, x in enumerate(t):
        if bad in ("all", ("q", "k", "v", "dout")[i]):
            x[kept(at), :, ::7] = float("inf") if i == 2 else float("nan")
    o = torch.tensor([0, n], device=DEV)
    got = both(*t, o, o, window)
    rows = np.zeros(n, dtype=bool)  # whose results may be anything
    if bad in ("q", "dout", "all"):
        rows |= at
    if bad in ("k", "v", "all"):
        rows |= seen[:, at].any(1)
    keys = seen[rows].any(0)
    assert (~rows).sum() >= 256
    for i, what in enumerate(("out", "lse", "dq", "dk", "dv")):
        keep = ~rows if i < 3 else ~keys
        error = np.abs(f64(got[i][kept(keep)]) - want[i][keep])
        assert (error <= bounds[i][keep] + (0.0 if i == 1 else TINY[dtype])).all(), what


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("window", [(40, 0, 0), (40, 0, 4), (None, 0, 0), (2, 3, 0), (600, 0, 40)])
@pytest.mark.parametrize("nq,nk,heads,kv_heads,d", [(700, 700, 2, 2, 64), (500, 900, 6, 2, 128), (3, 900, 12, 1, 96)])
def test_large_hidden_keys_and_other_queries(dtype, window, nq, nk, heads, kv_heads, d):
    # a key far above what a row sees, or another row's query: when their maxima rise the row's own stays where it is
    q, k, v, g = make(nq, nk, heads, kv_heads, d, dtype, nq + d)
    qo, ko = (torch.tensor([0, n], device=DEV) for n in (nq, nk))
    seen = ref.window_mask(nq, nk, *window)
    clean = both(q, k, v, g, qo, ko, window)
    for which, n in ((0, nq), (1, nk)):
        for at in sorted({0, n // 2, n - 40, n - 1} & set(range(n))):
            t = [q.clone(), k.clone()]
            t[which][at] *= 50.0
            got = both(*t, v, g, qo, ko, window)
            rows = np.arange(nq) == at if which == 0 else seen[:, at]
            keys = seen[rows].any(0)
            for i, what in enumerate(("out", "lse", "dq", "dk", "dv")):
                keep = kept(~(rows if i < 3 else keys))
                assert torch.equal(got[i][keep], clean[i][keep]), (which, at, what)
