"""What a row does not see leaves its window's results alone: rows without any key beside keys that are not
finite.  What is computed again in another order is within the componentwise bounds of
oracle.transformer_ref.window_attention_error_bounds."""
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
