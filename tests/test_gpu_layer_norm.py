"""GPU parity of layer norm, forward and backward, against the float64 oracle.

Bounds, componentwise, with f = 2^-23 (one float32 operation) and u the storage roundoff: a row
sum goes through at most 32 additions of a lane and 12 of the lanes, so statistics are off by at
most k f times the row's mean magnitude, k = 64; every output adds a few operations.
  y   : u |y| + k f (|g| rstd (|x - mean| + mean|x|) (1 + h^2) + |b|)
  dx  : u |dx| + k f rstd (|a| + mean|a| + |h| mean|a h| + (1 + |h|) mean|a| max|h| ...)
written out below; weight gradients sum n rows in float32: (n / 64 + 64) f of the magnitudes, since
a lane adds at most n / 2048 + ... rows and workgroups follow.
"""
import numpy as np
import pytest
import torch

import submanifold_sparse_convolution_amd as sc
import synth
from oracle import transformer_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}  # half the smallest subnormal of the storage
F, K = 2.0 ** -23, 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    sc.load_library()


def inputs(n, c, dtype, seed, shift=0.0, affine=True):
    rng = np.random.default_rng(seed)
    x = synth.round_to(rng.standard_normal((n, c)) * 2.0 + shift + rng.standard_normal(c), dtype)
    dy = synth.round_to(rng.standard_normal((n, c)) * 0.1, dtype)
    g = synth.round_to(1.0 + 0.3 * rng.standard_normal(c), dtype) if affine else None
    b = synth.round_to(0.3 * rng.standard_normal(c), dtype) if affine else None
    return x, dy, g, b


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def dev(t):
    return None if t is None else t.to(DEV)


def within(got, want, bound, what):
    got = f64(got)
    assert got.shape == want.shape and np.isfinite(got).all(), what
    worst = float((np.abs(got - want) / np.maximum(bound, 1e-300)).max()) if got.size else 0.0
    print(f"  {what}: worst error / bound {worst:.3f}", flush=True)
    assert worst <= 1.0, what


def check(x, dy, g, b, dtype, what):
    print(what, flush=True)
    y, mean, rstd = sc.sparse_layer_norm_forward(dev(x), dev(g), dev(b), 1e-5, stats=True)
    dx, dg, db = sc.sparse_layer_norm_backward(dev(dy), dev(x), mean, rstd, dev(g))
    torch.cuda.synchronize()
    u, tiny = U[dtype], TINY[dtype]
    X, DY, G, B = f64(x), f64(dy), f64(g), f64(b)
    n, c = X.shape
    wy, wm, wr = ref.layer_norm(X, G, B)
    ga = np.ones(c) if g is None else np.abs(G)
    ba = np.zeros(c) if b is None else np.abs(B)
    mag = np.abs(X).mean(axis=1, keepdims=True)      # of the row
    h = (X - wm[:, None]) * wr[:, None]
    eh = K * F * (wr[:, None] * (np.abs(X) + mag) + np.abs(h) * (1 + wr[:, None] * mag))  # of h
    within(mean, wm, K * F * mag[:, 0], "mean")
    within(rstd, wr, K * F * wr * (1 + wr * mag[:, 0]), "rstd")
    within(y, wy, u * np.abs(wy) + tiny + ga * eh + 4 * F * (ga * np.abs(h) + ba), "y")
    wdx, wdg, wdb = ref.layer_norm_grad(DY, X, G)
    a = np.abs(DY) * ga
    rows = lambda t: t.mean(axis=1, keepdims=True)  # noqa: E731
    parts = a + rows(a) + np.abs(h) * rows(a * np.abs(h))
    e = wr[:, None] * (K * F * parts * (1 + wr[:, None] * mag) + eh * rows(a * np.abs(h)) + np.abs(h) * rows(a * eh))
    within(dx, wdx, u * np.abs(wdx) + tiny + e, "dx")
    sums = (n / 64 + 64) * F
    within(dg, wdg, u * np.abs(wdg) + tiny + (np.abs(DY) * (eh + sums * np.abs(h))).sum(axis=0), "dgamma")
    within(db, wdb, u * np.abs(wdb) + tiny + sums * np.abs(DY).sum(axis=0), "dbeta")
    return y, mean, rstd, dx, dg, db


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,c", [(1, 1), (1, 8), (3, 7), (5, 64), (33, 100), (450, 768), (257, 675), (130, 1024), (70, 1025), (9, 2048),
                                 (7, 2056), (6, 4100), (5, 8192), (3, 9001), (2, 16384)])
def test_shapes(dtype, n, c):
    check(*inputs(n, c, dtype, n * 7 + c), dtype, f"{dtype} n={n} C={c}")


@pytest.mark.parametrize("dtype,n,c", [("f32", 1500, 1100), ("f16", 2100, 2056), ("bf16", 1030, 4100), ("f16", 1300, 8200), ("f32", 1100, 8193)])
def test_rows_over_several_waves_in_turn(dtype, n, c):
    # more rows than workgroups: each sums several through the same LDS slots
    check(*inputs(n, c, dtype, n + c), dtype, f"{dtype} n={n} C={c}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows_and_a_mean_far_from_zero(dtype):
    check(*inputs(22406, 96, dtype, 5, shift=50.0), dtype, f"{dtype} 22406 rows, mean 50")


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_without_weights(dtype):
    x, dy, _, _ = inputs(77, 200, dtype, 6, affine=False)
    y, mean, rstd, dx, _, _ = check(x, dy, None, None, dtype, f"{dtype} no weights")
    plain, none, none2 = sc.sparse_layer_norm_forward(dev(x))
    assert none is None and none2 is None and torch.equal(plain, y)
    only, g, b = sc.sparse_layer_norm_backward(dev(dy), dev(x), mean, rstd, weight_grads=False)
    assert g is None and b is None and torch.equal(only, dx)


def test_in_place_reproducible_unaligned_and_on_another_stream():
    x, dy, g, b = inputs(1000, 333, "bf16", 8)
    y, mean, rstd, dx, dg, db = check(x, dy, g, b, "bf16", "reference run")
    again = check(x, dy, g, b, "bf16", "again")
    assert all(torch.equal(p, q) for p, q in zip((y, mean, rstd, dx, dg, db), again))
    xd, dyd = dev(x), dev(dy)
    assert sc.sparse_layer_norm_forward(xd, dev(g), dev(b), out=xd)[0].data_ptr() == xd.data_ptr() and torch.equal(xd, y)
    sc.sparse_layer_norm_backward(dyd, dev(x), mean, rstd, dev(g), out=dyd)
    assert torch.equal(dyd, dx)
    for shift in (1, 3):  # rows that start on any element
        buf = torch.empty(1000 * 333 + 8, dtype=torch.bfloat16, device=DEV)
        xs = buf[shift:shift + 1000 * 333].view(1000, 333)
        xs.copy_(dev(x))
        assert torch.equal(sc.sparse_layer_norm_forward(xs, dev(g), dev(b))[0], y)
    s = torch.cuda.Stream()
    xd, gd, bd = dev(x), dev(g), dev(b)
    s.wait_stream(torch.cuda.current_stream())
    other, m2, r2 = sc.sparse_layer_norm_forward(xd, gd, bd, stats=True, stream=s)
    dx2, dg2, db2 = sc.sparse_layer_norm_backward(dev(dy), xd, m2, r2, gd, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(other, y) and torch.equal(dx2, dx) and torch.equal(dg2, dg) and torch.equal(db2, db)


def test_no_rows():
    x = torch.zeros((0, 64), dtype=torch.float16, device=DEV)
    y, mean, rstd = sc.sparse_layer_norm_forward(x, stats=True)
    assert y.shape == (0, 64) and mean.shape == (0,)
    _, dg, db = sc.sparse_layer_norm_backward(x, x, mean, rstd)
    torch.cuda.synchronize()
    assert not dg.any() and not db.any()


def test_values_that_are_not_finite_stay_in_their_row():
    x, _, g, b = inputs(8, 96, "f32", 9)
    clean = sc.sparse_layer_norm_forward(dev(x), dev(g), dev(b))[0]
    x[3, 5], x[6, 0] = float("nan"), float("inf")
    y = sc.sparse_layer_norm_forward(dev(x), dev(g), dev(b))[0]
    rows = [0, 1, 2, 4, 5, 7]
    assert torch.equal(y[rows], clean[rows]) and torch.isnan(y[3]).all() and torch.isnan(y[6]).all()


def test_refusals():
    x = torch.zeros((4, 8), device=DEV)
    with pytest.raises(ValueError):
        sc.sparse_layer_norm_forward(x, gamma=torch.ones(7, device=DEV))
    with pytest.raises(ValueError):
        sc.sparse_layer_norm_forward(x, gamma=torch.ones(8, device=DEV, dtype=torch.float16))
    with pytest.raises(ValueError):
        sc.sparse_layer_norm_forward(x.t())
    with pytest.raises(ValueError):
        sc.sparse_layer_norm_backward(x, x, None, None)
    with pytest.raises(sc.SubmError) as e:
        sc.sparse_layer_norm_forward(x, eps=0.0)
    assert e.value.name == "SUBM_ERR_INVALID_ARG"
    with pytest.raises(sc.SubmError) as e:
        sc.sparse_layer_norm_forward(torch.zeros((1, 16385), device=DEV))
    assert e.value.name == "SUBM_ERR_UNSUPPORTED"
