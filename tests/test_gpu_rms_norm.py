"""GPU parity of the root-mean-square norm with residual, in storage types and in 8 bits, forward and
backward, against the float64 oracle.

Bounds, componentwise, with f = 2^-23 (one float32 operation), u the storage roundoff and K = 64 (a row sum
goes through at most 32 additions of a lane and 12 of the lanes): the square sum is of positive terms, so it
is off by K f of itself and rstd by K f / 2 and a few operations.
  total: u |t| + f |t|;   rstd: (K / 2 + 4) f rstd;   y: u |y| + (K / 2 + 8) f |y|
  8 bits: the scale as y; q: half a step of e4m3 (2^-4 |q|, at least 2^-10) and the error of y / scale, twice that of y
  dx: u |dx| + rstd ((4 f |a| + |h| (K + 8) f mean|a h|)) + 2 f |dtotal|
  dgamma: (n / 64 + 64) f sum |dy h|, since a lane adds at most n / 1024 + 1 rows and workgroups follow.
Half the smallest subnormal is added for float16.
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
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}
F, K = 2.0 ** -23, 64
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    sc.load_library()


def inputs(n, c, dtype, seed, residual=True, affine=True):
    rng = np.random.default_rng(seed)
    r = lambda *shape, s=1.0, b=0.0: synth.round_to(b + s * rng.standard_normal(shape), dtype).to(DEV)  # noqa: E731
    return {"x": r(n, c, s=0.5), "residual": r(n, c, s=2.0) if residual else None, "gamma": r(c, s=0.3, b=1.0) if affine else None,
            "dy": r(n, c, s=0.1), "dtotal": r(n, c, s=0.1) if residual else None}


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def within(got, want, bound, what):
    got = f64(got)
    assert got.shape == want.shape and np.isfinite(got).all(), what
    worst = float((np.abs(got - want) / np.maximum(bound, 1e-300)).max()) if got.size else 0.0
    print(f"  {what}: worst error / bound {worst:.3f}", flush=True)
    assert worst <= 1.0, what


def check_8_bits(t, dtype, group, y, what):
    q, scales, total, _ = sc.sparse_rms_norm_quantize_forward(t["x"], t["gamma"], t["residual"], EPS, group=group)
    torch.cuda.synchronize()
    assert q.dtype == torch.float8_e4m3fn and q.shape == t["x"].shape
    s, rel = ref.group_scales(y, group), (K / 2 + 10) * F
    within(scales, s, rel * s, what + " scales")
    wide = np.repeat(s, group or y.shape[1], axis=1)[:, :y.shape[1]]
    v = y / wide
    within(q.float(), v, np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) + 2 * rel * np.abs(v) + 2.0 ** -30, what + " q")
    # and of nearly all values the same number as the oracle's rounding
    assert (f64(q.float()) != ref.e4m3(v)).mean() < 1e-3
    return q, scales, total


def check(t, dtype, what):
    print(what, flush=True)
    u, tiny = U[dtype], TINY[dtype]
    y, total, rstd = sc.sparse_rms_norm_forward(t["x"], t["gamma"], t["residual"], EPS, stats=True)
    base = t["x"] if t["residual"] is None else total
    dx, dg = sc.sparse_rms_norm_backward(t["dy"], base, rstd, t["gamma"], t["dtotal"])
    torch.cuda.synchronize()
    X, R, G, DY, DT = (f64(t[k]) for k in ("x", "residual", "gamma", "dy", "dtotal"))
    wy, wt, wr = ref.rms_norm(X, R, G, EPS)
    if R is None:
        assert total is None
    else:
        within(total, wt, (u + F) * np.abs(wt) + tiny, "total")
    within(rstd, wr, (K / 2 + 4) * F * wr, "rstd")
    within(y, wy, (u + (K / 2 + 8) * F) * np.abs(wy) + tiny, "y")
    r = f64(rstd)
    wdx, wdg = ref.rms_norm_grad(DY, f64(base), r, G, DT)
    a, h = np.abs(DY) * (1.0 if G is None else np.abs(G)), np.abs(f64(base)) * r[:, None]
    e = r[:, None] * (4 * F * a + (K + 8) * F * h * (a * h).mean(axis=1, keepdims=True)) + (0.0 if DT is None else 2 * F * np.abs(DT))
    within(dx, wdx, u * np.abs(wdx) + tiny + e, "dx")
    within(dg, wdg, u * np.abs(wdg) + tiny + (len(X) / 64 + 64) * F * (np.abs(DY) * h).sum(axis=0), "dgamma")
    for group in (0, 32, 64, 128):
        q = check_8_bits(t, dtype, group, wy, f"group {group}")
        if R is not None:
            assert torch.equal(q[2], total)
    return y, total, rstd, dx, dg


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,c", [(1, 1), (1, 8), (3, 7), (5, 64), (9, 72), (33, 100), (65, 130), (450, 768), (257, 675), (130, 1024), (70, 1025), (9, 2048),
                                 (7, 2056), (6, 4100), (5, 8192), (3, 9001), (2, 16384)])
def test_shapes(dtype, n, c):
    check(inputs(n, c, dtype, n * 7 + c, residual=n % 2 == 1), dtype, f"{dtype} n={n} C={c}")


@pytest.mark.parametrize("dtype,n,c", [("f32", 1500, 1100), ("f16", 2100, 2056), ("bf16", 1030, 4100), ("f16", 1300, 8200), ("f32", 1100, 8193)])
def test_rows_over_several_waves_in_turn(dtype, n, c):
    # more rows than workgroups: each takes several through the same LDS slots
    check(inputs(n, c, dtype, n + c), dtype, f"{dtype} n={n} C={c}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows(dtype):
    check(inputs(22406, 96, dtype, 5), dtype, f"{dtype} 22406 rows")


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_without_weights(dtype):
    t = inputs(77, 200, dtype, 6, affine=False)
    y, total, rstd, dx, _ = check(t, dtype, f"{dtype} no weights")
    plain, again, none = sc.sparse_rms_norm_forward(t["x"], None, t["residual"], EPS)
    assert none is None and torch.equal(plain, y) and torch.equal(again, total)
    only, g = sc.sparse_rms_norm_backward(t["dy"], total, rstd, None, t["dtotal"], weight_grads=False)
    assert g is None and torch.equal(only, dx)


def test_in_place_reproducible_and_unaligned():
    t = inputs(1000, 333, "bf16", 8)
    y, total, rstd, dx, dg = check(t, "bf16", "reference run")
    again = check(t, "bf16", "again")
    assert all(torch.equal(p, q) for p, q in zip((y, total, rstd, dx, dg), again))
    # total over the residual and y over x, as a residual stream is kept; dx over dtotal
    x, r = t["x"].clone(), t["residual"].clone()
    got = sc.sparse_rms_norm_forward(x, t["gamma"], r, EPS, stats=True, out=x, total=r)
    assert got[0] is x and got[1] is r and torch.equal(x, y) and torch.equal(r, total) and torch.equal(got[2], rstd)
    for over in ("dy", "dtotal"):
        d = {k: t[k].clone() for k in ("dy", "dtotal")}
        sc.sparse_rms_norm_backward(d["dy"], total, rstd, t["gamma"], d["dtotal"], out=d[over])
        assert torch.equal(d[over], dx)
    # rows that start at odd elements, and the other way round: total over x
    shift = lambda a: torch.cat([a.reshape(-1)[:1], a.reshape(-1)])[1:].view(a.shape)  # noqa: E731
    x = shift(t["x"])
    got = sc.sparse_rms_norm_forward(x, shift(t["gamma"]), shift(t["residual"]), EPS, total=x)
    assert torch.equal(got[0], y) and torch.equal(x, total)
    q = sc.sparse_rms_norm_quantize_forward(t["x"], t["gamma"], t["residual"], EPS, group=32, stats=True)
    over = t["residual"].clone()
    p = sc.sparse_rms_norm_quantize_forward(t["x"], shift(t["gamma"]), over, EPS, group=32, total=over)
    assert torch.equal(q[0].view(torch.uint8), p[0].view(torch.uint8)) and torch.equal(q[1], p[1]) and torch.equal(over, total) and torch.equal(q[3], rstd)


@pytest.mark.parametrize("c", [40, 256, 2000, 9000])
def test_nan_infinity_and_zeros_stay_in_their_rows(c):
    t = inputs(6, c, "f32", 9)
    clean = sc.sparse_rms_norm_forward(t["x"], t["gamma"], t["residual"], EPS)[0]
    t["x"][1, 3], t["residual"][2, 5] = float("nan"), float("inf")
    t["x"][4], t["residual"][4] = 0.0, 0.0
    y, _, rstd = sc.sparse_rms_norm_forward(t["x"], t["gamma"], t["residual"], EPS, stats=True)
    assert torch.isnan(y[1]).all() and torch.isnan(y[2, 5]) and rstd[2] == 0 and (y[2, :5] == 0).all() and (y[4] == 0).all()
    keep = [0, 3, 5]
    assert torch.equal(y[keep], clean[keep])
    q, scales, _, _ = sc.sparse_rms_norm_quantize_forward(t["x"], t["gamma"], t["residual"], EPS, group=32)
    assert torch.isnan(q[1].float()).all() and (q[4].float() == 0).all() and (scales[4] == 2.0 ** -126).all() and torch.isfinite(scales).all()
    # a weight that is not a number: its channel alone; an infinite one: its group
    t = inputs(5, c, "f32", 10)
    q, scales, _, _ = sc.sparse_rms_norm_quantize_forward(t["x"], t["gamma"], t["residual"], EPS, group=32)
    t["gamma"][1] = float("nan")
    t["gamma"][33] = float("inf")
    bad, bad_scales, _, _ = sc.sparse_rms_norm_quantize_forward(t["x"], t["gamma"], t["residual"], EPS, group=32)
    assert torch.isnan(bad[:, 1].float()).all() and torch.isnan(bad[:, 33].float()).all() and torch.isinf(bad_scales[:, 1]).all()
    assert not torch.isnan(bad[:, [0, *range(2, 33), *range(34, c)]].float()).any()
    assert torch.equal(bad[:, 64:].view(torch.uint8), q[:, 64:].view(torch.uint8)) and torch.equal(bad_scales[:, 2:], scales[:, 2:])


def test_no_rows():
    x, w = torch.empty(0, 40, device=DEV), torch.ones(40, device=DEV)
    y, total, rstd = sc.sparse_rms_norm_forward(x, w, x, stats=True)
    assert y.shape == total.shape == (0, 40) and rstd.shape == (0,)
    assert sc.sparse_rms_norm_quantize_forward(x, w, group=32)[1].shape == (0, 2)
    dx, dg = sc.sparse_rms_norm_backward(x, x, rstd, w)
    assert dx.shape == (0, 40) and torch.equal(dg, torch.zeros(40, device=DEV))


def test_gradients_against_differences():
    # float32, one direction through x, residual and gamma.  Richardson differences with h = 1/16: 1.5e-5 times a
    # fifth derivative of order 1; float32 outputs summed over 4,000 values and divided by h / 2: about 1e-5.
    t = inputs(20, 200, "f32", 11)
    w = {k: torch.from_numpy(np.random.default_rng(12).standard_normal(t["x"].shape)).to(DEV) for k in ("y", "total")}
    gen = torch.Generator(device="cpu").manual_seed(13)
    dirs = {k: (torch.randn(t[k].shape, generator=gen) * 0.2).to(DEV) for k in ("x", "residual", "gamma")}

    def loss(h):
        y, total, _ = sc.sparse_rms_norm_forward(*(t[k] + h * dirs[k] for k in ("x", "gamma", "residual")), EPS)
        return ((y.double() * w["y"]).sum() + (total.double() * w["total"]).sum()).item()

    _, total, rstd = sc.sparse_rms_norm_forward(t["x"], t["gamma"], t["residual"], EPS, stats=True)
    dx, dg = sc.sparse_rms_norm_backward(w["y"].float(), total, rstd, t["gamma"], w["total"].float())
    slope = sum((g.double() * d).sum().item() for g, d in ((dx, dirs["x"]), (dx, dirs["residual"]), (dg, dirs["gamma"])))
    d = [(loss(h) - loss(-h)) / (2 * h) for h in (1 / 16, 1 / 32)]
    got = (4 * d[1] - d[0]) / 3
    size = sum((g.double() * s).norm().item() for g, s in ((dx, dirs["x"]), (dx, dirs["residual"]), (dg, dirs["gamma"])))
    print(f"  {slope} {got} {size}", flush=True)
    assert abs(slope - got) < 1e-3 * size


@pytest.mark.parametrize("n,c", [(600, 1024), (2000, 333), (40, 9000)])
@pytest.mark.parametrize("group", [0, 32, 128])
def test_8_bits_are_the_quotients(n, c, group):
    # float32, whose y the other call gives as it is: max |y| / 448 and y / scale in float32, rounded to nearest even,
    # bit for bit (a product with the scale's reciprocal moves values next to a tie)
    t = inputs(n, c, "f32", n + c + group)
    y = sc.sparse_rms_norm_forward(t["x"], t["gamma"], t["residual"], EPS)[0].cpu()
    q, scales, _, _ = sc.sparse_rms_norm_quantize_forward(t["x"], t["gamma"], t["residual"], EPS, group=group)
    per = group or c
    parts = torch.nn.functional.pad(y.abs(), (0, -c % per)).reshape(n, -1, per)
    want = parts.amax(2) / torch.tensor(448.0)
    assert torch.equal(scales.cpu(), want)
    wide = want.repeat_interleave(per, 1)[:, :c]
    assert torch.equal(q.cpu().view(torch.uint8), (y / wide).to(torch.float8_e4m3fn).view(torch.uint8))
