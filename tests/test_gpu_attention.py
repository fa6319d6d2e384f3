"""GPU parity of attention within items, forward and backward, against the float64 oracle, with the
componentwise bounds of oracle.transformer_ref.attention_error_bounds.

Roundoffs u: 2^-24, 2^-11, 2^-8 (storage); u_p the same where probabilities are rounded to 16 bits, 0
in float32.  tiny: float16 rounds p <= 1 (forward) to 2^-25 at worst; bfloat16 and float32 have the
exponent range not to.
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


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    sc.load_library()


def f64(t):
    return t.double().cpu().numpy()


def offsets(lens):
    return np.cumsum([0, *lens])


def on_device(o):
    return torch.tensor(np.asarray(o), dtype=torch.int64, device=DEV)


def make(ql, kl, heads, kv_heads, d, dtype, seed, q_scale=1.0, g_scale=0.1):
    rng = np.random.default_rng(seed)
    r = lambda n, h, s: synth.round_to(rng.standard_normal((n, h, d)) * s, dtype).to(DEV)  # noqa: E731
    return r(sum(ql), heads, q_scale), r(sum(kl), kv_heads, 1.0), r(sum(kl), kv_heads, 1.0), r(sum(ql), heads, g_scale)


def within(got, want, bound, what):
    got = f64(got)
    assert got.shape == want.shape, what
    assert np.array_equal(np.isneginf(got), np.isneginf(want)), what
    fin = np.isfinite(want)
    assert np.isfinite(got[fin]).all(), what
    worst = float((np.abs(got[fin] - want[fin]) / np.maximum(bound[fin], 1e-300)).max()) if fin.any() else 0.0
    off = np.linalg.norm(got[fin] - want[fin]) / max(np.linalg.norm(want[fin]), 1e-300)
    print(f"  {what}: worst error / bound {worst:.3f}, relative norm {off:.2e}", flush=True)
    assert worst <= 1.0, what


def check(q, k, v, g, qo, ko, dtype, scale=None, backward=True, outs=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    qd, kd = on_device(qo), on_device(ko)
    out, lse = sc.sparse_attention_forward(q, k, v, qd, kd, scale)
    torch.cuda.synchronize()
    u, u_p = U[dtype], (0.0 if dtype == "f32" else U[dtype])
    want, wlse = ref.attention(f64(q), f64(k), f64(v), qo, ko, scale)
    bounds = ref.attention_error_bounds(f64(q), f64(k), f64(v), qo, ko, scale, u, TINY[dtype], u_p, f64(g) if backward else None)
    within(out, want, bounds[0] + TINY[dtype], "out")
    within(lse, wlse, bounds[1], "lse")
    if not backward:
        return out, lse
    grads = sc.sparse_attention_backward(g, q, k, v, out, lse, qd, kd, scale, *(outs or (None, None, None)))
    torch.cuda.synchronize()
    for name, got, w, b in zip(("dq", "dk", "dv"), grads, ref.attention_grad(f64(g), f64(q), f64(k), f64(v), qo, ko, scale), bounds[2:]):
        within(got, w, b + TINY[dtype], name)
    return (out, lse, *grads)


CASES = [  # query lengths, key lengths (None: the same), heads, key heads, head dim
    ([1], [1], 1, 1, 8),
    ([1], [33], 2, 1, 64),
    ([5, 1, 0, 40], None, 4, 4, 64),
    ([31, 32, 33], None, 3, 1, 32),
    ([127, 0, 129], [64, 65, 0], 2, 2, 128),
    ([128, 256], [63, 1], 4, 2, 96),
    ([300], [577], 6, 3, 40),
    ([450, 1, 587], None, 6, 6, 40),
    ([0, 70, 0, 0, 3], [9, 0, 5, 0, 200], 8, 2, 80),
    ([1, 1, 1, 1, 1], [700, 1, 0, 64, 129], 16, 4, 128),
    ([2, 3, 1], [1500, 10, 333], 12, 1, 64),
    ([17, 90], [1, 2], 2, 2, 120),
    ([600, 200], None, 2, 1, 128),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", CASES)
def test_ragged_items(dtype, case):
    ql, kl, heads, kv_heads, d = case
    kl = ql if kl is None else kl
    print(dtype, case, flush=True)
    check(*make(ql, kl, heads, kv_heads, d, dtype, sum(ql) + d), offsets(ql), offsets(kl), dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", [8, 16, 24, 48, 56, 72, 88, 104, 112])
def test_head_dims(dtype, d):
    check(*make([70, 5], [40, 100], 4, 2, d, dtype, d), offsets([70, 5]), offsets([40, 100]), dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("ql,kl", [([1, 1, 1], [4000, 17, 9001]), ([3, 1], [12000, 5000]), ([40], [6000])])
@pytest.mark.parametrize("heads,kv_heads", [(16, 4), (2, 2)])
def test_few_rows_against_long_caches(dtype, ql, kl, heads, kv_heads):
    print(dtype, ql, kl, heads, kv_heads, flush=True)
    q, k, v, g = make(ql, kl, heads, kv_heads, 128, dtype, 5)
    check(q, k, v, g, offsets(ql), offsets(kl), dtype, backward=False)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_that_grow_and_peak(dtype, d):
    # large scores (a softmax of few keys), growing along the keys so that the running maximum moves in
    # every tile, and a negative scale
    ql, kl = [150, 20], [200, 300]
    q, k, v, g = make(ql, kl, 2, 2, d, dtype, 7, q_scale=3.0)
    ramp = torch.linspace(0.1, 2.0, k.shape[0], device=DEV)[:, None, None]
    check(q, (k * ramp).to(k.dtype), v, g, offsets(ql), offsets(kl), dtype)
    check(q, (k * ramp.flip(0)).to(k.dtype), v, g, offsets(ql), offsets(kl), dtype, scale=-0.2)
    check(q, k, v, g, offsets(ql), offsets(kl), dtype, scale=0.0)


@pytest.mark.parametrize("dtype,ql,kl,heads,kv_heads,d", [
    ("f32", [2100], [2100], 17, 17, 32), ("bf16", [2100], [2100], 29, 29, 128), ("f16", [2100], [2100], 46, 46, 64),
    ("bf16", [900, 300], [2500, 2200], 64, 16, 96), ("f16", [2300], [2060], 30, 30, 120)])
def test_a_few_tiles_past_a_full_machine(dtype, ql, kl, heads, kv_heads, d):
    # the last tiles, those of the last heads, are worked on in parts: the first, a middle and the last
    # key head and their query heads against the oracle
    print(dtype, ql, kl, heads, kv_heads, d, flush=True)
    q, k, v, g = make(ql, kl, heads, kv_heads, d, dtype, 16)
    qo, ko = offsets(ql), offsets(kl)
    qd, kd = on_device(qo), on_device(ko)
    out, lse = sc.sparse_attention_forward(q, k, v, qd, kd)
    grads = sc.sparse_attention_backward(g, q, k, v, out, lse, qd, kd)
    torch.cuda.synchronize()
    group, u_p = heads // kv_heads, 0.0 if dtype == "f32" else U[dtype]
    for h in (0, kv_heads // 2, kv_heads - 1):
        qh, kh = slice(h * group, (h + 1) * group), slice(h, h + 1)
        a = [f64(t) for t in (q[:, qh], k[:, kh], v[:, kh])]
        gh = f64(g[:, qh])
        want = (*ref.attention(*a, qo, ko, d ** -0.5), *ref.attention_grad(gh, *a, qo, ko, d ** -0.5))
        bounds = ref.attention_error_bounds(*a, qo, ko, d ** -0.5, U[dtype], TINY[dtype], u_p, gh)
        got = (out[:, qh], lse[:, qh], grads[0][:, qh], grads[1][:, kh], grads[2][:, kh])
        for name, x, w, b in zip(("out", "lse", "dq", "dk", "dv"), got, want, bounds):
            within(x, w, b + (0.0 if name == "lse" else TINY[dtype]), name)


@pytest.mark.parametrize("g_scale", [1e-6, 1.0, 100.0])
def test_float16_gradients_of_any_size(g_scale):
    # (gradients below the subnormals of float16 cannot come out: dq, dk, dv carry 1e-6 * ... as far
    # as storage allows; the absolute half-subnormal is part of the bound)
    ql = [700, 90]
    check(*make(ql, ql, 2, 1, 64, "f16", 8, g_scale=g_scale), offsets(ql), offsets(ql), "f16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_packed_projections(dtype):
    # q, k, v and their gradients as views of one buffer, heads of different counts
    ql = [130, 0, 75]
    rng = np.random.default_rng(9)
    qkv = synth.round_to(rng.standard_normal((205, 8 + 2 * 2, 64)), dtype).to(DEV)
    g = synth.round_to(rng.standard_normal((205, 8, 64)) * 0.1, dtype).to(DEV)
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    d = torch.full_like(qkv, float("nan"))
    packed = check(q, k, v, g, offsets(ql), offsets(ql), dtype, outs=(d[:, :8], d[:, 8:10], d[:, 10:]))
    assert packed[2].data_ptr() == d.data_ptr() and torch.isfinite(d).all()
    apart = check(q.contiguous(), k.contiguous(), v.contiguous(), g, offsets(ql), offsets(ql), dtype)
    assert all(torch.equal(a, b) for a, b in zip(packed, apart))
    # heads outside tokens: [heads, N, d] storage
    turned = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v, g)]
    other = check(*turned, offsets(ql), offsets(ql), dtype)
    assert all(torch.equal(a, b) for a, b in zip(other, apart))


def test_items_never_meet():
    # NaN and infinity in one item leave every other item's results as they are, bit for bit
    ql, kl = [40, 50, 60], [70, 33, 90]
    q, k, v, g = make(ql, kl, 4, 2, 64, "bf16", 10)
    qo, ko = offsets(ql), offsets(kl)
    clean = check(q, k, v, g, qo, ko, "bf16")
    for t, (a, b) in ((q, (40, 90)), (k, (70, 103)), (v, (70, 103)), (g, (40, 90))):
        t[a:b:2] = float("nan")
        t[a + 1:b:2] = float("inf")
    qd, kd = on_device(qo), on_device(ko)
    out, lse = sc.sparse_attention_forward(q, k, v, qd, kd)
    grads = sc.sparse_attention_backward(g, q, k, v, out, lse, qd, kd)
    for got, want, o in zip((out, lse, *grads), clean, (qo, qo, qo, ko, ko)):
        keep = [*range(o[0], o[1]), *range(o[2], o[3])]
        assert torch.equal(got[keep], want[keep])
    assert torch.isnan(out[40:90]).all()


def test_reproducible_and_on_another_stream():
    ql = [500, 300]
    q, k, v, g = make(ql, ql, 4, 1, 128, "bf16", 11)
    qo = on_device(offsets(ql))
    runs = []
    side = torch.cuda.Stream()
    for stream in (None, None, side):
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        out, lse = sc.sparse_attention_forward(q, k, v, qo, stream=stream)
        runs.append((out, lse, *sc.sparse_attention_backward(g, q, k, v, out, lse, qo, stream=stream)))
    torch.cuda.synchronize()
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


def test_gradients_against_differences():
    # float32, one direction through q, k and v: Richardson differences of steps h and h / 2 have an
    # error of h^4 (h = 1/16: 1.5e-5 times a fifth derivative of order 1), and 2^-22-relative outputs
    # summed over 4096 values and divided by h / 2 about 5e-6: 1e-3 of the slope's scale is wide.
    ql, kl = [60, 4], [50, 80]
    q, k, v, w = make(ql, kl, 2, 1, 32, "f32", 12, g_scale=1.0)
    qo, ko = on_device(offsets(ql)), on_device(offsets(kl))
    gen = torch.Generator(device="cpu").manual_seed(13)
    dirs = [(torch.randn(t.shape, generator=gen) * 0.2).to(DEV) for t in (q, k, v)]

    def loss(h):
        out, _ = sc.sparse_attention_forward(*(t + h * s for t, s in zip((q, k, v), dirs)), qo, ko)
        return (out.double() * w.double()).sum().item()

    out, lse = sc.sparse_attention_forward(q, k, v, qo, ko)
    grads = sc.sparse_attention_backward(w, q, k, v, out, lse, qo, ko)
    slope = sum((a.double() * s.double()).sum().item() for a, s in zip(grads, dirs))
    h = 1.0 / 16
    wide, near = (loss(h) - loss(-h)) / (2 * h), (loss(h / 2) - loss(-h / 2)) / h
    size = sum((a.double().norm() * s.double().norm()).item() for a, s in zip(grads, dirs)) / 10
    print(f"  slope {slope:.6f}, differences {(4 * near - wide) / 3:.6f}, scale {size:.3f}", flush=True)
    assert abs((4 * near - wide) / 3 - slope) <= 1e-3 * max(size, abs(slope))


def test_offsets_that_are_wrong_stay_inside():
    # not an error (they are on the device), but no access may leave the tensors: the ends are clamped
    q, k, v, g = make([64], [64], 2, 2, 64, "bf16", 14)
    for bad in ([0, 1000], [-50, 64], [40, 10], [0, 64]):
        o = on_device(bad)
        out, lse = sc.sparse_attention_forward(q, k, v, o)
        sc.sparse_attention_backward(g, q, k, v, out, lse, o)
    torch.cuda.synchronize()


def test_nothing_to_do():
    e = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    k = torch.randn(7, 2, 64, device=DEV).to(torch.bfloat16)
    out, lse = sc.sparse_attention_forward(e, k, k, on_device([0, 0]), on_device([0, 7]))
    dq, dk, dv = sc.sparse_attention_backward(e, e, k, k, out, lse, on_device([0, 0]), on_device([0, 7]))
    assert out.shape == (0, 2, 64) and not dk.any() and not dv.any()
    out, lse = sc.sparse_attention_forward(k, e, e, on_device([0, 7]), on_device([0, 0]))
    dq, dk, dv = sc.sparse_attention_backward(k, k, e, e, out, lse, on_device([0, 7]), on_device([0, 0]))
    torch.cuda.synchronize()
    assert not out.any() and torch.isneginf(lse).all() and not dq.any() and dk.shape == (0, 2, 64)


def test_refusals():
    q = torch.zeros((8, 4, 64), dtype=torch.float16, device=DEV)
    o = on_device([0, 8])
    for bad in ((q, q[:, :3], q[:, :3]), (q[:, :, :60], q[:, :, :60], q[:, :, :60])):
        with pytest.raises(sc.SubmError):
            sc.sparse_attention_forward(*bad, o)
    for bad in ((q, q.float(), q.float()), (q, q, q[:, :, :32]), (q.transpose(1, 2), q, q), (q, q[:4], q[:4])):
        with pytest.raises(ValueError):
            sc.sparse_attention_forward(*bad, o)
    with pytest.raises(ValueError):
        sc.sparse_attention_forward(q, q, q, o.int())
    with pytest.raises(ValueError):
        sc.sparse_attention_forward(q, q, q, o, on_device([0, 4, 8]))
    with pytest.raises(sc.SubmError):
        sc.sparse_attention_forward(q, q, q, o, out=torch.empty((1, 4, 64), dtype=q.dtype, device=DEV).expand(8, 4, 64))
    with pytest.raises(ValueError):
        sc.sparse_attention_backward(q, q, q, q, q, None, o)


def check_large_values(q, k, v, g, ql, kl):
    """float16 gradients whose score gradients pass its range: the bounds of check, with the roundoff of
    e where its power of two is that of a bound B of 2 |dout|_2 |v|_2, up to 4 times it, with B unit >= 2^14:
    at most 2^-25 / unit <= 2^-39 B <= 2^-36 |dout|_2 |v|_2, |dout|_2 <= sqrt(D) max |dout|."""
    qo, ko, scale = offsets(ql), offsets(kl), q.shape[2] ** -0.5
    qd, kd = on_device(qo), on_device(ko)
    out, lse = sc.sparse_attention_forward(q, k, v, qd, kd, scale)
    grads = sc.sparse_attention_backward(g, q, k, v, out, lse, qd, kd, scale)
    torch.cuda.synchronize()
    a = [f64(t) for t in (q, k, v)]
    tiny = max(TINY["f16"], 2.0 ** -36 * q.shape[2] ** 0.5 * np.linalg.norm(a[2], axis=2).max())
    bounds = ref.attention_error_bounds(*a, qo, ko, scale, U["f16"], tiny, U["f16"], f64(g))[2:]
    for name, got, w, b in zip(("dq", "dk", "dv"), grads, ref.attention_grad(f64(g), *a, qo, ko, scale), bounds):
        assert np.abs(w).max() < 65504, name  # (float16 holds the gradient)
        within(got, w, b + TINY["f16"], name)


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_float16_gradients_against_large_values(sign):
    # two keys with equal scores and opposite values of 3,000: e is 94, 2^10 times that passes 65,504
    full = lambda *rows: torch.tensor(rows, device=DEV).half()[:, None, None].expand(-1, 1, 64).contiguous()  # noqa: E731
    q, k, v, g = full(0.0, 0.0), full(0.5, 0.5 * sign), full(3000.0, -3000.0), full(2.0 ** -10, 2.0 ** -10)
    check_large_values(q, k, v, g, [2], [2])


@pytest.mark.parametrize("heads,kv_heads,d", [(2, 2, 64), (6, 2, 128), (4, 1, 40)])
def test_float16_gradients_of_long_value_rows(heads, kv_heads, d):
    # some rows of v a thousand times the others, items of their own, gradients of any size
    ql, kl = [200, 0, 70, 300], [150, 40, 0, 1100]
    q, k, v, g = make(ql, kl, heads, kv_heads, d, "f16", 17, q_scale=2.0, g_scale=1e-3)
    v[::37] *= 3000
    v[1::74] *= 400
    check_large_values(q, k, v, g, ql, kl)
    check_large_values(q, k, v, g * 2.0 ** -10, ql, kl)


@pytest.mark.parametrize("ql,kl,heads,d", [([1], [60001], 2, 64), ([300], [9000], 2, 64), ([2, 700], [30000, 5000], 3, 128), ([1500], [5000], 16, 128)])
def test_float16_keys_far_below_the_largest(ql, kl, heads, d):
    # one key per item scores 2^25.5 times the others, whose values alone are not zero: their
    # probabilities are scaled by 2^11 at least before float16 rounds them (2^-25 / 2^11 = 2^-36)
    rng = np.random.default_rng(18)
    q, k, v, _ = make(ql, kl, heads, heads, d, "f16", 18)
    v = v.abs()
    q[..., 0], q[..., 1:] = 16.0, 0.0
    k[..., 0], k[..., 1:] = -0.84, 0.0
    qo, ko, scale = offsets(ql), offsets(kl), 0.125
    for b in range(len(kl)):
        top = ko[b] + rng.integers(kl[b])
        k[top, :, 0] = 8.0
        v[top] = 0.0
    out, lse = sc.sparse_attention_forward(q, k, v, on_device(qo), on_device(ko), scale)
    torch.cuda.synchronize()
    few = slice(0, min(q.shape[0], 310))  # (every row is alike)
    a = [f64(q[few]), f64(k), f64(v)]
    qo = np.minimum(qo, few.stop)
    want, wlse = ref.attention(*a, qo, ko, scale)
    bounds = ref.attention_error_bounds(*a, qo, ko, scale, U["f16"], 2.0 ** -36, U["f16"])
    within(out[few], want, bounds[0] + TINY["f16"], "out")
    within(lse[few], wlse, bounds[1], "lse")


# Kernels that the shapes above do not reach, on some heads as in test_a_few_tiles_past_a_full_machine.
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("ql,kl,heads,kv_heads,d", [
    ([1100], [1090], 60, 60, 128), ([700, 500], [1000, 800], 64, 32, 96), ([1100], [1090], 60, 60, 88)])
def test_eight_waves_on_whole_tiles(dtype, ql, kl, heads, kv_heads, d):
    # 96 and 128 channels, at least 256 tiles of 256 rows and of 256 keys, too short to cut the last of them
    test_a_few_tiles_past_a_full_machine(dtype, ql, kl, heads, kv_heads, d)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("ql,kl,heads,kv_heads", [([600], [610], 45, 45), ([300, 0, 130], [700, 40, 1300], 40, 20)])
def test_two_groups_of_waves_on_a_tile(dtype, d, ql, kl, heads, kv_heads):
    # up to 256 tiles of 128 rows, at least 512 keys an item, an odd and an even number of tiles of keys
    test_a_few_tiles_past_a_full_machine(dtype, ql, kl, heads, kv_heads, d)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 96])
@pytest.mark.parametrize("ql,kl", [([1, 1, 1], [4000, 17, 9001]), ([40], [6000])])
def test_keys_in_parts_of_narrow_heads(dtype, d, ql, kl):
    check(*make(ql, kl, 8, 2, d, dtype, 19), offsets(ql), offsets(kl), dtype, backward=False)


@pytest.mark.parametrize("dtype,heads,d", [("f32", 17, 64), ("f32", 17, 80), ("f32", 17, 128), ("f16", 46, 32), ("bf16", 46, 64)])
def test_last_tiles_in_parts(dtype, heads, d):
    test_a_few_tiles_past_a_full_machine(dtype, [2100], [2100], heads, heads, d)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_items_never_meet_in_other_types(dtype):
    # (float16: an item's power of two comes from its own gradients and values)
    ql, kl = [40, 50, 60], [70, 33, 90]
    q, k, v, g = make(ql, kl, 4, 2, 64, dtype, 20)
    qo, ko = offsets(ql), offsets(kl)
    clean = check(q, k, v, g, qo, ko, dtype)
    for t, (a, b) in ((q, (40, 90)), (k, (70, 103)), (v, (70, 103)), (g, (40, 90))):
        t[a:b:2] = float("nan")
        t[a + 1:b:2] = float("inf")
    qd, kd = on_device(qo), on_device(ko)
    out, lse = sc.sparse_attention_forward(q, k, v, qd, kd)
    grads = sc.sparse_attention_backward(g, q, k, v, out, lse, qd, kd)
    for got, want, o in zip((out, lse, *grads), clean, (qo, qo, qo, ko, ko)):
        keep = [*range(o[0], o[1]), *range(o[2], o[3])]
        assert torch.equal(got[keep], want[keep])


def test_offsets_that_are_wrong_stay_inside_in_float16():
    # (the clamps hold for the norms of v and the peaks of dout, too)
    q, k, v, g = make([700], [700], 2, 2, 64, "f16", 21)
    for bad in ([0, 9000, 700], [-50, 300, 700], [600, 10, 40], [0, 700, 700]):
        o = on_device(bad)
        out, lse = sc.sparse_attention_forward(q, k, v, o)
        sc.sparse_attention_backward(g, q, k, v, out, lse, o)
    torch.cuda.synchronize()
