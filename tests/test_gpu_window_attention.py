"""GPU parity of attention within a sliding window, forward and backward, against the float64 oracle, with
the componentwise bounds of oracle.transformer_ref.window_attention_error_bounds (derived there; roundoffs u:
2^-24, 2^-11, 2^-8, u_p the same where probabilities are rounded to 16 bits, tiny: float16's half subnormal of
scaled probabilities)."""
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
    print(f"  {what}: worst error / bound {worst:.3f}", flush=True)
    assert worst <= 1.0, what


def check(q, k, v, g, qo, ko, dtype, window, scale=None, backward=True, lengths=None, heads=None):
    """Parity of a call; `heads`: key heads to compare (default all)."""
    scale = q.shape[2] ** -0.5 if scale is None else scale
    qd, kd = on_device(qo), on_device(ko)
    left, right, sinks = window
    kl = None if lengths is None else on_device(lengths)
    out, lse = sc.sparse_window_attention_forward(q, k, v, qd, kd, left, right, sinks, kl, scale)
    grads = sc.sparse_window_attention_backward(g, q, k, v, out, lse, qd, kd, left, right, sinks, scale) if backward else ()
    torch.cuda.synchronize()
    group, u_p = q.shape[1] // k.shape[1], 0.0 if dtype == "f32" else U[dtype]
    for h in range(k.shape[1]) if heads is None else heads:
        qh, kh = slice(h * group, (h + 1) * group), slice(h, h + 1)
        a = [f64(t) for t in (q[:, qh], k[:, kh], v[:, kh])]
        gh = f64(g[:, qh]) if backward else None
        want = ref.window_attention(*a, qo, ko, scale, *window, k_lengths=lengths)
        bounds = ref.window_attention_error_bounds(*a, qo, ko, scale, U[dtype], TINY[dtype], u_p, gh, *window, k_lengths=lengths)
        got = [out[:, qh], lse[:, qh]]
        if backward:
            want = (*want, *ref.window_attention_grad(gh, *a, qo, ko, scale, *window))
            got += [grads[0][:, qh], grads[1][:, kh], grads[2][:, kh]]
        for name, x, w, b in zip(("out", "lse", "dq", "dk", "dv"), got, want, bounds):
            within(x, w, b + (0.0 if name == "lse" else TINY[dtype]), f"head {h} {name}")
    return (out, lse, *grads)


WINDOWS = [(None, 0, 0), (None, None, 0), (0, 0, 0), (31, 0, 0), (64, 0, 4), (100, 7, 1), (5, 200, 40), (None, 3, 9), (0, None, 0), (17, None, 33), (130, 0, 128), (3, 0, 64)]

CASES = [  # query lengths, key lengths (None: the same), heads, key heads, head dim
    ([1], [1], 1, 1, 8),
    ([5, 1, 0, 40], None, 4, 4, 64),
    ([31, 32, 33], None, 3, 1, 32),
    ([127, 0, 129], [64, 65, 0], 2, 2, 128),   # more queries than keys: the first see nothing before p + right = 0
    ([300], [577], 6, 3, 40),
    ([1, 1, 1, 1, 1], [700, 1, 0, 64, 129], 16, 4, 128),
    ([2, 3, 1], [1500, 10, 333], 12, 1, 64),
    ([450, 1, 287], None, 2, 2, 96),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("window", WINDOWS)
@pytest.mark.parametrize("case", CASES)
def test_ragged_items(dtype, case, window):
    ql, kl, heads, kv_heads, d = case
    kl = ql if kl is None else kl
    print(dtype, case, window, flush=True)
    check(*make(ql, kl, heads, kv_heads, d, dtype, sum(ql) + d), offsets(ql), offsets(kl), dtype, window, heads=[0, kv_heads - 1])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", [8, 16, 24, 48, 56, 72, 88, 104, 112, 120])
def test_head_dims(dtype, d):
    check(*make([170, 5], [190, 100], 4, 2, d, dtype, d), offsets([170, 5]), offsets([190, 100]), dtype, (40, 3, 2))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("ql,kl", [([1, 1, 1], [4000, 17, 9001]), ([3, 1], [12000, 5000]), ([40], [6000])])
@pytest.mark.parametrize("window", [(4095, 0, 4), (500, 0, 0), (None, 0, 0), (2000, 0, 128)])
def test_few_rows_against_long_caches(dtype, ql, kl, window):
    print(dtype, ql, kl, window, flush=True)
    q, k, v, g = make(ql, kl, 8, 2, 128, dtype, 5)
    check(q, k, v, g, offsets(ql), offsets(kl), dtype, window, backward=False)


@pytest.mark.parametrize("dtype,ql,kl,heads,kv_heads,d,window", [
    ("bf16", [2100], [2100], 29, 29, 128, (700, 0, 4)), ("f16", [2100], [2100], 46, 46, 64, (None, 0, 0)), ("bf16", [900, 300], [2500, 2200], 64, 16, 96, (1000, 100, 50)),
    ("f16", [2300], [2300], 30, 30, 120, (511, 512, 8)), ("bf16", [4000], [4000], 4, 2, 128, (1023, 0, 4)), ("bf16", [2500, 1500], [2500, 1500], 3, 3, 64, (None, 0, 0)),
    ("f32", [2100], [2100], 17, 17, 32, (300, 0, 2)), ("bf16", [3000], [3000], 16, 16, 128, (None, 0, 0)), ("f16", [1700], [1700], 1, 1, 64, (200, 0, 4))])
def test_machines_full_of_tiles(dtype, ql, kl, heads, kv_heads, d, window):
    # eight waves a tile, tiles in parts, two groups of waves a tile: the first, a middle and the last key head
    print(dtype, ql, kl, heads, kv_heads, d, window, flush=True)
    check(*make(ql, kl, heads, kv_heads, d, dtype, 16), offsets(ql), offsets(kl), dtype, window, heads=sorted({0, kv_heads // 2, kv_heads - 1}))


@pytest.mark.parametrize("items", [63, 64, 65, 130, 4500])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_items(dtype, items):
    # the search through the offsets goes 64 items at a time
    rng = np.random.default_rng(items)
    kl = rng.integers(0, 9, items)
    ql = np.minimum(rng.integers(0, 4, items), kl + 1)
    q, k, v, g = make([int(ql.sum())], [int(kl.sum())], 2, 1, 32, dtype, items)
    check(q, k, v, g, offsets(ql), offsets(kl), dtype, (3, 0, 1))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_open_windows_are_the_whole_item(dtype):
    ql, kl = [70, 3, 200], [90, 3, 180]
    q, k, v, g = make(ql, kl, 4, 2, 64, dtype, 3)
    qd, kd = on_device(offsets(ql)), on_device(offsets(kl))
    want = sc.sparse_attention_forward(q, k, v, qd, kd)
    for left, right in ((None, None), (10 ** 6, 2 ** 40)):
        got = sc.sparse_window_attention_forward(q, k, v, qd, kd, left, right)
        # the same sums in another order of tiles at most
        assert torch.allclose(got[0].float(), want[0].float(), atol=2 * U[dtype], rtol=4 * U[dtype]) and torch.allclose(got[1], want[1], atol=1e-5, rtol=1e-6)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_that_grow_and_peak(dtype, d):
    ql = [250, 20]
    q, k, v, g = make(ql, ql, 2, 2, d, dtype, 7, q_scale=3.0)
    ramp = torch.linspace(0.1, 2.0, k.shape[0], device=DEV)[:, None, None]
    o = offsets(ql)
    check(q, (k * ramp).to(k.dtype), v, g, o, o, dtype, (60, 0, 3))
    check(q, (k * ramp.flip(0)).to(k.dtype), v, g, o, o, dtype, (60, 5, 3), scale=-0.2)
    check(q, k, v, g, o, o, dtype, (33, 0, 0), scale=0.0)


def test_keys_of_a_hidden_range_may_be_the_largest():
    # the lowest score of all is the one that is seen, and hidden ones are far above it
    q, k, v, g = make([200], [200], 2, 2, 64, "f32", 8)
    k[:100] = 30.0 * q[150, :, :]
    check(q, k, v, g, [0, 200], [0, 200], "f32", (20, 0, 0))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lengths", [[0, 5, 70, 64], [100, 1, 3, 90], [-3, 10 ** 12, 64, 0]])
def test_caches_with_room_behind(dtype, lengths):
    # rows past an item's length hold NaN and are not read
    ql, kl = [1, 2, 30, 1], [100, 40, 130, 90]
    q, k, v, g = make(ql, kl, 4, 2, 64, dtype, 9)
    ko, n = offsets(kl), np.clip(lengths, 0, kl)
    for b in range(4):
        k[ko[b] + n[b]:ko[b + 1]] = float("nan")
        v[ko[b] + n[b]:ko[b + 1]] = float("inf")
    kz, vz = torch.nan_to_num(k, nan=0.0), torch.nan_to_num(v, posinf=0.0)
    got = [sc.sparse_window_attention_forward(q, a, b, on_device(offsets(ql)), on_device(ko), 50, 0, 4, on_device(lengths)) for a, b in ((k, v), (kz, vz))]
    assert all(torch.equal(a, b) for a, b in zip(*got))
    check(q, kz, vz, g, offsets(ql), ko, dtype, (50, 0, 4), lengths=n, backward=False)


HIDDEN = [((40, 0, 0), 300), ((40, 0, 4), 300), ((None, 0, 0), 300), ((30, 20, 10), 150)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("window,n", HIDDEN)
@pytest.mark.parametrize("d", [40, 128])
def test_hidden_values_do_not_matter(dtype, window, n, d):
    # keys and values that are not finite change the rows that see them and no others, and gradients that are
    # not finite no keys that their rows do not see
    heads, kv_heads = 4, 2
    q, k, v, g = make([n], [n], heads, kv_heads, d, dtype, 10)
    o = on_device([0, n])
    seen = ref.window_mask(n, n, *window)
    fw = lambda *t: sc.sparse_window_attention_forward(*t, o, o, *window)  # noqa: E731
    bw = lambda *t: sc.sparse_window_attention_backward(*t, o, o, *window)  # noqa: E731
    want = fw(q, k, v)
    grads = bw(g, q, k, v, *want)
    # rows of tiles that met such a value are computed in another way, within the bounds of any evaluation
    scale, u_p = d ** -0.5, 0.0 if dtype == "f32" else U[dtype]
    a = [f64(x) for x in (q, k, v)]
    oracle = (*ref.window_attention(*a, [0, n], [0, n], scale, *window), *ref.window_attention_grad(f64(g), *a, [0, n], [0, n], scale, *window))
    bounds = ref.window_attention_error_bounds(*a, [0, n], [0, n], scale, U[dtype], TINY[dtype], u_p, f64(g), *window)

    def near(got, which, keep, what):
        within(got[torch.from_numpy(keep).to(DEV)], oracle[which][keep], bounds[which][keep] + TINY[dtype], what)

    for j, x, y in ((n // 2, float("nan"), float("inf")), (2, -float("inf"), float("nan")), (n - 1, 1.0, float("nan")), (n // 3, 1.0, float("inf"))):
        kb, vb = k.clone(), v.clone()
        kb[j, :, 3] *= x
        vb[j, :, 5] = y
        got = fw(q, kb, vb)
        sees = seen[:, j]
        assert not torch.isfinite(got[0][torch.from_numpy(sees).to(DEV)][:, :, 5]).any()
        near(got[0], 0, ~sees, f"key {j} out")
        assert torch.equal(got[1][torch.from_numpy(~sees).to(DEV)], want[1][torch.from_numpy(~sees).to(DEV)])
        back = bw(g, q, kb, vb, *got)
        near(back[0], 2, ~sees, "dq")
        hit = seen[sees].any(axis=0)  # keys that a row that sees it sees
        near(back[1], 3, ~hit, "dk")
        near(back[2], 4, ~hit, "dv")
    for i in (0, n // 2, n - 1):
        gb = g.clone()
        gb[i, :, 1], gb[i, :, 2] = float("nan"), float("inf")
        back = bw(gb, q, k, v, *want)
        rows = torch.arange(n, device=DEV) != i
        assert torch.equal(back[0][rows], grads[0][rows])
        near(back[1], 3, ~seen[i], f"row {i} dk")
        near(back[2], 4, ~seen[i], "dv")
        assert not torch.isfinite(back[2][torch.from_numpy(seen[i]).to(DEV)][:, :, 1:3]).any()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [(40, 0, 4), (None, 0, 0), (700, 0, 4)])
def test_hidden_values_beside_few_rows(dtype, d, window):
    # a few tokens after long caches, whose older keys and values hold anything
    ql, kl = [5, 1, 8], [900, 2100, 64]
    q, k, v, g = make(ql, kl, 4, 1, d, dtype, 14)
    qo, ko = offsets(ql), offsets(kl)
    for b in range(3):
        last = ref.window_mask(ql[b], kl[b], *window)
        for j in np.flatnonzero(~last.all(axis=0)):  # some row does not see it
            if not last[:, j].any() or last[:, j].sum() < ql[b] and j % 2:
                k[ko[b] + j, :, 1], v[ko[b] + j, :, 2] = float("nan"), float("inf")
    out, lse = sc.sparse_window_attention_forward(q, k, v, on_device(qo), on_device(ko), *window)
    a = [f64(t) for t in (q, k, v)]
    clean = [a[0], np.nan_to_num(a[1], nan=0.0), np.nan_to_num(a[2], posinf=0.0)]
    want, wlse = ref.window_attention(*clean, qo, ko, d ** -0.5, *window)
    bound, blse = ref.window_attention_error_bounds(*clean, qo, ko, d ** -0.5, U[dtype], TINY[dtype], 0.0 if dtype == "f32" else U[dtype], None, *window)
    odd = ~np.isfinite(a[2]).all(axis=(1, 2))
    for b in range(3):
        seen = ref.window_mask(ql[b], kl[b], *window)
        for i in range(ql[b]):
            row = slice(qo[b] + i, qo[b] + i + 1)
            if (seen[i] & odd[ko[b]:ko[b + 1]]).any():
                assert not torch.isfinite(out[row]).all()
            else:
                within(out[row], want[row], bound[row] + TINY[dtype], f"item {b} row {i} out")
                within(lse[row], wlse[row], blse[row], "lse")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_packed_projections(dtype):
    # q, k, v and their gradients as views of one buffer; heads outside tokens
    ql = [230, 0, 75]
    rng = np.random.default_rng(9)
    qkv = synth.round_to(rng.standard_normal((305, 8 + 2 * 2, 64)), dtype).to(DEV)
    g = synth.round_to(rng.standard_normal((305, 8, 64)) * 0.1, dtype).to(DEV)
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    o, window = offsets(ql), (50, 0, 5)
    apart = check(q.contiguous(), k.contiguous(), v.contiguous(), g, o, o, dtype, window)
    d = torch.full_like(qkv, float("nan"))
    od = on_device(o)
    out, lse = sc.sparse_window_attention_forward(q, k, v, od, None, *window)
    sc.sparse_window_attention_backward(g, q, k, v, out, lse, od, None, *window, dq=d[:, :8], dk=d[:, 8:10], dv=d[:, 10:])
    assert torch.equal(out, apart[0]) and torch.equal(d, torch.cat(apart[2:], 1))
    turned = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v, g)]
    assert all(torch.equal(a, b) for a, b in zip(check(*turned, o, o, dtype, window), apart))
    over = q.contiguous()
    assert torch.equal(sc.sparse_window_attention_forward(over, k, v, od, None, *window, out=over)[0], apart[0])


def test_items_never_meet():
    ql, kl = [40, 50, 60], [70, 33, 90]
    q, k, v, g = make(ql, kl, 4, 2, 64, "bf16", 10)
    qo, ko, window = offsets(ql), offsets(kl), (30, 4, 3)
    clean = check(q, k, v, g, qo, ko, "bf16", window)
    for t, (a, b) in ((q, (40, 90)), (k, (70, 103)), (v, (70, 103)), (g, (40, 90))):
        t[a:b:2] = float("nan")
        t[a + 1:b:2] = float("inf")
    qd, kd = on_device(qo), on_device(ko)
    out, lse = sc.sparse_window_attention_forward(q, k, v, qd, kd, *window)
    grads = sc.sparse_window_attention_backward(g, q, k, v, out, lse, qd, kd, *window)
    for got, want, o in zip((out, lse, *grads), clean, (qo, qo, qo, ko, ko)):
        keep = [*range(o[0], o[1]), *range(o[2], o[3])]
        assert torch.equal(got[keep], want[keep])


def test_reproducible_and_on_another_stream():
    ql = [500, 300]
    q, k, v, g = make(ql, ql, 4, 1, 128, "bf16", 11)
    qo = on_device(offsets(ql))
    runs = []
    side = torch.cuda.Stream()
    for stream in (None, None, side):
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        out, lse = sc.sparse_window_attention_forward(q, k, v, qo, None, 100, 0, 4, stream=stream)
        runs.append((out, lse, *sc.sparse_window_attention_backward(g, q, k, v, out, lse, qo, None, 100, 0, 4, stream=stream)))
    torch.cuda.synchronize()
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


def test_offsets_that_are_wrong_stay_inside():
    # unspecified numbers, no access outside (guards around every tensor stay as they were)
    n, h, d = 200, 2, 64
    buf = torch.full((3, n + 64, h, d), 7.0, device=DEV)
    q, k, v = (torch.randn(n, h, d, device=DEV) for _ in range(3))
    out, dk = buf[0, 32:-32], buf[1, 32:-32]
    for bad in ([0, 10 ** 12], [-5, 150], [180, 20], [0, 90]):
        o = on_device(bad)
        _, lse = sc.sparse_window_attention_forward(q, k, v, o, None, 40, 0, 4, out=out)
        sc.sparse_window_attention_backward(q, q, k, v, out.clone(), lse, o, None, 40, 0, 4, dk=dk)
    torch.cuda.synchronize()
    assert all((b[:32] == 7).all() and (b[-32:] == 7).all() for b in buf[:2])


def test_gradients_against_differences():
    # float32, one direction through q, k and v: Richardson differences of steps h and h / 2 have an
    # error of h^4 (h = 1/16: 1.5e-5 times a fifth derivative of order 1), and 2^-22-relative outputs
    # summed over 4096 values and divided by h / 2 about 5e-6: 1e-3 of the slope's scale is wide.
    ql, kl, window = [60, 4], [60, 80], (20, 2, 3)
    q, k, v, w = make(ql, kl, 2, 1, 32, "f32", 12, g_scale=1.0)
    qo, ko = on_device(offsets(ql)), on_device(offsets(kl))
    gen = torch.Generator(device="cpu").manual_seed(13)
    dirs = [(torch.randn(t.shape, generator=gen) * 0.2).to(DEV) for t in (q, k, v)]

    def loss(h):
        out, _ = sc.sparse_window_attention_forward(*(t + h * s for t, s in zip((q, k, v), dirs)), qo, ko, *window)
        return (out.double() * w.double()).sum().item()

    out, lse = sc.sparse_window_attention_forward(q, k, v, qo, ko, *window)
    grads = sc.sparse_window_attention_backward(w, q, k, v, out, lse, qo, ko, *window)
    slope = sum((g.double() * s.double()).sum().item() for g, s in zip(grads, dirs))
    size = sum((g.double() * s.double()).norm().item() for g, s in zip(grads, dirs))
    d = [(loss(h) - loss(-h)) / (2 * h) for h in (1 / 16, 1 / 32)]
    print(f"  {slope} {(4 * d[1] - d[0]) / 3} {size}", flush=True)
    assert abs(slope - (4 * d[1] - d[0]) / 3) < 1e-3 * size


def test_no_rows():
    q, k = torch.empty(0, 2, 64, device=DEV), torch.ones(5, 2, 64, device=DEV)
    oq, ok = on_device([0, 0]), on_device([0, 5])
    out, lse = sc.sparse_window_attention_forward(q, k, k, oq, ok, 3, 0, 2)
    assert out.shape == (0, 2, 64)
    dq, dk, dv = sc.sparse_window_attention_backward(q, q, k, k, out, lse, oq, ok, 3, 0, 2)
    assert torch.equal(dk, torch.zeros_like(k)) and torch.equal(dv, dk)
    out, lse = sc.sparse_window_attention_forward(k, q, q, ok, oq, 3, 0, 2)
    assert torch.equal(out, torch.zeros_like(k)) and torch.isneginf(lse).all()
    dq, dk, dv = sc.sparse_window_attention_backward(k, k, q, q, out, lse, ok, oq, 3, 0, 2)
    assert torch.equal(dq, torch.zeros_like(k)) and dk.shape == (0, 2, 64)


@pytest.mark.parametrize("window", [(255, 0, 4), (None, 0, 0), (100, 100, 0)])
@pytest.mark.parametrize("bad", ["all", "v", "dout", "q"])
def test_values_that_are_not_finite_everywhere(bad, window):
    # where something non-finite is seen the results are, elsewhere they are what clean inputs give; the rows
    # beside what is hidden are computed again, which many of them must not do over all that they see
    n, heads, d = 2000, 2, 64
    rng = np.random.default_rng(15)
    q, k, v, g = (synth.round_to(rng.standard_normal((n, heads, d)), "bf16").to(DEV) for _ in range(4))
    o = on_device([0, n])
    clean_out, clean_lse = sc.sparse_window_attention_forward(q, k, v, o, None, *window)
    clean = sc.sparse_window_attention_backward(g, q, k, v, clean_out, clean_lse, o, None, *window)
    at = np.zeros(n, dtype=bool)
    at[::1 if bad == "all" else 301] = True
    where = torch.from_numpy(at).to(DEV)
    mask = ref.window_mask(n, n, *window)
    rows_hit, keys_hit = mask[:, at].any(1), mask[at].any(0)
    seen_by_hit = mask[rows_hit].any(0)
    for t in {"all": (q, k, v, g), "v": (v,), "dout": (g,), "q": (q,)}[bad]:
        t[where, :, ::7] = float("nan") if bad != "v" else float("inf")
    out, lse = sc.sparse_window_attention_forward(q, k, v, o, None, *window)
    dq, dk, dv = sc.sparse_window_attention_backward(g, q, k, v, out, lse, o, None, *window)
    odd = {"all": (rows_hit, rows_hit, seen_by_hit, seen_by_hit), "v": (rows_hit, rows_hit, seen_by_hit, ~seen_by_hit & False),
           "dout": (~rows_hit & False, at, keys_hit, keys_hit), "q": (at, at, keys_hit, keys_hit)}[bad]
    for got, want, hit, what in zip((out, dq, dk, dv), (clean_out, *clean), odd, ("out", "dq", "dk", "dv")):
        finite = torch.isfinite(got).all(2).all(1).cpu().numpy()
        assert np.array_equal(finite, ~hit), what
        rows = torch.from_numpy(~hit).to(DEV)
        near = np.abs(f64(got[rows]) - f64(want[rows])) <= 2 ** -6 * np.abs(f64(want[rows])).max(initial=1.0)  # (each is its clean value to roundings of 2^-8)
        assert near.all(), what


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("window", [(20, 0, 3), (None, 0, 0), (40, 11, 70)])
@pytest.mark.parametrize("heads", [128, 7])
def test_many_heads_a_key_head(dtype, window, heads):
    ql, kl = [1, 3, 40, 0], [300, 5, 40, 9]
    q, k, v, g = make(ql, kl, heads, 1, 16, dtype, 16)
    check(q, k, v, g, offsets(ql), offsets(kl), dtype, window)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.5])
@pytest.mark.parametrize("ql,kl", [([200, 3], [200, 90]), ([2, 1], [900, 400])])
def test_scales(dtype, scale, ql, kl):
    q, k, v, g = make(ql, kl, 2, 2, 48, dtype, 17)
    check(q, k, v, g, offsets(ql), offsets(kl), dtype, (50, 0, 5), scale=scale)
