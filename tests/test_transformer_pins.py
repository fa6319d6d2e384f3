"""Pins of the transformer-block oracle (CPU, float64): torch's autograd of the same definitions,
central differences, invariants and planted mistakes; and the host side of the C entry points."""
import ctypes
import math

import numpy as np
import pytest
import torch

import submanifold_sparse_convolution_amd as sc
from oracle import transformer_ref as ref

OK, INVALID, UNSUPPORTED = 0, 1, 5


def rel(a, b):
    return np.abs(a - b).max() / max(np.abs(b).max(), 1e-300)


@pytest.mark.parametrize("affine", [True, False])
def test_layer_norm_against_autograd(affine):
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((7, 13)) + 3.0, rng.standard_normal((7, 13))
    g, b = (rng.standard_normal(13), rng.standard_normal(13)) if affine else (None, None)
    t = [torch.tensor(v, requires_grad=True) if v is not None else None for v in (x, g, b)]
    y = torch.nn.functional.layer_norm(t[0], (13,), t[1], t[2], 1e-5)
    y.backward(torch.tensor(dy))
    assert rel(ref.layer_norm(x, g, b)[0], y.detach().numpy()) < 1e-12
    dx, dg, db = ref.layer_norm_grad(dy, x, g)
    assert rel(dx, t[0].grad.numpy()) < 1e-11
    if affine:
        assert rel(dg, t[1].grad.numpy()) < 1e-11 and rel(db, t[2].grad.numpy()) < 1e-12
    wrong = ref.layer_norm(x)[2][:, None] * dy * (1.0 if g is None else g)  # without the two means
    assert rel(wrong, t[0].grad.numpy()) > 1e-2


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("axes,count", [(3, 2), (1, 5)])
def test_rope_is_a_rotation_and_its_gradient_the_way_back(interleaved, axes, count):
    rng = np.random.default_rng(2)
    x, pos, f = rng.standard_normal((6, 2, 14)), rng.integers(0, 50, (6, axes)), 10.0 ** -rng.random(count)
    y = ref.rope(x, pos, f, interleaved)
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    assert rel(ref.rope(y, pos, f, interleaved, back=True), x) < 1e-12
    assert np.array_equal(y[..., 2 * axes * count:], x[..., 2 * axes * count:])
    # the gradient of sum(w y) is w turned back: differences in one direction
    w, dx, e = rng.standard_normal(x.shape), rng.standard_normal(x.shape), 1e-6
    slope = (w * (ref.rope(x + e * dx, pos, f, interleaved, 1.3) - ref.rope(x - e * dx, pos, f, interleaved, 1.3))).sum() / (2 * e)
    assert abs(slope - (ref.rope(w, pos, f, interleaved, 1.3, back=True) * dx).sum()) < 1e-7
    # products of two rotated heads depend on the difference of their positions alone
    a, b = x[:1], x[1:2]
    dot = lambda s: (ref.rope(a, pos[:1] + s, f, interleaved) * ref.rope(b, pos[1:2] + s, f, interleaved)).sum()  # noqa: E731
    assert abs(dot(0) - dot(17)) < 1e-10
    assert rel(ref.rope(x, pos, f, not interleaved), y) > 1e-2


def ragged(rng, ql, kl, heads, kv_heads, d):
    q = rng.standard_normal((sum(ql), heads, d))
    k, v = rng.standard_normal((2, sum(kl), kv_heads, d))
    return q, k, v, np.cumsum([0, *ql]), np.cumsum([0, *kl])


def test_attention_against_autograd_and_differences():
    rng = np.random.default_rng(3)
    q, k, v, qo, ko = ragged(rng, [4, 0, 3, 5], [6, 2, 0, 1], 4, 2, 5)
    out, lse = ref.attention(q, k, v, qo, ko, 0.4)
    assert np.all(out[4:7] == 0) and np.all(lse[4:7] == -np.inf)  # the item without keys
    t = [torch.tensor(a, requires_grad=True) for a in (q, k, v)]
    s = torch.einsum("ihd,jhd->hij", t[0], t[1].repeat_interleave(2, 1)) * 0.4
    item = lambda o: torch.tensor(np.searchsorted(o[1:], np.arange(o[-1]), side="right"))  # noqa: E731
    s = s.masked_fill(item(qo)[:, None] != item(ko)[None, :], -math.inf)
    p = torch.nan_to_num(torch.softmax(s, 2))
    o = torch.einsum("hij,jhd->ihd", p, t[2].repeat_interleave(2, 1))
    assert rel(out, o.detach().numpy()) < 1e-12
    w = rng.standard_normal(q.shape)
    grads = ref.attention_grad(w, q, k, v, qo, ko, 0.4)
    dirs, e = [rng.standard_normal(a.shape) for a in (q, k, v)], 1e-5
    loss = lambda f: (w * ref.attention(q + f * dirs[0], k + f * dirs[1], v + f * dirs[2], qo, ko, 0.4)[0]).sum()  # noqa: E731
    assert abs((loss(e) - loss(-e)) / (2 * e) - sum((g * x).sum() for g, x in zip(grads, dirs))) < 1e-7
    # a key item without queries gets no gradient, and the planted mistake (no row sum) is seen
    assert np.all(grads[1][6:8] == 0) and np.all(grads[2][6:8] == 0)
    a, b = slice(0, 4), slice(0, 6)
    pr, _ = ref._probabilities(q[a, 0], k[b, 0], 0.4)
    assert rel(0.4 * pr * (w[a, 0] @ v[b, 0].T) @ k[b, 0], grads[0][a, 0]) > 1e-2


# ------------------------------------------------------------------------- host side of the C ABI

@pytest.fixture(scope="module")
def lib():
    return sc.load_library()


def test_frequencies():
    f, m = sc.sparse_rope_frequencies(10, 10000.0)
    assert m == 1.0 and np.allclose(f.numpy(), 10000.0 ** (-np.arange(10) / 10), rtol=1e-7)
    lin, _ = sc.sparse_rope_frequencies(10, 10000.0, sc.SUBM_ROPE_LINEAR, 4.0)
    assert np.allclose(lin.numpy() * 4, f.numpy(), rtol=1e-6)
    big, _ = sc.sparse_rope_frequencies(10, 10000.0, sc.SUBM_ROPE_BASE, 4.0)
    assert big[0] == 1.0 and abs(big[9] * 4 / f[9] - 1) < 1e-6
    parts, m = sc.sparse_rope_frequencies(64, 10000.0, sc.SUBM_ROPE_PARTS, 4.0, 4096.0)
    full, _ = sc.sparse_rope_frequencies(64, 10000.0)
    turns = 4096.0 * full.numpy() / (2 * math.pi)
    ratio = parts.numpy() / full.numpy()
    assert abs(m - (0.1 * math.log(4.0) + 1.0)) < 1e-6
    assert np.allclose(ratio[turns > 32], 1.0) and np.allclose(ratio[turns < 1], 0.25)
    assert np.all(np.diff(ratio) <= 1e-6)
    one, _ = sc.sparse_rope_frequencies(1, 10000.0, sc.SUBM_ROPE_BASE, 4.0)
    assert one[0] == 1.0
    for bad in (dict(count=0), dict(base=1.0), dict(base=math.inf), dict(scaling=4), dict(factor=0.5), dict(factor=math.nan),
                dict(scaling=sc.SUBM_ROPE_PARTS, trained_length=0.0)):
        with pytest.raises(sc.SubmError):
            sc.sparse_rope_frequencies(**{"count": 4, **bad})


def test_layer_norm_rejects_bad_arguments(lib):
    def fw(x=256, n=4, c=8, dtype=2, g=None, b=None, eps=1e-5, y=512, mean=None, rstd=None):
        return lib.sparse_layer_norm_forward(x, n, c, dtype, g, b, eps, y, mean, rstd, None)

    assert fw(dtype=3) == UNSUPPORTED and fw(c=16385) == UNSUPPORTED
    for bad in (dict(n=-1), dict(n=2 ** 31), dict(c=0), dict(eps=0.0), dict(eps=math.nan), dict(eps=math.inf), dict(mean=1024),
                dict(x=None), dict(y=None), dict(x=257), dict(g=1025), dict(mean=1026, rstd=2048)):
        assert fw(**bad) == INVALID, bad
    assert fw(n=0, x=None, y=None) == OK

    def bw(dy=256, x=512, n=4, c=8, dtype=0, g=None, mean=1024, rstd=2048, dx=4096, dg=None, db=None):
        return lib.sparse_layer_norm_backward(dy, x, n, c, dtype, g, mean, rstd, dx, dg, db, None)

    assert bw(dtype=-1) == UNSUPPORTED and bw(c=16385) == UNSUPPORTED
    for bad in (dict(n=-1), dict(c=0), dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(dx=None), dict(dg=8192),
                dict(dy=258), dict(dg=8193, db=9000)):
        assert bw(**bad) == INVALID, bad
    assert bw(n=0, dy=None, x=None, mean=None, rstd=None, dx=None) == OK


def heads(p=4096, row=64, head=16):
    from submanifold_sparse_convolution_amd._binding import _HeadsArg
    return ctypes.byref(_HeadsArg(p, row, head))


@pytest.mark.parametrize("name", ["sparse_rope_forward", "sparse_rope_backward"])
def test_rope_rejects_bad_arguments(lib, name):
    def f(x=heads(), n=4, h=4, d=16, dtype=2, pos=256, stride=3, axes=3, freq=512, count=2, layout=0, mag=1.0, y=heads(8192)):
        return getattr(lib, name)(x, n, h, d, dtype, pos, stride, axes, freq, count, layout, mag, y, None)

    assert f(dtype=7) == UNSUPPORTED
    for bad in (dict(n=-1), dict(n=2 ** 31), dict(h=0), dict(h=65536), dict(d=0), dict(d=4097), dict(axes=0), dict(count=0), dict(count=3),
                dict(layout=2), dict(mag=math.nan), dict(x=None), dict(y=None), dict(x=heads(None)), dict(pos=None), dict(freq=None),
                dict(x=heads(4097)), dict(pos=258), dict(y=heads(4096, 128, 16)), dict(y=heads(8192, 0, 16)), dict(y=heads(8192, 64, 0))):
        assert f(**bad) == INVALID, bad
    assert f(n=0, x=None, y=None, pos=None, freq=None) == OK


def test_attention_rejects_bad_arguments(lib):
    def fw(q=heads(), k=heads(), v=heads(), nq=4, nk=4, qo=256, ko=512, items=1, h=4, kh=4, d=16, dtype=2, scale=0.25, out=heads(8192), lse=None):
        return lib.sparse_attention_forward(q, k, v, nq, nk, qo, ko, items, h, kh, d, dtype, scale, out, lse, None)

    def bw(g=heads(), q=heads(), k=heads(), v=heads(), o=heads(), lse=1024, nq=4, nk=4, qo=256, ko=512, items=1, h=4, kh=4, d=16, dtype=2,
           scale=0.25, dq=heads(8192), dk=heads(12288), dv=heads(16384)):
        return lib.sparse_attention_backward(g, q, k, v, o, lse, nq, nk, qo, ko, items, h, kh, d, dtype, scale, dq, dk, dv, None)

    for f, out in ((fw, "out"), (bw, "dk")):
        for bad in (dict(dtype=3), dict(d=12), dict(d=136), dict(q=heads(4100)), dict(k=heads(4096, 60, 16)), dict(v=heads(4096, 64, 12)),
                    dict(q=heads(4096, 2 ** 22, 16)), dict(k=heads(4096, -64, 16))):
            assert f(**bad) == UNSUPPORTED, bad
        for bad in (dict(nq=-1), dict(nk=2 ** 31), dict(items=0), dict(items=65536), dict(h=0), dict(kh=3), dict(kh=0), dict(d=0), dict(scale=math.inf),
                    dict(scale=math.nan), dict(qo=None), dict(ko=None), dict(qo=260), dict(q=None), dict(k=heads(None)), dict(lse=1026),
                    dict(nq=2 ** 29), {out: heads(8192, 0, 16)}, {out: heads(8192, 64, 0)}):
            assert f(**bad) == INVALID, bad
        assert b"" != lib.subm_last_error()
    assert bw(lse=None) == INVALID
    assert fw(nq=0, q=heads(None), out=heads(None)) == OK
    assert bw(nq=0, nk=0, lse=None) == OK


def test_attention_rows_stay_within_32_bits(lib):
    # (no queries: what passes the checks launches nothing)
    most = 2 ** 31 - 2 ** 24

    def fw(nq, nk, h=1):
        return lib.sparse_attention_forward(heads(), heads(4096, 0, 16), heads(4096, 0, 16), nq, nk, 256, 512, 1, h, 1, 16, 2, 0.25,
                                            heads(8192), None, None)

    assert fw(0, most) == OK
    assert fw(0, most + 1) == INVALID and fw(0, 2 ** 31 - 1) == INVALID
    assert fw(most + 1, 1) == INVALID and fw(most // 64 + 1, 1, 64) == INVALID


def test_attention_over_the_queries_needs_their_strides(lib):
    def fw(out, nq=4, h=4):  # (no device: what passes the checks fails to launch)
        return lib.sparse_attention_forward(heads(), heads(8192), heads(12288), nq, 4, 256, 512, 1, h, h, 16, 2, 0.25, out, None, None)

    assert fw(heads(4096, 128, 16)) == INVALID and fw(heads(4096, 64, 32)) == INVALID
    assert b"strides" in lib.subm_last_error()
    if not torch.cuda.is_available():
        for same in (fw(heads()), fw(heads(4096, 128, 16), nq=1), fw(heads(4096, 64, 32), h=1)):
            assert same not in (OK, INVALID)


def test_binding_checks_before_calling():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        sc.sparse_layer_norm_forward(x)
    with pytest.raises(ValueError):
        sc.sparse_rope_forward(torch.zeros(4, 2, 8), torch.zeros(4, 1, dtype=torch.int32), torch.ones(2), sc.SUBM_ROPE_HALF)
    with pytest.raises(ValueError):
        sc.sparse_attention_forward(torch.zeros(4, 2, 8), torch.zeros(4, 2, 8), torch.zeros(4, 2, 8), torch.tensor([0, 4]))
