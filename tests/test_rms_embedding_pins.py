"""Pins of the oracle of the root-mean-square norm and the embedding (CPU, float64): torch's autograd of the
same definitions, torch's own e4m3 rounding, planted mistakes; and the host side of their C entry points."""
import numpy as np
import pytest
import torch

import submanifold_sparse_convolution_amd as sc
from oracle import transformer_ref as ref

OK, INVALID, UNSUPPORTED = 0, 1, 5


def rel(a, b):
    return np.abs(a - b).max() / max(np.abs(b).max(), 1e-300)


@pytest.mark.parametrize("affine", [True, False])
def test_rms_norm_against_autograd(affine):
    rng = np.random.default_rng(1)
    x, res, dy, dt = rng.standard_normal((4, 7, 13)) + 0.5
    t = [torch.tensor(v, requires_grad=True) for v in (x, res)]
    g = torch.tensor(rng.standard_normal(13), requires_grad=True) if affine else None
    s = t[0] + t[1]
    y = torch.nn.functional.rms_norm(s, (13,), g, 1e-6)
    (y * torch.tensor(dy) + s * torch.tensor(dt)).sum().backward()
    gamma = None if g is None else g.detach().numpy()
    got, total, rstd = ref.rms_norm(x, res, gamma)
    assert rel(got, y.detach().numpy()) < 1e-12
    dx, dg = ref.rms_norm_grad(dy, total, rstd, gamma, dt)
    assert rel(dx, t[0].grad.numpy()) < 1e-11 and rel(dx, t[1].grad.numpy()) < 1e-11
    if affine:
        assert rel(dg, g.grad.numpy()) < 1e-11
    wrong = rstd[:, None] * dy * (1.0 if gamma is None else gamma) + dt  # without the mean
    assert rel(wrong, t[0].grad.numpy()) > 1e-2
    assert rel(ref.layer_norm(x + res, gamma, eps=1e-6)[0], got) > 1e-2  # nor is it the centred norm


def test_e4m3_rounding_and_scales():
    rng = np.random.default_rng(2)
    v = np.concatenate([rng.uniform(-448, 448, 4000), rng.standard_normal(4000) * 0.01, [448.0, -448.0, 0.0, 2.0 ** -10, 1.5 * 2.0 ** -9, 17.0, 19.0]])
    v = v.astype(np.float32).astype(np.float64)
    want = torch.tensor(v).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3(v), want)
    assert np.all(np.abs(ref.e4m3(v) - v) <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10))
    y = rng.standard_normal((3, 75))
    y[1] = 0.0
    s = ref.group_scales(y, 32)
    assert s.shape == (3, 3) and np.all(s[1] == 2.0 ** -126) and s[0, 2] == np.abs(y[0, 64:]).max() / 448
    assert np.array_equal(ref.group_scales(y, 0)[:, 0], np.abs(y).max(axis=1).clip(448 * 2.0 ** -126) / 448)


def test_embedding_against_autograd():
    rng = np.random.default_rng(3)
    tok, table, g = rng.integers(0, 9, 40), rng.standard_normal((11, 5)), rng.standard_normal((40, 5))
    t = torch.tensor(table, requires_grad=True)
    y = 0.3 * torch.nn.functional.embedding(torch.tensor(tok), t)
    (y * torch.tensor(g)).sum().backward()
    assert rel(ref.embedding(table, tok, 0.3), y.detach().numpy()) < 1e-14
    d = ref.embedding_grad(g, tok, 11, 0.3)
    assert rel(d, t.grad.numpy()) < 1e-13 and np.all(d[9:] == 0)
    once = np.zeros_like(d)
    once[tok] = 0.3 * g  # without the sum over equal tokens
    assert rel(once, d) > 1e-2
    out = ref.embedding(table, [2, -1, 11, 3])
    assert np.all(out[1:3] == 0) and np.array_equal(out[3], table[3])
    assert np.array_equal(ref.embedding_grad(g[:2], [-1, 11], 11), np.zeros((11, 5)))


# ------------------------------------------------------------------------- host side of the C ABI

@pytest.fixture(scope="module")
def lib():
    return sc.load_library()


def test_rms_norm_rejects_bad_arguments(lib):
    def fw(x=256, r=None, n=4, c=8, dtype=2, g=None, eps=1e-6, y=512, t=None, rstd=None):
        return lib.sparse_rms_norm_forward(x, r, n, c, dtype, g, eps, y, t, rstd, None)

    assert fw(dtype=3) == UNSUPPORTED and fw(c=16385) == UNSUPPORTED
    assert fw(n=-1) == INVALID and fw(n=2 ** 31) == INVALID and fw(c=0) == INVALID
    assert fw(x=None) == INVALID and fw(y=None) == INVALID
    assert fw(eps=0.0) == INVALID and fw(eps=float("nan")) == INVALID and fw(eps=float("inf")) == INVALID
    assert fw(r=1024) == INVALID and b"total" in lib.subm_last_error()
    assert fw(r=1024, t=512) == INVALID and b"alias" in lib.subm_last_error()
    assert fw(x=257) == INVALID and fw(y=513) == INVALID and fw(r=1025, t=2048) == INVALID and fw(g=3) == INVALID and fw(t=2049) == INVALID
    assert fw(rstd=1026) == INVALID and fw(dtype=0, x=258) == INVALID
    assert fw(n=0, x=None, y=None) == OK

    def q8(x=256, r=None, n=4, c=8, dtype=2, g=None, eps=1e-6, group=32, q=512, s=1024, t=None, rstd=None):
        return lib.sparse_rms_norm_quantize_forward(x, r, n, c, dtype, g, eps, group, q, s, t, rstd, None)

    assert all(q8(group=g) == INVALID for g in (-1, 1, 16, 48, 256))
    assert q8(q=None) == INVALID and q8(s=None) == INVALID and q8(s=1026) == INVALID and q8(dtype=5) == UNSUPPORTED
    assert q8(r=2048) == INVALID and q8(q=256) == INVALID and q8(r=4096, t=8192, q=4096) == INVALID and q8(r=4096, t=8192, q=8192) == INVALID
    assert b"alias" in lib.subm_last_error()
    assert q8(n=0, x=None, q=None, s=None) == OK

    def bw(dy=256, t=512, dt=None, n=4, c=8, dtype=2, g=None, rstd=1024, dx=2048, dg=None):
        return lib.sparse_rms_norm_backward(dy, t, dt, n, c, dtype, g, rstd, dx, dg, None)

    assert bw(dtype=9) == UNSUPPORTED and bw(c=16385) == UNSUPPORTED and bw(n=-1) == INVALID and bw(n=2 ** 31) == INVALID
    assert bw(dy=None) == INVALID and bw(t=None) == INVALID and bw(rstd=None) == INVALID and bw(dx=None) == INVALID
    assert bw(dy=257) == INVALID and bw(t=513) == INVALID and bw(dt=1) == INVALID and bw(rstd=1026) == INVALID and bw(dx=2049) == INVALID and bw(dg=1) == INVALID
    assert bw(dx=512) == INVALID and b"alias" in lib.subm_last_error()
    assert bw(n=0, dy=None, t=None, rstd=None, dx=None) == OK


def test_embedding_rejects_bad_arguments(lib):
    def fw(table=256, rows=10, c=8, dtype=2, tok=512, size=8, n=4, scale=1.0, out=1024):
        return lib.sparse_embedding_forward(table, rows, c, dtype, tok, size, n, scale, out, None)

    def bw(dout=256, rows=10, c=8, dtype=2, tok=512, size=8, n=4, scale=1.0, d=1024):
        return lib.sparse_embedding_backward(dout, rows, c, dtype, tok, size, n, scale, d, None)

    for f in (fw, bw):
        assert f(dtype=3) == UNSUPPORTED and f(rows=2 ** 21 + 1) == UNSUPPORTED and f(c=16385) == UNSUPPORTED
        assert f(rows=0) == INVALID and f(c=0) == INVALID and f(n=-1) == INVALID and f(n=2 ** 31) == INVALID
        assert f(size=2) == INVALID and f(scale=float("inf")) == INVALID and f(scale=float("nan")) == INVALID
        assert f(tok=None) == INVALID and f(tok=516) == INVALID and f(size=4, tok=514) == INVALID
    assert fw(table=None) == INVALID and fw(out=None) == INVALID and fw(table=257) == INVALID and fw(out=256) == INVALID
    assert bw(dout=None) == INVALID and bw(d=None) == INVALID and bw(d=1025) == INVALID and bw(d=256) == INVALID
    assert fw(n=0, table=None, tok=None, out=None) == OK
    assert bw(n=0, d=None) == INVALID


def test_binding_names_the_fault():
    x = torch.zeros(4, 8)
    for call in (lambda: sc.sparse_rms_norm_forward(x), lambda: sc.sparse_rms_norm_quantize_forward(x), lambda: sc.sparse_rms_norm_backward(x, x, x[:, 0]),
                 lambda: sc.sparse_embedding_forward(x, torch.zeros(3, dtype=torch.int64)), lambda: sc.sparse_embedding_backward(x, torch.zeros(4, dtype=torch.int64), 5)):
        with pytest.raises(ValueError):  # CPU tensors
            call()
