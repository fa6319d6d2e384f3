"""Pins of the sliding window's oracle (CPU, float64): torch's autograd of the same definition, a hand-worked
mask, differences, planted mistakes; and the host side of the C entry points."""
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


def test_masks_by_hand():
    # three queries behind two older keys, two keys back, one sink
    want = [[1, 1, 1, 0, 0], [1, 1, 1, 1, 0], [1, 0, 1, 1, 1]]
    assert ref.window_mask(3, 5, 2, 0, 1).astype(int).tolist() == want
    # more queries than keys: the first stand before key 0
    assert ref.window_mask(4, 2, None, 0).astype(int).tolist() == [[0, 0], [0, 0], [1, 0], [1, 1]]
    assert ref.window_mask(4, 2, 0, 1, 2).astype(int).tolist() == [[0, 0], [1, 0], [1, 1], [1, 1]]
    assert ref.window_mask(3, 3).all()


@pytest.mark.parametrize("window", [(None, 0, 0), (2, 0, 1), (1, 2, 0), (0, None, 2), (3, 1, 4)])
def test_against_autograd_and_differences(window):
    rng = np.random.default_rng(3)
    ql, kl = [4, 0, 3, 5], [6, 2, 0, 2]
    q, k, v = rng.standard_normal((12, 4, 5)), *rng.standard_normal((2, 10, 2, 5))
    qo, ko = np.cumsum([0, *ql]), np.cumsum([0, *kl])
    out, lse = ref.window_attention(q, k, v, qo, ko, 0.4, *window)
    t = [torch.tensor(a, requires_grad=True) for a in (q, k, v)]
    seen = torch.zeros(12, 10, dtype=torch.bool)
    for b in range(4):
        seen[qo[b]:qo[b + 1], ko[b]:ko[b + 1]] = torch.from_numpy(ref.window_mask(ql[b], kl[b], *window))
    s = (torch.einsum("ihd,jhd->hij", t[0], t[1].repeat_interleave(2, 1)) * 0.4).masked_fill(~seen, -math.inf)
    some = seen.any(1)
    p = torch.softmax(s[:, some], 2)
    o = torch.einsum("hij,jhd->ihd", p, t[2].repeat_interleave(2, 1))
    assert rel(out[some], o.detach().numpy()) < 1e-12 and np.all(out[~some] == 0)
    assert np.all(np.isneginf(lse[~some])) and rel(lse[some], torch.logsumexp(s[:, some], 2).t().detach().numpy()) < 1e-12
    w = rng.standard_normal(q.shape)
    (o * torch.tensor(w)[some]).sum().backward()
    grads = ref.window_attention_grad(w, q, k, v, qo, ko, 0.4, *window)
    for g, x in zip(grads, t):
        assert rel(g, x.grad.numpy()) < 1e-11
    dirs, e = [rng.standard_normal(a.shape) for a in (q, k, v)], 1e-5
    loss = lambda f: (w * ref.window_attention(q + f * dirs[0], k + f * dirs[1], v + f * dirs[2], qo, ko, 0.4, *window)[0]).sum()  # noqa: E731
    assert abs((loss(e) - loss(-e)) / (2 * e) - sum((g * x).sum() for g, x in zip(grads, dirs))) < 1e-7
    # positions from the first key (not aligned at the last) would be another mask
    if window[1] == 0:
        assert not np.array_equal(ref.window_mask(4, 6, *window), ref.window_mask(6, 6, *window)[:4])


def test_an_open_window_is_the_whole_item_and_lengths_shorten_it():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((7, 2, 5)), *rng.standard_normal((2, 9, 2, 5))
    qo, ko = [0, 3, 7], [0, 4, 9]
    a, b = ref.window_attention(q, k, v, qo, ko, 0.3), ref.attention(q, k, v, qo, ko, 0.3)
    assert rel(a[0], b[0]) < 1e-13 and rel(a[1], b[1]) < 1e-13
    keep = [0, 1, 4, 5, 6]
    short = ref.window_attention(q, k, v, qo, ko, 0.3, 1, 0, 1, k_lengths=[2, 3])
    want = ref.window_attention(q, k[keep], v[keep], qo, [0, 2, 5], 0.3, 1, 0, 1)
    assert np.array_equal(short[0], want[0]) and np.array_equal(short[1], want[1])


# ------------------------------------------------------------------------- host side of the C ABI

@pytest.fixture(scope="module")
def lib():
    return sc.load_library()


def heads(data=256, row=128, head=64):
    return ctypes.byref(sc._binding._HeadsArg(data, row, head))


def test_rejects_bad_arguments(lib):
    def fw(q=None, k=None, v=None, nq=4, nk=4, qo=1024, ko=1024, kn=None, items=1, h=2, kh=2, d=64, dtype=2, scale=0.1, left=3, right=0, sinks=1, out=None, lse=None):
        return lib.sparse_window_attention_forward(q or heads(), k or heads(512), v or heads(768), nq, nk, qo, ko, kn, items, h, kh, d, dtype, scale, left, right, sinks,
                                                   out or heads(2048), lse, None)

    def bw(nq=4, nk=4, qo=1024, ko=1024, items=1, h=2, kh=2, d=64, dtype=2, scale=0.1, left=3, right=0, sinks=1, lse=4096, dq=None, dk=None, dv=None):
        return lib.sparse_window_attention_backward(heads(8192), heads(), heads(512), heads(768), heads(2048), lse, nq, nk, qo, ko, items, h, kh, d, dtype, scale, left, right,
                                                    sinks, dq or heads(16384), dk or heads(32768), dv or heads(65536), None)

    for f in (fw, bw):
        assert f(left=-1) == INVALID and f(right=-1) == INVALID and f(sinks=-1) == INVALID
        assert f(sinks=129) == UNSUPPORTED and b"sinks" in lib.subm_last_error()
        assert f(dtype=3) == UNSUPPORTED and f(d=12) == UNSUPPORTED and f(d=136) == UNSUPPORTED and f(d=0) == INVALID
        assert f(nq=-1) == INVALID and f(nk=2 ** 31) == INVALID and f(items=0) == INVALID and f(items=65536) == INVALID
        assert f(h=3) == INVALID and f(scale=float("inf")) == INVALID and f(qo=None) == INVALID and f(ko=1028) == INVALID
    assert fw(kn=1028) == INVALID and b"k_lengths" in lib.subm_last_error()
    assert fw(q=heads(264)) == UNSUPPORTED and fw(k=heads(None)) == INVALID and fw(out=heads(512)) == INVALID and fw(out=heads(256, 192)) == INVALID
    assert fw(lse=4098) == INVALID and fw(nq=0) == OK
    assert bw(lse=None) == INVALID and bw(dq=heads(256)) == INVALID and bw(dk=heads(16384)) == INVALID and bw(dv=heads(32768)) == INVALID
    assert bw(nq=0, nk=0) == OK


def test_binding_names_the_fault():
    with pytest.raises(ValueError, match="left"):
        sc._binding._window_args(-1, 0, 0)
    with pytest.raises(ValueError, match="right"):
        sc._binding._window_args(0, -2, 0)
    with pytest.raises(ValueError, match="sinks"):
        sc._binding._window_args(0, 0, -2)
    assert sc._binding._window_args(None, 2 ** 70, 3) == (2 ** 31, 2 ** 31, 3)


def test_binding_takes_whole_numbers():
    # a window of 2.5 keys was one of 2
    for bad in ((2.5, 0, 0), (0, 1.0, 0), (None, None, 0.5), (float("inf"), 0, 0), (0, "1", 0)):
        with pytest.raises(TypeError):
            sc._binding._window_args(*bad)
    assert sc._binding._window_args(np.int64(7), torch.tensor(3), np.int32(2)) == (7, 3, 2)
