"""GPU parity of the embedding lookup and its gradient against the float64 oracle.

Bounds: the lookup is one product (float32) and one rounding: (u + 2^-24) |out|, u alone in float32.  The
gradient of a row that m tokens name is m float32 additions in some fixed order and a product:
u |d| + (m + 4) 2^-24 scale sum |dout|.  Half the smallest subnormal is added for float16.
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


def within(got, want, bound, what):
    got = f64(got)
    assert got.shape == want.shape and np.isfinite(got).all(), what
    worst = float((np.abs(got - want) / np.maximum(bound, 1e-300)).max()) if got.size else 0.0
    print(f"  {what}: worst error / bound {worst:.3f}", flush=True)
    assert worst <= 1.0, what


def tokens_of(kind, n, rows, rng):
    if kind == "even":
        return rng.integers(0, rows, n)
    if kind == "skewed":
        return np.minimum(np.exp(rng.random(n) * np.log(rows + 1)) - 1, rows - 1).astype(np.int64)
    if kind == "one":
        return np.full(n, rows // 2)
    if kind == "sorted":
        return np.sort(rng.integers(0, rows, n))
    if kind == "padded":  # outside the table on both sides, also far outside
        t = rng.integers(0, rows, n)
        t[::3] = rng.choice([-1, -2 ** 31, rows, rows + 1, 2 ** 31 - 1], len(t[::3]))
        return t
    return np.full(n, -1)  # none


def check(n, c, rows, dtype, kind, bits=64, scale=1.7, seed=0):
    print(f"{dtype} n={n} C={c} rows={rows} {kind}", flush=True)
    rng = np.random.default_rng(seed + n + c + rows)
    tok = tokens_of(kind, n, rows, rng)
    t = torch.from_numpy(tok.astype(np.int64 if bits == 64 else np.int32)).to(DEV)
    table = synth.round_to(rng.standard_normal((rows, c)), dtype).to(DEV)
    dout = synth.round_to(0.1 * rng.standard_normal((n, c)), dtype).to(DEV)
    u, tiny, s = U[dtype], TINY[dtype], float(np.float32(scale))
    out = sc.sparse_embedding_forward(table, t, scale)
    d = sc.sparse_embedding_backward(dout, t, rows, scale, out=torch.full((rows, c), float("nan"), device=DEV, dtype=table.dtype))
    torch.cuda.synchronize()
    there = (tok >= 0) & (tok < rows)
    want = np.where(there[:, None], s * f64(table)[np.where(there, tok, 0)], 0.0)
    within(out, want, (u + (0 if dtype == "f32" else 2.0 ** -24)) * np.abs(want) + tiny, "out")
    wd, mag, count = np.zeros((rows, c)), np.zeros((rows, c)), np.bincount(tok[there], minlength=rows)
    np.add.at(wd, tok[there], s * f64(dout)[there])
    np.add.at(mag, tok[there], s * np.abs(f64(dout)[there]))
    within(d, wd, u * np.abs(wd) + (count[:, None] + 4) * 2.0 ** -24 * mag + np.where(count[:, None] > 0, tiny, 0.0), "dtable")
    assert (d[torch.from_numpy(count == 0).to(DEV)] == 0).all()
    return t, table, dout, out, d


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,c,rows", [(1, 1, 1), (1, 8, 3), (5, 7, 2), (31, 64, 63), (32, 65, 64), (33, 100, 65), (64, 128, 5), (450, 768, 8192), (257, 675, 1021),
                                      (130, 1024, 300), (70, 1030, 17), (65, 2056, 9), (40, 4100, 12), (9, 9001, 30), (4, 16384, 3)])
def test_shapes(dtype, n, c, rows):
    check(n, c, rows, dtype, "even")
    check(n, c, rows, dtype, "padded", bits=32)


@pytest.mark.parametrize("kind", ["even", "skewed", "one", "sorted", "padded", "none"])
@pytest.mark.parametrize("n,c,rows", [(4099, 36, 1021), (8192, 20, 70000), (8193, 20, 70000), (20000, 40, 7), (30001, 136, 2000), (20000, 8, 1)])
def test_distributions(kind, n, c, rows):
    check(n, c, rows, "bf16", kind)


@pytest.mark.parametrize("n,rows", [(1000, 2 ** 21), (600000, 300001), (600000, 3)])
def test_long_lists_and_tables(n, rows):
    check(n, 8, rows, "f32", "skewed")
    check(n, 8, rows, "f16", "even", bits=32)


def test_channels_in_slices():
    check(3000, 2100, 50, "f32", "skewed")
    check(12000, 1100, 600, "bf16", "skewed")


def test_reproducible_unaligned_and_untouched_rows():
    t, table, dout, out, d = check(9000, 75, 333, "bf16", "skewed")
    for _ in range(3):
        assert torch.equal(sc.sparse_embedding_backward(dout, t, 333, 1.7), d)
    shift = lambda a: torch.cat([a.reshape(-1)[:1], a.reshape(-1)])[1:].view(a.shape)  # noqa: E731
    assert torch.equal(sc.sparse_embedding_forward(shift(table), shift(t), 1.7), out)
    buf = torch.full((333 * 75 + 3,), 7.0, device=DEV, dtype=torch.bfloat16)
    sc.sparse_embedding_backward(shift(dout), shift(t), 333, 1.7, out=buf[1:-2].view(333, 75))
    assert torch.equal(buf[1:-2].view(333, 75), d) and buf[0] == 7 and (buf[-2:] == 7).all()


def test_values_behind_padding_do_not_matter():
    # NaN in row 0, which padding must not read into its zeros, and in the gradients of padding
    table, t = torch.randn(5, 16, device=DEV), torch.tensor([1, -1, 3, 5, 1], device=DEV)
    table[0] = float("nan")
    out = sc.sparse_embedding_forward(table, t)
    assert (out[[1, 3]] == 0).all() and torch.equal(out[[0, 2]], table[[1, 3]])
    g = torch.randn(5, 16, device=DEV)
    g[1], g[3] = float("nan"), float("inf")
    d = sc.sparse_embedding_backward(g, t, 5)
    assert torch.isfinite(d).all() and torch.equal(d[1], g[0] + g[4]) and torch.equal(d[3], g[2])
    assert torch.isinf(sc.sparse_embedding_backward(g, torch.tensor([0, 1, 2, 3, 4], device=DEV), 5)[3]).all()


def test_no_tokens():
    t, g = torch.empty(0, dtype=torch.int32, device=DEV), torch.empty(0, 24, device=DEV)
    assert sc.sparse_embedding_forward(torch.ones(4, 24, device=DEV), t).shape == (0, 24)
    assert torch.equal(sc.sparse_embedding_backward(g, t, 100), torch.zeros(100, 24, device=DEV))


def test_against_the_plain_oracle():
    rng = np.random.default_rng(3)
    tok, table, g = rng.integers(-1, 9, 40), rng.standard_normal((8, 6)), rng.standard_normal((40, 6))
    t = torch.from_numpy(tok).to(DEV)
    out = sc.sparse_embedding_forward(torch.from_numpy(table).float().to(DEV), t, 0.5)
    d = sc.sparse_embedding_backward(torch.from_numpy(g).float().to(DEV), t, 8, 0.5)
    # float32 inputs (2^-24), at most 40 additions
    assert np.abs(f64(out) - ref.embedding(table, tok, 0.5)).max() < 1e-6 and np.abs(f64(d) - ref.embedding_grad(g, tok, 8, 0.5)).max() < 1e-5


@pytest.mark.parametrize("n,rows,kind", [(1100000, 2 ** 20 + 5, "even"), (9000, 2 ** 21, "skewed"), (70000, 600000, "padded"), (1100000, 900, "one")])
def test_longest_lists_and_tables(n, rows, kind):
    check(n, 5, rows, "f32", kind)
