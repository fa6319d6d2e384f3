"""GPU parity of the rotary positions against the float64 oracle.

Bound, componentwise: the angle is exact to 2^-24 turns after its reduction in float64, so sine and
cosine are within 2 pi 2^-24 + 2^-23 < 2^-21 and
  |y - ref| <= u |ref| + 2^-20 magnitude (|u| + |v|) + half the smallest subnormal.
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
LAYOUT = {True: sc.SUBM_ROPE_INTERLEAVED, False: sc.SUBM_ROPE_HALF}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    sc.load_library()


def check(x, pos, freq, interleaved, mag, dtype, back=False, out=None):
    call = sc.sparse_rope_backward if back else sc.sparse_rope_forward
    y = call(x, pos, freq, LAYOUT[interleaved], mag, out=out)
    torch.cuda.synchronize()
    X = x.double().cpu().numpy()
    want = ref.rope(X, pos.cpu().numpy(), freq.double().cpu().numpy(), interleaved, mag, back)
    pairs = pos.shape[1] * freq.shape[0]
    size = np.abs(X)
    both = np.zeros_like(size)
    for i in range(pairs):
        u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        both[:, :, u] = both[:, :, v] = size[:, :, u] + size[:, :, v]
    bound = U[dtype] * np.abs(want) + 2.0 ** -20 * abs(mag) * both + (2.0 ** -25 if dtype == "f16" else 0)
    got = y.double().cpu().numpy()
    worst = float((np.abs(got - want) / np.maximum(bound, 1e-300))[..., :2 * pairs].max())
    print(f"  worst error / bound {worst:.3f}", flush=True)
    assert worst <= 1.0
    assert np.array_equal(got[..., 2 * pairs:], X[..., 2 * pairs:])  # the other channels, bit for bit
    return y


def make(n, heads, dim, dtype, seed):
    rng = np.random.default_rng(seed)
    return synth.round_to(rng.standard_normal((n, heads, dim)), dtype).to(DEV), rng


CASES = [  # n, heads, dim, axes, frequencies of an axis
    (1, 1, 2, 1, 1), (1, 3, 64, 3, 10), (450, 16, 64, 3, 10), (7, 5, 80, 1, 40), (33, 2, 96, 3, 16), (100, 20, 128, 1, 48),
    (65, 3, 30, 3, 4), (9, 2, 7, 3, 1), (4, 70, 66, 1, 33), (1000, 1, 40, 2, 10), (3, 2, 4096, 1, 2048),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("case", CASES)
def test_shapes(dtype, interleaved, case):
    n, heads, dim, axes, count = case
    print(dtype, interleaved, case, flush=True)
    x, rng = make(n, heads, dim, dtype, n + dim)
    pos = torch.from_numpy(rng.integers(-40, 512, (n, axes)).astype(np.int32)).to(DEV)
    freq = sc.sparse_rope_frequencies(count)[0].to(DEV)
    y = check(x, pos, freq, interleaved, 1.0, dtype)
    check(y, pos, freq, interleaved, 1.25, dtype, back=True)


MANY = [  # several rows a workgroup (from 2,048 rows), the last one short; 40,001: as many as its sines leave; groups of heads
    (2049, 2, 64, 3, 10), (5003, 3, 40, 1, 20), (70001, 1, 16, 1, 5), (40001, 1, 256, 1, 128), (2, 20, 4096, 1, 100),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("case", MANY)
def test_many_rows_and_heads(dtype, interleaved, case):
    test_shapes(dtype, interleaved, case)


@pytest.mark.parametrize("interleaved", [True, False])
def test_positions_beyond_the_digits_of_float32(interleaved):
    x, _ = make(6, 2, 32, "f32", 3)
    pos = torch.tensor([[0], [-1], [1 << 20], [(1 << 24) + 1], [2 ** 31 - 1], [-2 ** 31]], dtype=torch.int32, device=DEV)
    for scaling in (sc.SUBM_ROPE_PLAIN, sc.SUBM_ROPE_LINEAR, sc.SUBM_ROPE_BASE, sc.SUBM_ROPE_PARTS):
        freq, mag = sc.sparse_rope_frequencies(16, 500000.0, scaling, 8.0, 8192.0)
        check(x, pos, freq.to(DEV), interleaved, mag, "f32")


@pytest.mark.parametrize("interleaved", [True, False])
def test_packed_views_in_place_and_coordinate_columns(interleaved):
    rng = np.random.default_rng(4)
    packed = synth.round_to(rng.standard_normal((300, 24, 64)), "bf16").to(DEV)  # 8 q, 8 k, 8 v heads
    coords = torch.from_numpy(rng.integers(0, 64, (300, 4)).astype(np.int32)).to(DEV)
    freq = sc.sparse_rope_frequencies(10)[0].to(DEV)
    before = packed.clone()
    want = check(packed[:, :16], coords[:, 1:], freq, interleaved, 1.0, "bf16")
    got = sc.sparse_rope_forward(packed[:, :16], coords[:, 1:], freq, LAYOUT[interleaved], out=packed[:, :16])
    assert got.data_ptr() == packed.data_ptr() and torch.equal(packed[:, :16], want)
    assert torch.equal(packed[:, 16:], before[:, 16:])  # values are not touched
    # every second head, rows and heads on odd strides (no 16-byte alignment anywhere)
    odd = torch.empty((300, 17, 67), dtype=torch.bfloat16, device=DEV)
    view = odd[:, 1::2, 1:65]
    view.copy_(before[:, :8])
    check(view, coords[:, 1:], freq, interleaved, 1.0, "bf16", out=torch.zeros_like(odd)[:, ::2, 3:][:, :8])


def test_another_stream_and_refusals():
    x, rng = make(50, 4, 64, "f16", 5)
    pos = torch.from_numpy(rng.integers(0, 99, (50, 1)).astype(np.int32)).to(DEV)
    freq = sc.sparse_rope_frequencies(32)[0].to(DEV)
    want = sc.sparse_rope_forward(x, pos, freq, sc.SUBM_ROPE_HALF)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sc.sparse_rope_forward(x, pos, freq, sc.SUBM_ROPE_HALF, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert sc.sparse_rope_forward(x[:0], pos[:0], freq, sc.SUBM_ROPE_HALF).shape == (0, 4, 64)
    with pytest.raises(sc.SubmError):
        sc.sparse_rope_forward(x, pos, torch.ones(33, device=DEV), sc.SUBM_ROPE_HALF)  # 66 channels of 64
    with pytest.raises(ValueError):
        sc.sparse_rope_forward(x, pos.long(), freq, sc.SUBM_ROPE_HALF)
    with pytest.raises(ValueError):
        sc.sparse_rope_forward(x, pos[:9], freq, sc.SUBM_ROPE_HALF)
    with pytest.raises(ValueError):
        sc.sparse_rope_forward(x.transpose(1, 2), pos, freq, sc.SUBM_ROPE_HALF)
    with pytest.raises(sc.SubmError):
        sc.sparse_rope_forward(x, pos, freq, 2)
    with pytest.raises(sc.SubmError):
        sc.sparse_rope_forward(x, pos, freq, sc.SUBM_ROPE_HALF, out=torch.empty((1, 4, 64), dtype=x.dtype, device=DEV).expand(50, 4, 64))
