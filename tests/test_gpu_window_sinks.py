"""Gradients of windows with sinks over thousands of items of several heads, and the scratch memory that they take:
float32 sums of dk and dv of each chunk of rows (an item has one at least) for the sinks that there are."""
import ctypes

import numpy as np
import pytest
import torch

import submanifold_sparse_convolution_amd as sc
import synth
from oracle import transformer_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f16": 2.0 ** -25, "bf16": 0.0}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    sc.load_library()


def pool_used():
    """Bytes of the device's memory pool in use (the library's stream-ordered allocations)."""
    hip = sc.load_library()  # (its dependencies resolve through it)
    pool, used = ctypes.c_void_p(), ctypes.c_uint64()
    assert hip.hipDeviceGetDefaultMemPool(ctypes.byref(pool), ctypes.c_int(0)) == 0
    assert hip.hipMemPoolGetAttribute(pool, ctypes.c_int(0x7), ctypes.byref(used)) == 0  # hipMemPoolAttrUsedMemCurrent
    return used.value


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dtype,sinks", [("bf16", 4), ("f16", 4), ("bf16", 33), ("bf16", 1)])
def test_thousands_of_items(dtype, sinks):
    items, heads, d = 2500, 16, 128
    rng = np.random.default_rng(sinks)
    lens = rng.integers(0, 13, items)
    lens[100] = 700  # (several chunks)
    o = np.cumsum([0, *lens])
    n = int(o[-1])
    q, k, v, g = (synth.round_to(rng.standard_normal((n, heads, d)) * s, dtype).to(DEV) for s in (1.0, 1.0, 1.0, 0.1))
    od, window = torch.from_numpy(o).to(DEV), (3, 0, sinks)
    out, lse = sc.sparse_window_attention_forward(q, k, v, od, None, *window)
    torch.cuda.synchronize()
    sc.subm_release_cached_memory()
    before = pool_used()
    grads = sc.sparse_window_attention_backward(g, q, k, v, out, lse, od, None, *window)
    torch.cuda.synchronize()
    held = pool_used() - before
    # chunks of 128 rows at least, dk and dv of each sink; beside them at most 32 bytes a row and head
    most = (n // 128 + items) * heads * sinks * 2 * d * 4 + 32 * n * heads + (4 << 20)
    print(f"  {held} bytes of scratch memory, at most {most}", flush=True)
    assert held <= most
    scale, u_p = d ** -0.5, U[dtype]
    for h in (0, 7, 15):
        a = [f64(t[:, h:h + 1]) for t in (q, k, v)]
        gh = f64(g[:, h:h + 1])
        want = ref.window_attention_grad(gh, *a, o, o, scale, *window)
        bounds = ref.window_attention_error_bounds(*a, o, o, scale, U[dtype], TINY[dtype], u_p, gh, *window)[2:]
        for x, w, b, name in zip(grads, want, bounds, ("dq", "dk", "dv")):
            assert (np.abs(f64(x[:, h:h + 1]) - w) <= b + TINY[dtype]).all(), (h, name)
