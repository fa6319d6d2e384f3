"""The scratch memory of the transformer-block operators: many streams, captured graphs, streams that
share a handle."""
import ctypes

import numpy as np
import pytest
import torch

import submanifold_sparse_convolution_amd as sc
import synth

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    sc.load_library()


def on_device(lens):
    return torch.tensor(np.cumsum([0, *lens]), dtype=torch.int64, device=DEV)


def training_step(n, heads, d, seed, dtype="bf16"):
    """A call that keeps partial results in scratch memory: inputs, and the step itself."""
    rng = np.random.default_rng(seed)
    q, k, v, g = (synth.round_to(rng.standard_normal((n, heads, d)), dtype).to(DEV) for _ in range(4))
    offsets = on_device([n // 3, n - n // 3])

    def step():
        out, lse = sc.sparse_attention_forward(q, k, v, offsets)
        return [out, lse, *sc.sparse_attention_backward(g, q, k, v, out, lse, offsets)]

    return (q, k, v, g), step


def test_a_graph_outlives_the_scratch_of_many_streams():
    # a captured call keeps its scratch memory however many streams ask for some afterwards
    inputs, step = training_step(600, 4, 64, 1)
    home = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(home):
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=home):
            captured = step()
    x = torch.randn(300, 640, device=DEV)
    _, mean, rstd = sc.sparse_layer_norm_forward(x, stats=True)
    torch.cuda.synchronize()
    others, handles = [], set()
    while len(handles) < 24:  # (torch hands out 32 streams in turn)
        s = torch.cuda.Stream()
        if s.cuda_stream != home.cuda_stream:
            handles.add(s.cuda_stream)
            others.append(s)
    norms = [sc.sparse_layer_norm_backward(x, x, mean, rstd, stream=s) for s in others]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for run in norms[1:] for a, b in zip(run, norms[0]))
    with torch.cuda.stream(home):
        for round_ in range(3):
            for z in inputs:
                z.copy_(torch.randn(z.shape, device=DEV))
            eager = [e.clone() for e in step()]
            norms = [sc.sparse_layer_norm_backward(x, x, mean, rstd, stream=s) for s in others]
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(captured, eager)), round_


def test_a_graph_replays_beside_its_stream():
    # the graph's scratch memory is not that of eager calls on the stream it was captured on: both may run at once
    inputs, step = training_step(1500, 4, 64, 2)
    home, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(home):
        want = [e.clone() for e in step()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=home):
            captured = step()
    rows, eager_step = training_step(1400, 4, 64, 3)
    eager_want = [e.clone() for e in eager_step()]
    torch.cuda.synchronize()
    for round_ in range(10):
        with torch.cuda.stream(home):
            eager = [eager_step() for _ in range(3)]
        with torch.cuda.stream(other):
            for _ in range(3):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, want)), round_
        for run in eager:
            assert all(torch.equal(a, b) for a, b in zip(run, eager_want)), round_


def pool_used():
    """Bytes of the device's memory pool in use (the library's stream-ordered allocations)."""
    hip = sc.load_library()  # (its dependencies resolve through it)
    pool, used = ctypes.c_void_p(), ctypes.c_uint64()
    assert hip.hipDeviceGetDefaultMemPool(ctypes.byref(pool), ctypes.c_int(0)) == 0
    assert hip.hipMemPoolGetAttribute(pool, ctypes.c_int(0x7), ctypes.byref(used)) == 0  # hipMemPoolAttrUsedMemCurrent
    return used.value


def test_scratch_memory_is_that_of_the_largest_call():
    sc.subm_release_cached_memory()
    base, sizes = pool_used(), (1000, 1700, 2500, 4000, 6000, 9000)
    for n in sizes:  # the backward pass keeps two floats a query row and head, 64 heads of 8: 512 n bytes, whole tiles
        inputs, step = training_step(n, 64, 8, 4)
        step()
        torch.cuda.synchronize()
    held = pool_used() - base
    sc.subm_release_cached_memory()
    alone = training_step(sizes[-1], 64, 8, 4)[1]
    before = pool_used()
    alone()
    torch.cuda.synchronize()
    print(f"  after {sizes} queries {held} bytes, after the last alone {pool_used() - before}", flush=True)
    assert held == pool_used() - before
