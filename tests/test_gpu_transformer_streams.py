"""The scratch memory of the transformer-block operators: many streams, captured graphs, streams that
share a handle."""
import ctypes
import threading

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


PER_THREAD = 2  # hipStreamPerThread: one handle, a stream of its own in every thread


def in_threads(*work):
    """Runs each function in a thread of its own, all at once; raises what one of them raised."""
    errors, start = [], threading.Barrier(len(work))

    def run(f):
        try:
            start.wait(30)
            f()
            assert sc.load_library().hipStreamSynchronize(ctypes.c_void_p(PER_THREAD)) == 0
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(f,)) for f in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    if errors:
        raise errors[0]


def test_threads_on_their_own_streams():
    # scratch memory under the handle that all threads share is not shared
    sets = {}
    for n in (900, 1500):
        (q, k, v, g), step = training_step(n, 4, 64, n)
        x = torch.randn(n, 256, device=DEV)
        _, mean, rstd = sc.sparse_layer_norm_forward(x, stats=True)
        want = [*step(), *sc.sparse_layer_norm_backward(x, x, mean, rstd)[:1]]
        runs = [[torch.empty_like(t) for t in want] for _ in range(12)]
        sets[n] = (q, k, v, g, on_device([n // 3, n - n // 3]), x, mean, rstd, want, runs)
    torch.cuda.synchronize()

    def work(n):
        q, k, v, g, o, x, mean, rstd, want, runs = sets[n]
        for out, lse, dq, dk, dv, dx in runs:
            sc.sparse_attention_forward(q, k, v, o, out=out, lse=lse, stream=PER_THREAD)
            sc.sparse_attention_backward(g, q, k, v, out, lse, o, dq=dq, dk=dk, dv=dv, stream=PER_THREAD)
            sc.sparse_layer_norm_backward(x, x, mean, rstd, weight_grads=False, out=dx, stream=PER_THREAD)

    in_threads(lambda: work(900), lambda: work(1500))
    for *_, want, runs in sets.values():
        for run in runs:
            assert all(torch.equal(a, b) for a, b in zip(run, want))


def test_maps_of_threads_on_their_own_streams():
    # nor are the memory blocks of freed maps
    sets = []
    for key, step in (("2a", 1), ("2a", 2)):
        coords = torch.from_numpy(np.ascontiguousarray(synth.coords_for(key)[::step])).to(DEV)
        feats = torch.randn(coords.shape[0], 64, device=DEV).to(torch.bfloat16)
        weight = (torch.randn(64, 3, 3, 3, 64, device=DEV) / 40).to(torch.bfloat16)
        with sc.sparse_indice_map_build(coords) as m:
            want = sc.subm_conv3d_forward(m, feats, weight)
        sets.append((coords, feats, weight, want, [torch.empty_like(want) for _ in range(12)]))
    torch.cuda.synchronize()

    def work(coords, feats, weight, want, runs):
        for out in runs:
            with sc.sparse_indice_map_build(coords, stream=PER_THREAD) as m:
                sc.subm_conv3d_forward(m, feats, weight, out=out, stream=PER_THREAD)

    in_threads(*(lambda s=s: work(*s) for s in sets))
    for *_, want, runs in sets:
        assert all(torch.equal(run, want) for run in runs)


def conv_case(cout):
    """A set of at least 131,072 rows, 64 input channels: 128 output channels take the neighbour-pool
    kernel, 64 the walk that a second call reorders."""
    gen = torch.Generator(device="cpu").manual_seed(cout)
    coords = torch.from_numpy(synth.coords_for("3a")).to(DEV)
    feats = torch.randn(coords.shape[0], 64, generator=gen).to(torch.bfloat16).to(DEV)
    weight = (torch.randn(cout, 3, 3, 3, 64, generator=gen) / 40).to(torch.bfloat16).to(DEV)
    return coords, feats, weight


def capture(m, feats, weight, stream):
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = sc.subm_conv3d_forward(m, feats, weight)
    return graph, out


def test_a_convolution_is_captured_without_any_call_before(monkeypatch):
    monkeypatch.delenv("SUBMCONV_POOL", raising=False)
    coords, feats, weight = conv_case(128)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s), sc.sparse_indice_map_build(coords) as m:
        graph, captured = capture(m, feats, weight, s)  # neither plan nor packed weights yet
        assert sc.sparse_indice_map_plan_state(m) == sc.SUBM_PLAN_NONE
        monkeypatch.setenv("SUBMCONV_POOL", "0")
        general = sc.subm_conv3d_forward(m, feats, weight)
        monkeypatch.delenv("SUBMCONV_POOL")
        pool = sc.subm_conv3d_forward(m, feats, weight)
        torch.cuda.synchronize()
        assert sc.sparse_indice_map_plan_state(m) == sc.SUBM_PLAN_READY
        warm, captured_pool = capture(m, feats, weight, s)
        for _ in range(3):
            captured.zero_()
            captured_pool.zero_()
            torch.cuda.synchronize()
            graph.replay()
            warm.replay()
            again = sc.subm_conv3d_forward(m, feats, weight)
            torch.cuda.synchronize()
            assert torch.equal(captured, general) and torch.equal(captured_pool, pool) and torch.equal(again, pool)


def test_a_second_call_on_a_map_is_captured():
    coords, feats, weight = conv_case(64)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s), sc.sparse_indice_map_build(coords) as m:
        want = sc.subm_conv3d_forward(m, feats, weight)
        graph, captured = capture(m, feats, weight, s)
        assert sc.sparse_indice_map_row_order_state(m) == sc.SUBM_ORDER_NONE  # left to a later call
        ordered = sc.subm_conv3d_forward(m, feats, weight)
        assert sc.sparse_indice_map_row_order_state(m) != sc.SUBM_ORDER_NONE
        for _ in range(3):
            captured.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(captured, want) and torch.equal(ordered, want)
