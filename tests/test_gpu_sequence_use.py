"""The root-mean-square norm, embedding and sliding-window operators as a program uses them: differentiated
through torch, captured in graphs, on several streams and from threads, single tokens after a prompt, and the
sequence example."""
import ctypes
import importlib.util
import math
import os
import threading

import numpy as np
import pytest
import torch

import submanifold_sparse_convolution_amd as sc
import synth
from oracle import transformer_ref as ref
from submanifold_sparse_convolution_amd import autograd as sa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PER_THREAD = 2  # hipStreamPerThread: one handle, a stream of its own in every thread


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    sc.load_library()


def leaf(rng, *shape):
    return synth.round_to(rng.standard_normal(shape), "f32").to(DEV).requires_grad_()


def f64(t):
    return t.detach().double().cpu().numpy()


def near(got, want, what):
    # float32 chains of four operators with sums of at most 128 terms: 512 * 2^-23 < 1e-4 of the norm
    off = np.linalg.norm(f64(got) - want) / np.linalg.norm(want)
    print(f"  {what}: {off:.2e}", flush=True)
    assert off < 1e-4, what


def test_block_gradients_through_autograd():
    rng = np.random.default_rng(0)
    n, heads, d, rows = 90, 4, 16, 20
    offsets, window = [0, 50, 50, 90], (12, 0, 3)
    off = torch.tensor(offsets, device=DEV)
    tok = torch.from_numpy(rng.integers(-1, rows, n)).to(DEV)
    table, g1, g2 = leaf(rng, rows, heads * d), leaf(rng, heads * d), leaf(rng, heads * d)
    k, v = leaf(rng, n, heads // 2, d), leaf(rng, n, heads, d)
    wy, ws = (torch.from_numpy(rng.standard_normal((n, heads * d))).float().to(DEV) for _ in range(2))
    x = sa.embedding(table, tok, 0.7)
    q = sa.rms_norm(x, g1).view(n, heads, d)
    a = sa.window_attention(q, k, v[:, ::2], off, None, *window)
    y, s = sa.rms_norm(a.reshape(n, heads * d), g2, residual=x)
    (y * wy + s * ws).sum().backward()

    scale = d ** -0.5
    X = ref.embedding(f64(table), f64(tok).astype(int), 0.7)
    Q, _, r1 = ref.rms_norm(X, None, f64(g1))
    args = (Q.reshape(n, heads, d), f64(k), f64(v)[:, ::2], offsets, offsets, scale)
    A = ref.window_attention(*args, *window)[0].reshape(n, -1)
    Y, S, r2 = ref.rms_norm(A, X, f64(g2))
    near(y, Y, "y")
    near(s, S, "sum")
    ds, dg2 = ref.rms_norm_grad(f64(wy), S, r2, f64(g2), f64(ws))
    dq, dk, dv = ref.window_attention_grad(ds.reshape(n, heads, d), *args, *window)
    dx, dg1 = ref.rms_norm_grad(dq.reshape(n, -1), X, r1, f64(g1))
    near(g2.grad, dg2, "dgamma2")
    near(k.grad, dk, "dk")
    near(v.grad[:, ::2], dv, "dv")
    near(g1.grad, dg1, "dgamma1")
    near(table.grad, ref.embedding_grad(dx + ds, f64(tok).astype(int), rows, 0.7), "dtable")


def test_partial_gradients():
    rng = np.random.default_rng(1)
    x, r, g = leaf(rng, 20, 24), leaf(rng, 20, 24), leaf(rng, 24)
    _, s = sa.rms_norm(x, g, residual=r)  # the sum alone
    (3.0 * s).sum().backward()
    assert torch.equal(x.grad, torch.full_like(x, 3.0)) and torch.equal(r.grad, x.grad) and g.grad is None
    x.grad = r.grad = None
    y, _ = sa.rms_norm(x.detach(), g, residual=r)
    y.sum().backward()
    both = r.grad.clone()
    assert x.grad is None and g.grad is not None
    r.grad = None
    y, _ = sa.rms_norm(x, g.detach(), residual=r.detach())
    y.sum().backward()
    assert torch.equal(x.grad, both) and r.grad is None
    x.grad = None
    (sa.rms_norm(x).sum() + sa.rms_norm(x, g).sum()).backward()  # one leaf through two calls
    assert torch.isfinite(x.grad).all()
    x.grad = r.grad = None
    y, s = sa.rms_norm(x, g, residual=x)  # the same tensor twice
    y.sum().backward()
    twice = x.grad.clone()
    x.grad = None
    z = sa.rms_norm(2.0 * x, g)
    z.sum().backward()
    assert torch.allclose(twice, x.grad, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_that_start_anywhere(dtype):
    # the gradient of a part of a concatenation is a view of the whole one, at an odd element
    rng = np.random.default_rng(4)
    n, heads, d = 40, 2, 16
    off = torch.tensor([0, 15, 40], device=DEV)
    tok = torch.from_numpy(rng.integers(0, n, n)).to(DEV)
    x, gamma = (leaf(rng, *shape).detach().to(dtype).requires_grad_() for shape in ((n, heads * d), (heads * d,)))
    w = leaf(rng, 1 + n * heads * d).detach().to(dtype)
    grads = []
    for front in (1, 0):
        for f in (lambda: sa.rms_norm(x, gamma), lambda: sa.rms_norm(x, gamma, residual=x)[1], lambda: sa.embedding(x, tok, 2.0),
                  lambda: sa.window_attention(*[x.view(n, heads, d)] * 3, off, None, 5, 0, 2)):
            x.grad = None
            y = f().reshape(-1)
            y = torch.cat([y[:1].detach(), y]) if front else y
            (y * w[1 - front:]).sum().backward()
            grads.append(x.grad)
    assert all(torch.equal(a, b) for a, b in zip(grads[:4], grads[4:]))


def steps(seed, n=600, dtype="bf16"):
    """Inputs that change between runs, and a run of every entry point over them."""
    rng = np.random.default_rng(seed)
    heads, d, rows = 4, 64, 3000
    t = lambda *shape: synth.round_to(rng.standard_normal(shape), dtype).to(DEV)  # noqa: E731
    x, r, gamma, dy, q, k, v, g = t(n, 256), t(n, 256), t(256), t(n, 256), t(n, heads, d), t(n, heads, d), t(n, heads, d), t(n, heads, d)
    off = torch.tensor([0, n // 3, n], device=DEV)
    one, caches, ko = t(2, heads, d), t(8000, heads, d), torch.tensor([0, 3000, 8000], device=DEV)
    oo, lengths = torch.tensor([0, 1, 2], device=DEV), torch.tensor([2500, 5000], device=DEV)
    tok, many = torch.from_numpy(rng.integers(-1, rows, n)).to(DEV), torch.from_numpy(rng.integers(0, rows, 10000)).to(DEV)
    table, dout = t(rows, 96), t(10000, 96)

    def step():
        y, total, rstd = sc.sparse_rms_norm_forward(x, gamma, r, stats=True)
        grads = sc.sparse_rms_norm_backward(dy, total, rstd, gamma, dy)
        q8, scales, _, _ = sc.sparse_rms_norm_quantize_forward(x, gamma, r, group=64)
        e = sc.sparse_embedding_forward(table, tok, 2.0)
        de = [sc.sparse_embedding_backward(dout, many, rows), sc.sparse_embedding_backward(dout[:n], tok, rows)]
        out, lse = sc.sparse_window_attention_forward(q, k, v, off, None, 100, 0, 4)
        back = sc.sparse_window_attention_backward(g, q, k, v, out, lse, off, None, 100, 0, 4)
        causal = sc.sparse_window_attention_forward(q, k, v, off, None, None, 0)
        few = sc.sparse_window_attention_forward(one, caches, caches, oo, ko, 2000, 0, 4, lengths)
        return [y, total, rstd, *grads, q8.view(torch.uint8), scales, e, *de, out, lse, *back, *causal, *few]

    return (x, r, dy, q, k, v, g, one, dout), step


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_captured_in_a_graph(dtype):
    inputs, step = steps(2, dtype=dtype)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        step()  # the stream's scratch memory grows here, not under capture
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            captured = step()
        for round_ in range(4):
            for z in inputs:
                z.copy_(torch.randn(z.shape, device=DEV))
            eager = [e.clone() for e in step()]
            if round_ == 1:  # a larger call on the stream: what the graph holds must stay
                sc.sparse_embedding_backward(torch.randn(200000, 96, device=DEV), torch.randint(0, 50, (200000,), device=DEV), 50)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(captured, eager)), round_


def test_a_graph_replays_beside_its_stream():
    _, step = steps(3)
    home, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(home):
        want = [e.clone() for e in step()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=home):
            captured = step()
    _, eager_step = steps(4, n=500)
    eager_want = [e.clone() for e in eager_step()]
    torch.cuda.synchronize()
    for round_ in range(6):
        with torch.cuda.stream(home):
            eager = [eager_step() for _ in range(2)]
        with torch.cuda.stream(other):
            for _ in range(2):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, want)), round_
        for run in eager:
            assert all(torch.equal(a, b) for a, b in zip(run, eager_want)), round_


def test_scratch_cannot_grow_under_capture():
    x, tok, o = torch.randn(64, 2, 64, device=DEV), torch.randint(0, 9, (64,), device=DEV), torch.tensor([0, 64], device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    m = x.view(64, 128)
    out, lse = sc.sparse_window_attention_forward(x, x, x, o, None, 10, 0)
    _, _, rstd = sc.sparse_rms_norm_forward(m, stats=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y = x + 1.0
        for call in (lambda: sc.sparse_window_attention_backward(x, x, x, x, out, lse, o, None, 10, 0), lambda: sc.sparse_embedding_backward(m, tok, 9),
                     lambda: sc.sparse_rms_norm_backward(m, m, rstd)):
            with pytest.raises(sc.SubmError) as e:
                call()
            assert e.value.name == "SUBM_ERR_UNSUPPORTED" and "capture" in e.value.detail
        z = sc.sparse_rms_norm_forward(m)[0]  # (needs none)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, x + 1.0) and torch.equal(z, sc.sparse_rms_norm_forward(m)[0])


def in_threads(*work):
    errors, start = [], threading.Barrier(len(work))

    def run(f):
        try:
            start.wait(30)
            f()
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


def test_two_threads_on_one_stream():
    sets = [steps(5, n=300)[1], steps(6, n=900)[1]]
    want = [[e.clone() for e in s()] for s in sets]
    torch.cuda.synchronize()
    side, got = torch.cuda.Stream(), [[], []]

    def loop(i):
        with torch.cuda.stream(side):
            for _ in range(10):
                got[i].append(sets[i]())

    in_threads(lambda: loop(0), lambda: loop(1))
    for w, runs in zip(want, got):
        for run in runs:
            assert all(torch.equal(a, b) for a, b in zip(run, w))


def test_threads_on_their_own_streams():
    # scratch memory under the handle that all threads share is not shared
    sets = []
    for n in (900, 1500):
        rng = np.random.default_rng(n)
        q = synth.round_to(rng.standard_normal((n, 4, 64)), "bf16").to(DEV)
        off, tok = torch.tensor([0, n], device=DEV), torch.from_numpy(rng.integers(0, 500, n)).to(DEV)
        x = q.reshape(n, 256)
        out, lse = sc.sparse_window_attention_forward(q, q, q, off, None, 50, 0, 4)
        want = [out, lse, *sc.sparse_window_attention_backward(q, q, q, q, out, lse, off, None, 50, 0, 4), sc.sparse_embedding_backward(x, tok, 500)]
        sets.append((q, off, tok, x, want, [[torch.empty_like(t) for t in want] for _ in range(8)]))
    torch.cuda.synchronize()

    def work(q, off, tok, x, want, runs):
        for out, lse, dq, dk, dv, dt in runs:
            sc.sparse_window_attention_forward(q, q, q, off, None, 50, 0, 4, out=out, lse=lse, stream=PER_THREAD)
            sc.sparse_window_attention_backward(q, q, q, q, out, lse, off, None, 50, 0, 4, dq=dq, dk=dk, dv=dv, stream=PER_THREAD)
            sc.sparse_embedding_backward(x, tok, 500, out=dt, stream=PER_THREAD)
        assert sc.load_library().hipStreamSynchronize(ctypes.c_void_p(PER_THREAD)) == 0

    in_threads(*(lambda s=s: work(*s) for s in sets))
    for *_, want, runs in sets:
        for run in runs:
            assert all(torch.equal(a, b) for a, b in zip(run, want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tokens_after_a_prompt(dtype):
    # a prompt at once, in chunks, and token by token into caches with room: the same rows within the
    # roundings of the oracle's bounds
    rng = np.random.default_rng(7)
    lens, room, window, heads, kv_heads, d = [70, 33], 100, (20, 0, 3), 8, 2, 32
    u = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}[dtype]
    t = lambda n, h: synth.round_to(rng.standard_normal((n, h, d)), dtype).to(DEV)  # noqa: E731
    q, k, v = t(sum(lens), heads), t(sum(lens), kv_heads), t(sum(lens), kv_heads)
    o = np.cumsum([0, *lens])
    od = torch.tensor(o, device=DEV)
    a = [f64(x) for x in (q, k, v)]
    want, wlse = ref.window_attention(*a, o, o, d ** -0.5, *window)
    bound, blse = ref.window_attention_error_bounds(*a, o, o, d ** -0.5, u, 0.0, 0.0 if dtype == "f32" else u, None, *window)

    def check(got, rows, lse):
        assert (np.abs(f64(got) - want[rows]) <= bound[rows]).all() and (np.abs(f64(lse) - wlse[rows]) <= blse[rows]).all()

    check(*[sc.sparse_window_attention_forward(q, k, v, od, None, *window)[0], slice(None), sc.sparse_window_attention_forward(q, k, v, od, None, *window)[1]])
    kc, vc = (torch.full((2 * room, kv_heads, d), float("nan"), device=DEV, dtype=q.dtype) for _ in range(2))
    ko = torch.tensor([0, room, 2 * room], device=DEV)
    done = np.array([0, 0])
    for chunk in ([30, 7], [10, 1], [1, 1], [1, 0], [1, 20], [27, 4]):
        rows = np.concatenate([np.arange(o[b] + done[b], o[b] + done[b] + chunk[b]) for b in range(2)])
        for b in range(2):
            new = slice(o[b] + done[b], o[b] + done[b] + chunk[b])
            at = slice(b * room + done[b], b * room + done[b] + chunk[b])
            kc[at], vc[at] = k[new], v[new]
        done += chunk
        qo = torch.tensor([0, chunk[0], sum(chunk)], device=DEV)
        out, lse = sc.sparse_window_attention_forward(q[torch.from_numpy(rows).to(DEV)], kc, vc, qo, ko, *window, k_lengths=torch.from_numpy(done).to(DEV))
        check(out, rows, lse)
    assert list(done) == lens


def test_what_is_refused():
    x, o = torch.randn(64, 2, 64, device=DEV), torch.tensor([0, 64], device=DEV)
    out, lse = sc.sparse_window_attention_forward(x, x.clone(), x.clone(), o, None, 3, 0)
    for bad in (dict(dq=x), dict(dk=x), dict(dv=out)):
        with pytest.raises(sc.SubmError) as e:
            sc.sparse_window_attention_backward(torch.ones_like(x), x, x, x, out, lse, o, None, 3, 0, **bad)
        assert e.value.name == "SUBM_ERR_INVALID_ARG"
    with pytest.raises(sc.SubmError) as e:
        sc.sparse_window_attention_forward(x, x, x, o, None, 3, 0, sinks=129)
    assert e.value.name == "SUBM_ERR_UNSUPPORTED"
    m, tok = x.view(64, 128), torch.zeros(64, dtype=torch.int64, device=DEV)
    for call in (lambda: sc.sparse_rms_norm_forward(m.t()), lambda: sc.sparse_rms_norm_forward(m, residual=m[:5]), lambda: sc.sparse_rms_norm_forward(m, m[0].half()),
                 lambda: sc.sparse_rms_norm_backward(m, m, None), lambda: sc.sparse_rms_norm_backward(m[:3], m, m[:, 0].contiguous()),
                 lambda: sc.sparse_embedding_forward(m, tok.float()), lambda: sc.sparse_embedding_forward(m, tok.view(8, 8)),
                 lambda: sc.sparse_embedding_backward(m, tok[:5], 9), lambda: sc.sparse_embedding_backward(m, tok, 0), lambda: sc.sparse_embedding_backward(m, tok, 2 ** 40),
                 lambda: sc.sparse_window_attention_forward(x, x, x, o, None, -1, 0), lambda: sc.sparse_window_attention_forward(x, x, x, o, None, 3, 0, k_lengths=o)):
        with pytest.raises(ValueError):
            call()
    for group in (16, 100, -1):
        with pytest.raises(sc.SubmError):
            sc.sparse_rms_norm_quantize_forward(m, group=group)
    big = torch.empty(1, 20000, device=DEV)
    with pytest.raises(sc.SubmError):
        sc.sparse_rms_norm_forward(big)


def load_example():
    spec = importlib.util.spec_from_file_location("train_sparse_sequence", os.path.join(ROOT, "examples", "train_sparse_sequence.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    return example


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sequence_example_runs(dtype):
    losses, model = load_example().train(steps=3, dtype=dtype, device=DEV, log=lambda *_: None)
    assert np.isfinite(losses).all() and all(torch.isfinite(p).all() and p.grad is not None for p in model.parameters())


def test_sequence_example_gradients():
    # every parameter's gradient against the same model in float64 on the CPU, from elementary operations
    ex = load_example()
    tokens, targets, offsets = ex.batch(DEV, keys=("1",), every=(3,))
    model = ex.Model(torch.float32, DEV)
    torch.nn.functional.cross_entropy(model(tokens, offsets), targets, ignore_index=-1).backward()
    p = {name: w.detach().double().cpu().requires_grad_() for name, w in model.named_parameters()}
    n, tok = tokens.shape[0], tokens.cpu()
    norm = lambda x, g: x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6) * g  # noqa: E731
    x = math.sqrt(ex.CHANNELS) * p["table"][tok]
    qkv = (norm(x, p["gamma1"]) @ p["qkv"].t()).view(n, -1, ex.HEAD_DIM)
    q, k, v = qkv[:, :ex.HEADS], qkv[:, ex.HEADS:ex.HEADS + ex.KV_HEADS], qkv[:, ex.HEADS + ex.KV_HEADS:]
    k, v = (t.repeat_interleave(ex.HEADS // ex.KV_HEADS, 1) for t in (k, v))
    seen = torch.from_numpy(ref.window_mask(n, n, ex.LEFT, 0, ex.SINKS))
    w = (torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(ex.HEAD_DIM)).masked_fill(~seen, -math.inf).softmax(2)
    s = torch.einsum("hij,jhd->ihd", w, v).reshape(n, -1) @ p["proj"].t() + x
    z = torch.nn.functional.silu(norm(s, p["gamma2"]) @ p["up"].t()) @ p["down"].t() + s
    torch.nn.functional.cross_entropy(norm(z, p["gamma3"]) @ p["table"].t(), targets.cpu(), ignore_index=-1).backward()
    for name, g in model.named_parameters():
        near(g.grad, p[name].grad.numpy(), name)
