"""The transformer-block operators as a program uses them: differentiated through torch, captured in
a graph, called from two threads on one stream, and the training example."""
import importlib.util
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


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    sc.load_library()


def leaf(rng, *shape):
    return synth.round_to(rng.standard_normal(shape), "f32").to(DEV).requires_grad_()


def near(got, want, what):
    # float32 chains of three operators with sums of at most 128 terms: 512 * 2^-23 < 1e-4 of the norm
    off = np.linalg.norm(got.detach().double().cpu().numpy() - want) / np.linalg.norm(want)
    print(f"  {what}: {off:.2e}", flush=True)
    assert off < 1e-4, what


def test_block_gradients_through_autograd():
    rng = np.random.default_rng(0)
    n, heads, d = 90, 4, 16
    offsets = [0, 50, 50, 90]
    off = torch.tensor(offsets, device=DEV)
    pos = torch.from_numpy(rng.integers(0, 30, (n, 4)).astype(np.int32)).to(DEV)[:, 1:]
    freq = sc.sparse_rope_frequencies(2)[0].to(DEV)
    x, gamma, beta, v = leaf(rng, n, heads * d), leaf(rng, heads * d), leaf(rng, heads * d), leaf(rng, n, heads, d)
    k = leaf(rng, n, heads // 2, d)
    w = torch.from_numpy(rng.standard_normal((n, heads, d))).float().to(DEV)
    h = sa.layer_norm(x, gamma, beta).view(n, heads, d)
    q = sa.rope(h, pos, freq, sc.SUBM_ROPE_HALF, 1.1)
    out = sa.attention(q, k, v[:, ::2], off)
    (out * w).sum().backward()  # (an expanded gradient on the way)

    f = lambda t: t.detach().double().cpu().numpy()  # noqa: E731
    y, _, _ = ref.layer_norm(f(x), f(gamma), f(beta))
    rq = ref.rope(y.reshape(n, heads, d), f(pos), f(freq), False, 1.1)
    scale = d ** -0.5
    near(out, ref.attention(rq, f(k), f(v)[:, ::2], offsets, offsets, scale)[0], "out")
    dq, dk, dv = ref.attention_grad(f(w), rq, f(k), f(v)[:, ::2], offsets, offsets, scale)
    dh = ref.rope(dq, f(pos), f(freq), False, 1.1, back=True).reshape(n, heads * d)
    dx, dg, db = ref.layer_norm_grad(dh, f(x), f(gamma))
    near(k.grad, dk, "dk")
    near(v.grad[:, ::2], dv, "dv")
    near(x.grad, dx, "dx")
    near(gamma.grad, dg, "dgamma")
    near(beta.grad, db, "dbeta")


def test_plain_norm_and_partial_gradients():
    rng = np.random.default_rng(1)
    x, beta = leaf(rng, 20, 24), leaf(rng, 24)
    sa.layer_norm(x).sum().backward()
    assert x.grad.abs().max() < 1e-4  # a normalised row's sum does not depend on the row
    x.grad = None
    sa.layer_norm(x.detach(), None, beta).sum().backward()
    assert torch.equal(beta.grad, torch.full_like(beta, 20.0)) and x.grad is None


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_that_start_anywhere(dtype):
    # the gradient of a part of a concatenation is a view of the whole one, at an odd element
    rng = np.random.default_rng(4)
    n, heads, d = 40, 2, 16
    off = torch.tensor([0, 15, 40], device=DEV)
    pos = torch.arange(n, device=DEV, dtype=torch.int32)[:, None]
    freq = sc.sparse_rope_frequencies(4)[0].to(DEV)
    x, gamma = (leaf(rng, *shape).detach().to(dtype).requires_grad_() for shape in ((n, heads * d), (heads * d,)))
    w = leaf(rng, 1 + n * heads * d).detach().to(dtype)
    grads = []
    for front in (1, 0):
        for f in (lambda: sa.layer_norm(x, gamma), lambda: sa.rope(x.view(n, heads, d), pos, freq, sc.SUBM_ROPE_HALF),
                  lambda: sa.attention(*[x.view(n, heads, d)] * 3, off)):
            x.grad = None
            y = f().reshape(-1)
            y = torch.cat([y[:1].detach(), y]) if front else y
            (y * w[1 - front:]).sum().backward()
            grads.append(x.grad)
    assert all(torch.equal(a, b) for a, b in zip(grads[:3], grads[3:]))


def test_captured_in_a_graph():
    rng = np.random.default_rng(2)
    n, heads, d = 600, 4, 64
    s = torch.cuda.Stream()
    t = lambda *shape: synth.round_to(rng.standard_normal(shape), "bf16").to(DEV)  # noqa: E731
    x, gamma, beta, dy, q, k, v, g = t(n, 256), t(256), t(256), t(n, 256), t(n, heads, d), t(n, heads, d), t(n, heads, d), t(n, heads, d)
    qo = torch.tensor([0, 200, 600], device=DEV)
    one, caches, ko = t(2, heads, d), t(8000, heads, d), torch.tensor([0, 3000, 8000], device=DEV)
    oo = torch.tensor([0, 1, 2], device=DEV)
    pos, freq = torch.arange(n, device=DEV, dtype=torch.int32)[:, None], sc.sparse_rope_frequencies(32)[0].to(DEV)

    def step():
        y, mean, rstd = sc.sparse_layer_norm_forward(x, gamma, beta, stats=True)
        grads = sc.sparse_layer_norm_backward(dy, x, mean, rstd, gamma)
        r = sc.sparse_rope_forward(q, pos, freq, sc.SUBM_ROPE_INTERLEAVED)
        out, lse = sc.sparse_attention_forward(r, k, v, qo)
        back = sc.sparse_attention_backward(g, r, k, v, out, lse, qo)
        few = sc.sparse_attention_forward(one, caches, caches, oo, ko)
        return [y, mean, rstd, *grads, r, out, lse, *back, *few]

    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        step()  # the stream's scratch memory grows here, not under capture
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            captured = step()
        for round_ in range(4):
            for z in (x, dy, q, k, v, g, one):
                z.copy_(torch.randn(z.shape, device=DEV))
            eager = [e.clone() for e in step()]
            if round_ == 1:  # a larger call on the stream: what the graph holds must stay
                big = torch.randn(40000, heads, d, device=DEV).to(torch.bfloat16)
                sc.sparse_attention_backward(big, big, big, big, *sc.sparse_attention_forward(big, big, big, torch.tensor([0, 40000], device=DEV)), torch.tensor([0, 40000], device=DEV))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(captured, eager)), round_


def test_scratch_cannot_grow_under_capture():
    q = torch.randn(64, 2, 64, device=DEV)
    o = torch.tensor([0, 64], device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = sc.sparse_attention_forward(q, q, q, o)  # (on another stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y = q + 1.0
        with pytest.raises(sc.SubmError) as e:
            sc.sparse_attention_backward(q, q, q, q, out, lse, o)
    assert e.value.name == "SUBM_ERR_UNSUPPORTED" and "capture" in e.value.detail
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, q + 1.0)


def test_two_threads_on_one_stream():
    rng = np.random.default_rng(3)
    o = {n: torch.tensor([0, n], device=DEV) for n in (300, 900)}
    sets = {n: [synth.round_to(rng.standard_normal((n, 4, 64)), "f16").to(DEV) for _ in range(4)] for n in o}
    want, got, errors = {}, {n: [] for n in o}, []

    def work(n):
        q, k, v, g = sets[n]
        out, lse = sc.sparse_attention_forward(q, k, v, o[n])
        return [out, lse, *sc.sparse_attention_backward(g, q, k, v, out, lse, o[n])]

    for n in o:
        want[n] = work(n)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    def loop(n):
        try:
            with torch.cuda.stream(side):
                for _ in range(20):
                    got[n].append(work(n))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=loop, args=(n,)) for n in o]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for n in o:
        for run in got[n]:
            assert all(torch.equal(a, b) for a, b in zip(run, want[n]))


def test_gradients_must_not_alias_inputs():
    q = torch.randn(64, 2, 64, device=DEV)
    o = torch.tensor([0, 64], device=DEV)
    out, lse = sc.sparse_attention_forward(q, q, q, o)
    for bad in (dict(dq=q), dict(dk=q), dict(dv=out)):
        with pytest.raises(sc.SubmError) as e:
            sc.sparse_attention_backward(torch.ones_like(q), q, q, q, out, lse, o, **bad)
        assert e.value.name == "SUBM_ERR_INVALID_ARG"
    with pytest.raises(sc.SubmError):
        sc.sparse_attention_forward(q, q.clone(), out, o, out=out)
    k = q.clone()
    want = sc.sparse_attention_forward(q, k, k, o)[0]
    assert torch.equal(sc.sparse_attention_forward(q, k, k, o, out=q)[0], want)  # over the queries


@pytest.mark.parametrize("dtype,least", [(torch.float32, 0.5), (torch.bfloat16, 0.6)])
def test_training_example(dtype, least):
    spec = importlib.util.spec_from_file_location("train_sparse_block", os.path.join(ROOT, "examples", "train_sparse_block.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.train(steps=40, dtype=dtype, device=DEV)
    assert losses[-1] < least * losses[0]
