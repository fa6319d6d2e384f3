"""Trains one sparse transformer block on voxel shells: the convolution, norm, rotary position and
attention operators as a model uses them together.

    python examples/train_sparse_block.py [--steps 60] [--dtype f32|bf16]

A batch of two synthetic shells (the tiny sphere shell and the sphere-and-torus union).  A fixed
SubMConv3d (k = 3) turns random voxel features into local ones; then, trained:

    h = x + Wo attention(rope(Wqkv norm(x)));   y = Wout (h + W2 silu(W1 norm(h)))

to tell every voxel its direction from the centre of its shell, which needs the positions of the
others.  Prints the loss as it falls.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import numpy as np  # noqa: E402
import torch  # noqa: E402

import submanifold_sparse_convolution_amd as sc  # noqa: E402
import synth  # noqa: E402
from submanifold_sparse_convolution_amd import autograd as sa  # noqa: E402

HEADS, HEAD_DIM, AXES = 4, 32, 3
CHANNELS = HEADS * HEAD_DIM


def batch(device, keys=("1", "2a"), every=(1, 8)):
    """(coords int32 [N, 4], offsets int64 [items + 1], directions float32 [N, 3])."""
    rows, offsets, targets = [], [0], []
    for item, (key, step) in enumerate(zip(keys, every)):
        c = synth.coords_for(key)[::step].copy()
        c[:, 0] = item
        centre = synth.config(key).grid / 2.0
        d = c[:, 1:] - centre
        targets.append(d / np.linalg.norm(d, axis=1, keepdims=True))
        rows.append(c)
        offsets.append(offsets[-1] + len(c))
    coords = torch.from_numpy(np.ascontiguousarray(np.concatenate(rows), dtype=np.int32)).to(device)
    return coords, torch.tensor(offsets, device=device), torch.from_numpy(np.concatenate(targets)).float().to(device)


class Block(torch.nn.Module):
    def __init__(self, dtype, device, seed=0):
        super().__init__()
        g = torch.Generator().manual_seed(seed)
        w = lambda o, i, s=1.0: torch.nn.Parameter((torch.randn(o, i, generator=g) * s / math.sqrt(i)).to(device, dtype))  # noqa: E731
        ones = lambda: torch.nn.Parameter(torch.ones(CHANNELS, device=device, dtype=dtype))  # noqa: E731
        zeros = lambda: torch.nn.Parameter(torch.zeros(CHANNELS, device=device, dtype=dtype))  # noqa: E731
        self.gamma1, self.beta1, self.gamma2, self.beta2 = ones(), zeros(), ones(), zeros()
        self.qkv, self.proj = w(3 * CHANNELS, CHANNELS), w(CHANNELS, CHANNELS, 0.3)
        self.up, self.down = w(2 * CHANNELS, CHANNELS), w(CHANNELS, 2 * CHANNELS, 0.3)
        self.out = w(3, CHANNELS)
        freq, self.magnitude = sc.sparse_rope_frequencies(HEAD_DIM // 2 // AXES, 100.0)
        self.register_buffer("freq", freq.to(device))

    def forward(self, x, coords, offsets):
        n = x.shape[0]
        qkv = (sa.layer_norm(x, self.gamma1, self.beta1) @ self.qkv.t()).view(n, 3 * HEADS, HEAD_DIM)
        qk = sa.rope(qkv[:, :2 * HEADS], coords[:, 1:], self.freq, sc.SUBM_ROPE_INTERLEAVED, self.magnitude)
        a = sa.attention(qk[:, :HEADS], qk[:, HEADS:], qkv[:, 2 * HEADS:], offsets)
        h = x + a.reshape(n, CHANNELS) @ self.proj.t()
        m = torch.nn.functional.silu(sa.layer_norm(h, self.gamma2, self.beta2) @ self.up.t()) @ self.down.t()
        return (h + m) @ self.out.t()


def features(coords, dtype, seed=1):
    """Local voxel features: a fixed SubMConv3d of random ones and the coordinates."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(coords.shape[0], CHANNELS, generator=g)
    x[:, :3] = coords[:, 1:].cpu().float() / 16.0
    w = torch.randn(CHANNELS, 3, 3, 3, CHANNELS, generator=g) / math.sqrt(27 * CHANNELS)
    with sc.sparse_indice_map_build(coords) as m:
        out = sc.subm_conv3d_forward(m, x.to(coords.device, dtype), w.to(coords.device, dtype))
        torch.cuda.synchronize()
    return out


def train(steps=60, dtype=torch.float32, device="cuda:0", log=print):
    """The losses of `steps` steps."""
    coords, offsets, target = batch(device)
    x = features(coords, dtype)
    block = Block(dtype, device)
    optimiser = torch.optim.Adam(block.parameters(), lr=2e-3)
    losses = []
    for step in range(steps):
        optimiser.zero_grad(set_to_none=True)
        loss = (block(x, coords, offsets).float() - target).square().sum(1).mean()
        loss.backward()
        optimiser.step()
        losses.append(loss.item())
        if step % 10 == 0 or step == steps - 1:
            log(f"step {step:3d}: {coords.shape[0]} voxels, loss {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--dtype", choices=("f32", "bf16"), default="f32")
    a = ap.parse_args()
    train(a.steps, {"f32": torch.float32, "bf16": torch.bfloat16}[a.dtype])
