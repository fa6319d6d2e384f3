"""Trains a causal transformer on the voxels of shells in Morton order: the embedding, root-mean-square norm
and sliding-window attention operators as a sequence model uses them together.

    python examples/train_sparse_sequence.py [--steps 60] [--dtype f32|bf16]

A voxel's token is how many of its 26 neighbours are there (read from the indice map); the model tells the
next voxel's token from those before it, of which each sees the last 64 and the first 4 of its shell:

    x = sqrt(C) T[token];   y, s = norm(Wo window_attention(Wqkv norm(x)) + x)
    logits = norm(W2 silu(W1 y) + s) T^t

Prints the loss as it falls.
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

HEADS, KV_HEADS, HEAD_DIM = 4, 2, 32
CHANNELS = HEADS * HEAD_DIM
TOKENS = 27
LEFT, SINKS = 63, 4


def morton(coords):
    """Positions along the Morton curve of int coordinates [N, 3]."""
    code = np.zeros(len(coords), dtype=np.int64)
    for bit in range(10):
        for axis in range(3):
            code |= ((coords[:, axis].astype(np.int64) >> bit) & 1) << (3 * bit + axis)
    return code


def batch(device, keys=("1", "2a"), every=(1, 8)):
    """(tokens int64 [N], targets int64 [N] with -1 at the last voxel of a shell, offsets int64 [items + 1])."""
    tokens, targets, offsets = [], [], [0]
    for key, step in zip(keys, every):
        c = synth.coords_for(key)
        with sc.sparse_indice_map_build(torch.from_numpy(np.ascontiguousarray(c)).to(device)) as m:
            there = (sc.sparse_indice_map_copy_nbr(m) >= 0).sum(1) - 1
        t = there.cpu().numpy()[np.argsort(morton(c[:, 1:]), kind="stable")][:len(c) // step]
        tokens.append(t)
        targets.append(np.append(t[1:], -1))
        offsets.append(offsets[-1] + len(t))
    cat = lambda parts: torch.from_numpy(np.concatenate(parts).astype(np.int64)).to(device)  # noqa: E731
    return cat(tokens), cat(targets), torch.tensor(offsets, device=device)


class Model(torch.nn.Module):
    def __init__(self, dtype, device, seed=0):
        super().__init__()
        g = torch.Generator().manual_seed(seed)
        w = lambda o, i, s=1.0: torch.nn.Parameter((torch.randn(o, i, generator=g) * s / math.sqrt(i)).to(device, dtype))  # noqa: E731
        ones = lambda: torch.nn.Parameter(torch.ones(CHANNELS, device=device, dtype=dtype))  # noqa: E731
        self.table = w(TOKENS, CHANNELS)
        self.gamma1, self.gamma2, self.gamma3 = ones(), ones(), ones()
        self.qkv, self.proj = w((HEADS + 2 * KV_HEADS) * HEAD_DIM, CHANNELS), w(CHANNELS, CHANNELS, 0.3)
        self.up, self.down = w(2 * CHANNELS, CHANNELS), w(CHANNELS, 2 * CHANNELS, 0.3)

    def forward(self, tokens, offsets):
        n = tokens.shape[0]
        x = sa.embedding(self.table, tokens, math.sqrt(CHANNELS))
        qkv = (sa.rms_norm(x, self.gamma1) @ self.qkv.t()).view(n, HEADS + 2 * KV_HEADS, HEAD_DIM)
        a = sa.window_attention(qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:], offsets, left=LEFT, right=0, sinks=SINKS)
        y, s = sa.rms_norm(a.reshape(n, CHANNELS) @ self.proj.t(), self.gamma2, residual=x)
        z, _ = sa.rms_norm(torch.nn.functional.silu(y @ self.up.t()) @ self.down.t(), self.gamma3, residual=s)
        return z @ self.table.t()


def train(steps=60, dtype=torch.float32, device="cuda:0", log=print):
    """(the losses of `steps` steps, the model)."""
    tokens, targets, offsets = batch(device)
    model = Model(dtype, device)
    optimiser = torch.optim.Adam(model.parameters(), lr=2e-3)
    losses = []
    for step in range(steps):
        optimiser.zero_grad(set_to_none=True)
        loss = torch.nn.functional.cross_entropy(model(tokens, offsets).float(), targets, ignore_index=-1)
        loss.backward()
        optimiser.step()
        losses.append(loss.item())
        if step % 10 == 0 or step == steps - 1:
            log(f"step {step:3d}: {tokens.shape[0]} voxels, loss {losses[-1]:.4f}")
    return losses, model


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--dtype", choices=("f32", "bf16"), default="f32")
    a = ap.parse_args()
    train(a.steps, {"f32": torch.float32, "bf16": torch.bfloat16}[a.dtype])
