"""The operators of a sparse transformer block as differentiable functions.

Each is the forward entry point of the same name joined to its backward entry point through
torch.autograd; they run on torch's current stream.  Gradients come out in the dtype of their
input.
"""
from __future__ import annotations

import torch

from . import _binding as _b


def _plain(t: torch.Tensor) -> torch.Tensor:
    """A gradient as the library takes it: autograd may hand over expanded or permuted ones, and parts
    of larger ones (of a concatenation) that start anywhere."""
    return t if t.is_contiguous() and t.data_ptr() % 16 == 0 else t.clone(memory_format=torch.contiguous_format)


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma, beta, eps):
        y, mean, rstd = _b.sparse_layer_norm_forward(x, gamma, beta, eps, stats=True)
        ctx.save_for_backward(x, gamma, mean, rstd)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, gamma, mean, rstd = ctx.saved_tensors
        wanted = ctx.needs_input_grad[1] or ctx.needs_input_grad[2]
        dx, dgamma, dbeta = _b.sparse_layer_norm_backward(_plain(dy), x, mean, rstd, gamma, weight_grads=wanted)
        return dx, dgamma if ctx.needs_input_grad[1] else None, dbeta if ctx.needs_input_grad[2] else None, None


def layer_norm(x: torch.Tensor, gamma: torch.Tensor | None = None, beta: torch.Tensor | None = None,
               eps: float = 1e-5) -> torch.Tensor:
    """Layer norm of the rows of x [N, C]; see sparse_layer_norm_forward."""
    return _LayerNorm.apply(x, gamma, beta, eps)


class _Rope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, positions, freq, layout, magnitude):
        ctx.save_for_backward(positions, freq)
        ctx.layout, ctx.magnitude = layout, magnitude
        return _b.sparse_rope_forward(x, positions, freq, layout, magnitude)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        positions, freq = ctx.saved_tensors
        return _b.sparse_rope_backward(_plain(dy), positions, freq, ctx.layout, ctx.magnitude), None, None, None, None


def rope(x: torch.Tensor, positions: torch.Tensor, freq: torch.Tensor, layout: int,
         magnitude: float = 1.0) -> torch.Tensor:
    """Rotary positions of x [N, heads, head_dim]; see sparse_rope_forward."""
    return _Rope.apply(x, positions, freq, layout, magnitude)


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, q_offsets, k_offsets, scale):
        out, lse = _b.sparse_attention_forward(q, k, v, q_offsets, k_offsets, scale)
        ctx.save_for_backward(q, k, v, out, lse, q_offsets, k_offsets)
        ctx.scale = scale
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        q, k, v, out, lse, q_offsets, k_offsets = ctx.saved_tensors
        dq, dk, dv = _b.sparse_attention_backward(_plain(dout), q, k, v, out, lse, q_offsets, k_offsets, ctx.scale)
        return dq, dk, dv, None, None, None


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_offsets: torch.Tensor,
              k_offsets: torch.Tensor | None = None, scale: float | None = None) -> torch.Tensor:
    """Attention within items; see sparse_attention_forward."""
    return _Attention.apply(q, k, v, q_offsets, k_offsets, scale)
