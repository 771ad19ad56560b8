"""torch.autograd glue for the CUDA kernels: the forward saves (L, Q, K, V, O)
and the backward recomputes from them ("CS336 Assignment 2 notes" §1.4, the
FlashAttention-2 autograd function), so the kernels drop into a model in place
of its attention core ("CS324 lecture 8: 03_online_softmax_and_flash.py",
patched_model).  Argument marshalling only: every step runs in the library.
"""
from __future__ import annotations

import torch

from . import attention_backward, attention_forward


class FlashAttentionFunction(torch.autograd.Function):
    """O = softmax(Q K^T scale) V with the mask of fa_fwd_ex; bf16 CUDA tensors
    q [B,H,Nq,d], k, v [B,H,Nk,d].  Saves L (fp32 [B,H,Nq]), Q, K, V and O; no
    N x N tensor is kept."""

    @staticmethod
    def forward(ctx, q, k, v, causal: bool = False, scale=None, window: int = 0):
        q, k, v = (t.contiguous() for t in (q, k, v))
        o, lse = attention_forward(q, k, v, causal, scale, window)
        ctx.save_for_backward(lse, q, k, v, o)
        ctx.causal, ctx.scale, ctx.window = causal, scale, window
        return o

    @staticmethod
    def backward(ctx, do):
        lse, q, k, v, o = ctx.saved_tensors
        dq, dk, dv, _ = attention_backward(q, k, v, o, lse, do.contiguous(), ctx.causal, ctx.scale, ctx.window)
        return dq, dk, dv, None, None, None


def flash_attention(q, k, v, causal: bool = False, scale=None, window: int = 0):
    """Differentiable exact attention through the CUDA kernels."""
    return FlashAttentionFunction.apply(q, k, v, causal, scale, window)


class QKNormRopeFunction(torch.autograd.Function):
    """Per-head norm and rotation of q and k (fa_qk_norm_rope).  Saves its inputs only: the gradients recompute the
    rows' norms.  No gradient for the tables and the positions."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved):
        ctx.save_for_backward(q, k, q_weight, k_weight, cos, sin, positions)
        ctx.eps, ctx.interleaved = eps, interleaved
        from . import operators  # here, as flash_attention does not need its native module
        return operators.qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, q_weight, k_weight, cos, sin, positions = ctx.saved_tensors
        from . import operators
        grads = operators.qk_norm_rope_backward(q, k, _rows(dq_out), _rows(dk_out), q_weight, k_weight, cos, sin,
                                                positions, ctx.eps, ctx.interleaved)
        return (*grads, None, None, None, None, None)


def _rows(t):
    """t with strides the kernels take: contiguous rows that start on 16 bytes."""
    if t.dim() != 4:
        return t  # refused with the other shapes
    fits = t.stride(3) == 1 and all(s % 8 == 0 for n, s in zip(t.shape, t.stride()[:3]) if n > 1)
    return t if fits and t.data_ptr() % 16 == 0 else t.contiguous()


def qk_norm_rope(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, eps=1e-6, interleaved=False):
    """Differentiable qk_norm_rope: q and k of any layout (rows that the kernels cannot take as they lie are copied).

    Before a backward is captured into a CUDA graph, let go of every eager graph of the same leaves: PyTorch adds a
    leaf's gradient on the stream that graph was made on, which a capture on another stream may not touch."""
    return QKNormRopeFunction.apply(_rows(q), _rows(k), q_weight, k_weight, cos, sin, positions, eps, interleaved)
