"""Differentiable layers around the linear layers of a training step: a scaled
embedding table and causal attention, on libdpnorm's kernels.

`Embedding` is the table that RandomizedClipping covers: its per-sample norm is
exact and its gradient is the library's. `attention` is causal softmax
attention with grouped heads over packed or batched sequences; its backward
pass keeps no T x T matrix, and may run twice on one forward pass, as the
DP-SGD-RC step does. Both run on the GPU only, in bfloat16 or float32.

Under HIP graph capture call the functions of the package itself
(attention_forward, attention_backward, embed_*): autograd runs a captured
backward pass on the streams of the eager graphs that hold the same leaves.
"""
from __future__ import annotations

from typing import Optional

import torch
from torch import nn
from torch.autograd.function import once_differentiable

import sample_grad_norms_amd as dp


class _Lookup(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, tokens, scale):
        ctx.save_for_backward(tokens)   # (the caller's own, so that autograd sees a write to them)
        ctx.rows, ctx.scale = weight.shape[0], scale
        return dp.embed_lookup(tokens.contiguous(), weight, scale=scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        (tokens,) = ctx.saved_tensors
        grad = grad.reshape(1, -1, grad.shape[-1])
        if not grad.is_contiguous() or grad.data_ptr() % 16 != 0:
            grad = grad.clone(memory_format=torch.contiguous_format)
        return dp.embed_grad(tokens.reshape(1, -1).contiguous(), grad, ctx.rows, scale=ctx.scale), None, None


class Embedding(nn.Module):
    """A table [rows][dim] looked up as scale * weight[tokens].

    tokens: int32 or int64 of any shape, on the GPU. An id outside
    [0, rows) (a padded position) gives a zero row and adds nothing to the
    gradient. dim: a multiple of 8 (bfloat16) or 4 (float32).
    """

    def __init__(self, rows: int, dim: int, scale: float = 1.0, device=None, dtype=None):
        super().__init__()
        self.scale = float(scale)
        self.weight = nn.Parameter(torch.randn(rows, dim, device=device, dtype=dtype))

    def forward(self, tokens: torch.Tensor) -> torch.Tensor:
        return _Lookup.apply(self.weight, tokens, self.scale)


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, sequences, scale):
        o, lse = dp.attention_forward(q, k, v, cu_seqlens=cu_seqlens, sequences=sequences, scale=scale)
        ctx.save_for_backward(q, k, v, o, lse, cu_seqlens)
        ctx.sequences, ctx.scale = sequences, scale
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        q, k, v, o, lse, cu_seqlens = ctx.saved_tensors
        return dp.attention_backward(_rows(grad), q, k, v, o, lse, cu_seqlens=cu_seqlens, sequences=ctx.sequences,
                                     scale=ctx.scale) + (None, None, None)


def _rows(t: torch.Tensor) -> torch.Tensor:
    """t as the library reads it: rows contiguous, on 16-byte boundaries, tokens less than 2^22 elements apart."""
    step = 16 // t.element_size()
    st, sh, sd = t.stride()
    ok = sd == 1 and st % step == 0 and sh % step == 0 and st < 1 << 22 and t.data_ptr() % 16 == 0
    return t if ok else t.clone(memory_format=torch.contiguous_format)


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
              scale: Optional[float] = None) -> torch.Tensor:
    """Causal attention o of q over k, v, differentiable in all three.

    Either batched, q [B][T][Hq][D], k and v [B][T][Hkv][D], every batch row a
    sequence of its own; or packed, q [N][Hq][D], k and v [N][Hkv][D], with
    cu_seqlens the int32 [S + 1] row offsets of the sequences on the GPU (one
    sequence without them). Hq is a multiple of Hkv, D a multiple of 8
    (bfloat16) or 4 (float32) up to 128; scale defaults to 1 / sqrt(D). Rows of
    a packed call that belong to no sequence give zeros and get zero gradients.
    Sums are float32; in bfloat16 the softmax weights are rounded to bfloat16
    before they multiply rows.
    """
    if q.dim() == 4:
        if cu_seqlens is not None:
            raise ValueError("batched tensors [B][T][H][D] take no cu_seqlens")
        B, T = q.shape[:2]
        if k.dim() != 4 or v.dim() != 4 or k.shape[:2] != (B, T) or v.shape[:2] != (B, T):
            raise ValueError("shapes must be q [B][T][Hq][D], k and v [B][T][Hkv][D]")
        flat = (_rows(t.reshape(B * T, *t.shape[2:])) for t in (q, k, v))
        return _Attention.apply(*flat, None, B if B * T > 0 else 1, scale).view(q.shape)
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be [B][T][H][D] or [N][H][D]")
    return _Attention.apply(_rows(q), _rows(k), _rows(v), cu_seqlens, None, scale)
