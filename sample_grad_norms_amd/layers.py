"""Differentiable layers around the linear layers of a training step: a scaled
embedding table, layer norm and RMS norm, and causal attention, on libdpnorm's
kernels.

`Embedding`, `LayerNorm` and `RMSNorm` are modules that RandomizedClipping
covers: their per-sample norms are exact and their gradients are the library's.
`attention` is causal softmax attention with grouped heads over packed or
batched sequences, its scores as they are or capped, biased by distance or with
a prefix that every row sees; its backward pass keeps no T x T matrix, and may
run twice on one forward pass, as the DP-SGD-RC step does. All run on the GPU
only, in bfloat16 or float32.

Under HIP graph capture call the functions of the package itself
(attention_forward, attention_backward, embed_*, layernorm_*): autograd runs a
captured backward pass on the streams of the eager graphs that hold the same leaves.
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


def _aligned(t: torch.Tensor) -> torch.Tensor:
    """t as the library reads rows: contiguous, from a 16-byte boundary."""
    return t if t.is_contiguous() and t.data_ptr() % 16 == 0 else t.clone(memory_format=torch.contiguous_format)


class _Normed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, rms):
        x, weight = _aligned(x), _aligned(weight)
        y, mean, rstd = dp.layernorm_forward(x, weight, bias if bias is None else _aligned(bias), eps=eps, rms=rms)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        x, weight, mean, rstd = ctx.saved_tensors
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        dx, dw, db = dp.layernorm_backward(_aligned(grad), x, weight, mean, rstd, bias=need_b, need_dx=need_x, need_dw=need_w)
        return dx, dw, db, None, None


class LayerNorm(nn.Module):
    """Layer norm of the last dimension: (x - mean) / sqrt(variance + eps) * weight + bias.

    dim: a multiple of 8 (bfloat16) or 4 (float32) up to 32768. The input is of
    the weights' type; sums are float32 and the result is rounded once.
    """

    rms = False

    def __init__(self, dim: int, eps: float = 1e-5, bias: bool = True, device=None, dtype=None):
        super().__init__()
        self.eps = float(eps)
        self.weight = nn.Parameter(torch.ones(dim, device=device, dtype=dtype))
        self.bias = nn.Parameter(torch.zeros(dim, device=device, dtype=dtype)) if bias else None

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return _Normed.apply(x, self.weight, self.bias, self.eps, self.rms)


class RMSNorm(LayerNorm):
    """RMS norm of the last dimension: x / sqrt(mean(x^2) + eps) * weight, as LayerNorm."""

    rms = True

    def __init__(self, dim: int, eps: float = 1e-5, device=None, dtype=None):
        super().__init__(dim, eps, bias=False, device=device, dtype=dtype)


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, sequences, scale, cap, slopes, prefix):
        ctx.how = dict(sequences=sequences, scale=scale, cap=cap)
        o, lse = dp.attention_forward(q, k, v, cu_seqlens=cu_seqlens, slopes=slopes, prefix=prefix, **ctx.how)
        ctx.save_for_backward(q, k, v, o, lse, cu_seqlens, slopes, prefix)
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        q, k, v, o, lse, cu_seqlens, slopes, prefix = ctx.saved_tensors
        return dp.attention_backward(_rows(grad), q, k, v, o, lse, cu_seqlens=cu_seqlens, slopes=slopes, prefix=prefix,
                                     **ctx.how) + (None,) * 6


def _rows(t: torch.Tensor) -> torch.Tensor:
    """t as the library reads it: rows contiguous, on 16-byte boundaries, tokens less than 2^22 elements apart."""
    step = 16 // t.element_size()
    st, sh, sd = t.stride()
    ok = sd == 1 and st % step == 0 and sh % step == 0 and st < 1 << 22 and t.data_ptr() % 16 == 0
    return t if ok else t.clone(memory_format=torch.contiguous_format)


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
              scale: Optional[float] = None, cap: Optional[float] = None, slopes: Optional[torch.Tensor] = None,
              prefix: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Causal attention o of q over k, v, differentiable in all three.

    Either batched, q [B][T][Hq][D], k and v [B][T][Hkv][D], every batch row a
    sequence of its own; or packed, q [N][Hq][D], k and v [N][Hkv][D], with
    cu_seqlens the int32 [S + 1] row offsets of the sequences on the GPU (one
    sequence without them). Hq is a multiple of Hkv, D a multiple of 8
    (bfloat16) or 4 (float32) up to 128; scale defaults to 1 / sqrt(D). Rows of
    a packed call that belong to no sequence give zeros and get zero gradients.
    Sums are float32; in bfloat16 the softmax weights are rounded to bfloat16
    before they multiply rows.

    cap: a score s becomes cap * tanh(s / cap). slopes, float32 [Hq]: row t and
    key u get a bias of -slopes[h] * |t - u|; it is fixed, and refused if it
    requires a gradient (a slope below zero is at most 2^14 / (length - 1) steep; a
    steeper one gives NaN). prefix, int32, one for each sequence: every row of a
    sequence sees its first prefix rows.
    """
    if slopes is not None and slopes.requires_grad:
        raise ValueError("slopes are not differentiable here: detach them")
    if q.dim() == 4:
        if cu_seqlens is not None:
            raise ValueError("batched tensors [B][T][H][D] take no cu_seqlens")
        B, T = q.shape[:2]
        if k.dim() != 4 or v.dim() != 4 or k.shape[:2] != (B, T) or v.shape[:2] != (B, T):
            raise ValueError("shapes must be q [B][T][Hq][D], k and v [B][T][Hkv][D]")
        flat = (_rows(t.reshape(B * T, *t.shape[2:])) for t in (q, k, v))
        sequences = B if B * T > 0 else 1
        if prefix is not None and B * T == 0:
            prefix = None
        return _Attention.apply(*flat, None, sequences, scale, cap, slopes, prefix).view(q.shape)
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be [B][T][H][D] or [N][H][D]")
    return _Attention.apply(_rows(q), _rows(k), _rows(v), cu_seqlens, None, scale, cap, slopes, prefix)
