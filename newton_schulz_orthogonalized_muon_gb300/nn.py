"""The training operators for autograd: what a transformer block needs around
the Muon step, with the library's kernels in both directions.

``LayerNorm``   layer norm whose weight and bias gradients are summed in fp32;
``attention``   attention that keeps its output and lse and recomputes the
                probabilities in the backward pass;
``Linear8``     a linear layer that keeps its input in 8 bits (half of a bf16
                copy) and takes its weight's gradient from the codes.

The weights of ``Linear8`` are the 2-D matrices that ``Muon`` orthogonalises;
the vectors of ``LayerNorm`` go to its AdamW fallback.
"""
from __future__ import annotations

import math

import torch
from torch.autograd.function import once_differentiable

from . import ops


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = ops.layer_norm(x, weight, bias, eps=eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        dx, dw, db = ops.layer_norm_backward(dy, x, mean, rstd, weight)
        return (dx, None if weight is None else dw.to(weight.dtype),
                None if ctx.bias_dtype is None else db.to(ctx.bias_dtype), None)


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5):
    """Differentiable layer norm over the last dimension (see ops.layer_norm)."""
    return _LayerNorm.apply(x, weight, bias, eps)


class LayerNorm(torch.nn.Module):
    """Layer norm over the last dimension; weight and bias are fp32 unless
    ``dtype`` says otherwise (the type of the activations)."""

    def __init__(self, cols: int, eps: float = 1e-5, bias: bool = True, device=None, dtype=torch.float32):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(cols, device=device, dtype=dtype))
        self.bias = torch.nn.Parameter(torch.zeros(cols, device=device, dtype=dtype)) if bias else None

    def forward(self, x):
        return layer_norm(x, self.weight, self.bias, self.eps)


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens_q, cu_seqlens_k, options):
        o, lse = ops.attention(q, k, v, cu_seqlens_q=cu_seqlens_q, cu_seqlens_k=cu_seqlens_k, **options)
        # the offsets too: the backward pass reads them on the device, and only
        # saved tensors are watched for a write in between
        ctx.save_for_backward(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k)
        ctx.options = options
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k = ctx.saved_tensors
        grads = ops.attention_backward(do, q, k, v, o, lse, cu_seqlens_q=cu_seqlens_q, cu_seqlens_k=cu_seqlens_k,
                                       **ctx.options)
        return (*grads, None, None, None)


def attention(q, k, v, *, causal: bool = False, window: int = 0, scale=None, cu_seqlens_q=None, cu_seqlens_k=None):
    """Differentiable attention (see ops.attention); returns the output.  The
    offsets are kept for the backward pass like the other inputs: writing to
    them before it raises."""
    return _Attention.apply(q, k, v, cu_seqlens_q, cu_seqlens_k, dict(causal=causal, window=window, scale=scale))


class _Linear8(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight):
        # the input is kept for the weight's gradient, the weight for the input's
        codes = scales = None
        if ctx.needs_input_grad[1]:
            codes, scales = ops.act8_store(x.reshape(-1, x.shape[-1]))
        ctx.save_for_backward(codes, scales, weight if ctx.needs_input_grad[0] else None)
        ctx.dtype = weight.dtype
        return x @ weight.t()

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        codes, scales, weight = ctx.saved_tensors
        dw = None if codes is None else \
            ops.act8_weight_grad(dy.reshape(-1, dy.shape[-1]), codes, scales, dtype=ctx.dtype)
        return None if weight is None else dy @ weight, dw


def linear8(x, weight):
    """x weight^T, both bf16; the input is kept in 8 bits for the weight's
    gradient (see ops.act8_store for the format), if there will be one."""
    if x.dtype != torch.bfloat16 or weight.dtype != torch.bfloat16:
        raise ValueError("linear8 takes bfloat16 inputs and weights")
    if not torch.is_grad_enabled():
        return x @ weight.t()
    return _Linear8.apply(x, weight)


class Linear8(torch.nn.Module):
    """A bf16 linear layer without bias whose input is kept in 8 bits."""

    def __init__(self, cols: int, out: int, device=None):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.empty(out, cols, device=device, dtype=torch.bfloat16))
        torch.nn.init.normal_(self.weight, std=1.0 / math.sqrt(cols))

    def forward(self, x):
        return linear8(x, self.weight)
