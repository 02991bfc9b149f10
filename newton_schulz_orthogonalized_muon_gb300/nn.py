"""The training operators for autograd: what a transformer block needs around
the Muon step, with the library's kernels in both directions.

``LayerNorm``   layer norm whose weight and bias gradients are summed in fp32;
``attention``   attention that keeps its output and lse and recomputes the
                probabilities in the backward pass;
``Linear8``     a linear layer that keeps its input in 8 bits (half of a bf16
                copy) and takes its weight's gradient from the codes; with
                ``products8`` its products run in 8 bits too;
``ExpertLinear``  a layer of experts over tokens grouped by expert.

The weights of ``Linear8`` and ``ExpertLinear`` are the 2-D matrices that
``Muon`` orthogonalises (an expert's block of rows each, with ``split_heads``);
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


class _Linear8Products(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight):
        needs_x, needs_w = ctx.needs_input_grad
        codes, scales = ops.act8_store(x.reshape(-1, x.shape[-1]))
        # the transpose's codes serve the input's gradient
        wcodes, wscales, *wcodes_t = ops.act8_store_weight(weight, transposed=needs_x)
        y = ops.act8_matmul(codes, scales, wcodes, wscales, dtype=x.dtype)
        ctx.save_for_backward(codes if needs_w else None, scales if needs_w else None, *(wcodes_t or [None]),
                              wscales if needs_x else None)
        ctx.dtype = weight.dtype
        return y.view(*x.shape[:-1], weight.shape[0])

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        codes, scales, wcodes_t, wscales = ctx.saved_tensors
        dx, flat = None, dy.reshape(-1, dy.shape[-1])
        if wcodes_t is not None:
            dx = ops.act8_matmul(*ops.act8_store(flat), wcodes_t, wscales.t(), dtype=dy.dtype)
            dx = dx.view(*dy.shape[:-1], wcodes_t.shape[0])
        return dx, None if codes is None else ops.act8_weight_grad(flat, codes, scales, dtype=ctx.dtype)


def linear8(x, weight, *, products8: bool = False):
    """x weight^T, both bf16; the input is kept in 8 bits for the weight's
    gradient (see ops.act8_store for the format), if there will be one.

    products8: the product and the input's gradient run in 8 bits too, of the
    stored input, weight and gradient of the output (ops.act8_matmul), each
    value of which is rounded to e4m3, by up to 2^-4 of itself.  The weight is
    stored anew by each call, which a step needs; for many calls on one weight
    store it once (ops.act8_store_weight) and call ops.act8_matmul."""
    if x.dtype != torch.bfloat16 or weight.dtype != torch.bfloat16:
        raise ValueError("linear8 takes bfloat16 inputs and weights")
    if products8:
        return _Linear8Products.apply(x, weight)
    if not torch.is_grad_enabled():
        return x @ weight.t()
    return _Linear8.apply(x, weight)


class Linear8(torch.nn.Module):
    """A bf16 linear layer without bias whose input is kept in 8 bits;
    ``products8``: its products run in 8 bits too (see linear8)."""

    def __init__(self, cols: int, out: int, device=None, products8: bool = False):
        super().__init__()
        self.products8 = products8
        self.weight = torch.nn.Parameter(torch.empty(out, cols, device=device, dtype=torch.bfloat16))
        torch.nn.init.normal_(self.weight, std=1.0 / math.sqrt(cols))

    def forward(self, x):
        return linear8(x, self.weight, products8=self.products8)


class _ExpertLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, offsets):
        # the offsets too: the backward pass reads them on the device, and only
        # saved tensors are watched for a write in between
        ctx.save_for_backward(x if ctx.needs_input_grad[1] else None, weight if ctx.needs_input_grad[0] else None, offsets)
        ctx.dtype = weight.dtype
        return ops.expert_matmul(x, weight, offsets)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, offsets = ctx.saved_tensors
        dx = None if weight is None else ops.expert_matmul(dy, weight, offsets, transpose=True)
        dw = None if x is None else ops.expert_weight_grad(dy, x, offsets, dtype=ctx.dtype)
        return dx, dw, None


def expert_linear(x, weight, offsets):
    """Differentiable ops.expert_matmul: x [tokens, cols], weight [experts,
    out, cols], offsets int32 [experts + 1], which are kept for the backward
    pass like the other inputs: writing to them before it raises.  cols is 2^16
    at most, and where x needs a gradient out is too."""
    return _ExpertLinear.apply(x, weight, offsets)


class ExpertLinear(torch.nn.Module):
    """A linear layer without bias for each of a number of experts, over tokens
    grouped by expert.

    The weight is 2-D, [experts * out, cols], one expert below the other, so that
    ``Muon`` takes it: with ``split_heads={name: experts}`` each expert's matrix
    is orthogonalised on its own, and ``scale_dims={name: max(out, cols)}``
    gives the update the size that a matrix of one expert has."""

    def __init__(self, experts: int, cols: int, out: int, device=None, dtype=torch.bfloat16):
        super().__init__()
        self.experts = experts
        self.weight = torch.nn.Parameter(torch.empty(experts * out, cols, device=device, dtype=dtype))
        torch.nn.init.normal_(self.weight, std=1.0 / math.sqrt(cols))

    def forward(self, x, offsets):
        return expert_linear(x, self.weight.unflatten(0, (self.experts, -1)), offsets)
