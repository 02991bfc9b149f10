"""Training operators around the Muon step, as calls on torch tensors.

Layer norm, attention (with the backward pass that recomputes the
probabilities) and activations kept in 8 bits.  Each is a call of the C ABI
in include/muon.h by way of an extension module (csrc/torch_ops.cpp): the
tensors are checked, outputs and scratch are allocated by torch on the stream
that the kernels run on, arguments that do not go together raise ValueError,
a non-OK status raises MuonError.

These calls are outside autograd: they take the values of tensors that require
gradients and return results without a graph (or a tangent).  ``nn`` wraps
them for autograd.

Every function takes ``stream`` (default: the current stream of the tensors'
device) and ``handle`` (default: that device's handle).  Inputs that are
written on another stream have to be ready there, as for any call.
"""
from __future__ import annotations

import torch

from . import _binding

try:
    from . import _torch_ops as _native
    _why = None
except ImportError as _e:            # said when a function is called: importing needs no build
    _native, _why = None, _e


def _target(first, handle):
    """The handle for a call whose first tensor is `first`."""
    dev = first.get_device() if isinstance(first, torch.Tensor) else -1     # -1: not on a GPU
    if dev < 0:
        raise ValueError("the operators take CUDA tensors")
    if _native is None:
        raise RuntimeError("the extension module of the operators does not load: build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`") from _why
    if handle is None:
        return _binding.default_handle(dev)
    if handle.device != dev:
        raise ValueError(f"the handle is on device {handle.device}, the tensors on {dev}")
    return handle


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5, handle=None, stream=None):
    """Layer norm over the last dimension: ``(y, mean, rstd)``.

    x: [.., cols] fp32, bf16 or fp16, cols up to 16384; weight and bias:
    [cols], fp32 or x's type, or None (ones, zeros).  y has x's type and
    shape, mean and rstd (fp32, x.shape[:-1]) are what the backward pass
    takes."""
    if stream is not None:
        with torch.cuda.stream(stream):  # torch ties outputs and scratch to it
            return layer_norm(x, weight, bias, eps=eps, handle=handle)
    h = _target(x, handle)
    got = _native.layer_norm(h.address, h.device, x, weight, bias, eps)
    if type(got) is int:
        h._raise(got, "layer_norm")
    return got


def layer_norm_backward(dy, x, mean, rstd, weight=None, *, handle=None, stream=None):
    """``(dx, dweight, dbias)`` of layer_norm: dx in x's type, dweight and
    dbias fp32 [cols], summed over all rows in a fixed order."""
    if stream is not None:
        with torch.cuda.stream(stream):  # torch ties outputs and scratch to it
            return layer_norm_backward(dy, x, mean, rstd, weight, handle=handle)
    h = _target(x, handle)
    got = _native.layer_norm_backward(h.address, h.device, dy, x, mean, rstd, weight)
    if type(got) is int:
        h._raise(got, "layer_norm_backward")
    return got


def attention(q, k, v, *, causal: bool = False, window: int = 0, scale=None, cu_seqlens_q=None, cu_seqlens_k=None,
              handle=None, stream=None):
    """Attention, ``(o, lse)``.

    q: [batch, sq, heads, dim], k and v: [batch, sk, kv_heads, dim], bf16 or
    fp16, dim a multiple of 8 up to 128, kv_heads a divisor of heads; any
    strides that are multiples of 8, the last dimension contiguous.  With
    ``cu_seqlens_q`` and ``cu_seqlens_k`` (int32 on the device, one offset
    more than sequences) the tensors are [tokens, heads, dim], sequences one
    after another.  Query i stands at place i + sk - sq of its sequence;
    ``causal``: it sees keys up to its place, with ``window`` only the last
    ``window`` of them.  scale (above 0): 1 / sqrt(dim) by default.
    o has q's shape and type (a query that sees no key: 0); lse is fp32
    [batch, heads, sq] or [heads, tokens] (there: -inf).  The softmax is fp32;
    the probabilities are rounded to q's type for their product with v."""
    if stream is not None:
        with torch.cuda.stream(stream):  # torch ties outputs and scratch to it
            return attention(q, k, v, causal=causal, window=window, scale=scale, cu_seqlens_q=cu_seqlens_q,
                             cu_seqlens_k=cu_seqlens_k, handle=handle)
    h = _target(q, handle)
    got = _native.attention(h.address, h.device, q, k, v, causal, window, scale, cu_seqlens_q, cu_seqlens_k)
    if type(got) is int:
        h._raise(got, "attention")
    return got


def attention_backward(do, q, k, v, o, lse, *, causal: bool = False, window: int = 0, scale=None, cu_seqlens_q=None,
                       cu_seqlens_k=None, handle=None, stream=None):
    """``(dq, dk, dv)`` of attention, from its output and lse: the
    probabilities are recomputed, nothing of size sq x sk is kept.  dk and dv
    are summed over the query heads that share them, in a fixed order.  The
    probabilities and the scores' gradients are rounded to q's type for their
    products; with fp16 `do` has to be scaled so that the latter fit it."""
    if stream is not None:
        with torch.cuda.stream(stream):  # torch ties outputs and scratch to it
            return attention_backward(do, q, k, v, o, lse, causal=causal, window=window, scale=scale, cu_seqlens_q=cu_seqlens_q,
                                      cu_seqlens_k=cu_seqlens_k, handle=handle)
    h = _target(q, handle)
    got = _native.attention_backward(h.address, h.device, do, q, k, v, o, lse, causal, window, scale, cu_seqlens_q,
                                     cu_seqlens_k)
    if type(got) is int:
        h._raise(got, "attention_backward")
    return got


def act8_store(x, *, handle=None, stream=None):
    """x [rows, cols] (fp32, bf16, fp16) in 8 bits: ``(codes, scales)``.

    codes: float8_e4m3fn [rows, cols]; scales: uint8 [ceil(cols / 128),
    rows], one exponent a row and 128 columns: the stored value is code times
    2^(scale - 127), with the smallest power of two that fits the block's
    largest value (at least 2^-111).  A block with a NaN or an infinity is
    stored as scale 255, codes 0 and stands for NaN.  Both have padded row
    strides (whole blocks, 16 rows), which act8_weight_grad reads in place;
    copies in other layouts are taken too, at the cost of one more copy."""
    if stream is not None:
        with torch.cuda.stream(stream):  # torch ties outputs and scratch to it
            return act8_store(x, handle=handle)
    h = _target(x, handle)
    got = _native.act8_store(h.address, h.device, x)
    if type(got) is int:
        h._raise(got, "act8_store")
    return got


def act8_restore(codes, scales, *, dtype=torch.bfloat16, handle=None, stream=None):
    """The values that act8_store kept, [rows, cols] in ``dtype``."""
    if stream is not None:
        with torch.cuda.stream(stream):  # torch ties outputs and scratch to it
            return act8_restore(codes, scales, dtype=dtype, handle=handle)
    h = _target(codes, handle)
    got = _native.act8_restore(h.address, h.device, codes, scales, dtype)
    if type(got) is int:
        h._raise(got, "act8_restore")
    return got


def act8_weight_grad(dy, codes, scales, *, add=None, out=None, dtype=None, handle=None, stream=None):
    """dw [out, cols] = dy^T x (+ add) of a linear layer y = x w^T whose
    input x is kept in 8 bits.

    dy: bf16 [rows, out]; add: the gradient so far; out: where dw is written
    (``out=add`` adds in place); dtype: float32 (default) or bfloat16, that
    of add and out if they are given."""
    if stream is not None:
        with torch.cuda.stream(stream):  # torch ties outputs and scratch to it
            return act8_weight_grad(dy, codes, scales, add=add, out=out, dtype=dtype, handle=handle)
    h = _target(dy, handle)
    got = _native.act8_weight_grad(h.address, h.device, dy, codes, scales, add, out, dtype)
    if type(got) is int:
        h._raise(got, "act8_weight_grad")
    return got
