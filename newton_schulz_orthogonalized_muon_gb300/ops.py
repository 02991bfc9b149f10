"""Training operators around the Muon step, as calls on torch tensors.

Layer norm, attention (with the backward pass that recomputes the
probabilities) and activations kept in 8 bits, each a thin call of the C ABI
in include/muon.h: the tensors are checked, outputs and scratch are allocated
by torch on the stream that the kernels run on, and a non-OK status raises
MuonError.  ``nn`` wraps them for autograd.

Every function takes ``stream`` (default: the current stream of the tensors'
device) and ``handle`` (default: that device's handle).  Inputs that are
written on another stream have to be ready there, as for any call.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import _binding
from ._binding import MUON_BF16, MUON_F16, MUON_F32, MuonAttentionC

BLOCK = 128                       # columns that share one scale

_CODE = {torch.float32: MUON_F32, torch.bfloat16: MUON_BF16, torch.float16: MUON_F16}
_CODE16 = {torch.bfloat16: MUON_BF16, torch.float16: MUON_F16}
_CODE_BF16 = {torch.bfloat16: MUON_BF16}


def _code(t: torch.Tensor, what: str, allowed=_CODE) -> int:
    code = allowed.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be one of {', '.join(str(d) for d in allowed)}, not {t.dtype}")
    return code


def _device(what: str, first, *rest) -> int:
    """The index of the CUDA device that all the tensors (None aside) are on."""
    try:
        dev = first.get_device()         # -1: not on a GPU
        for t in rest:
            if t is not None and t.get_device() != dev:
                dev = -1
    except AttributeError:
        dev = -1
    if dev < 0:
        raise ValueError(f"{what} must be CUDA tensors on one device")
    return dev


# the current stream of a device as an integer; the private call skips the
# construction of a Stream object (2 us of a 20 us call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _handle(dev: int, handle):
    if handle is None:
        return _binding.default_handle(dev)
    if handle.device != dev:
        raise ValueError(f"the handle is on device {handle.device}, the tensors on {dev}")
    return handle


def _rows(t: torch.Tensor, what: str):
    """(tensor, rows, row stride) of [.., cols] seen as rows: the last
    dimension contiguous, the others with one stride between rows.  Anything
    else is copied once."""
    shape = t.shape
    if len(shape) == 0:
        raise ValueError(f"{what} must have at least one dimension")
    cols = shape[-1]
    if len(shape) == 2:
        ld, one = t.stride()
        if one == 1 or cols <= 1:
            if ld >= cols or shape[0] <= 1:
                return t, shape[0], max(ld, cols)
    if not t.is_contiguous():
        try:
            flat = t.view(-1, cols)
            if flat.stride(1) == 1 and flat.stride(0) >= cols:
                return flat, flat.shape[0], flat.stride(0)
        except RuntimeError:
            pass
        t = t.contiguous()
    return t, t.numel() // cols if cols else 0, cols


# ---------------------------------------------------------------- layer norm
def _affine(t, what, dtype, cols):
    """Pointer and type code of a weight or bias vector."""
    if t is None:
        return None, MUON_F32
    if t.shape != (cols,) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous vector of {cols} elements")
    own = t.dtype
    if own is not torch.float32 and own is not dtype:
        raise ValueError(f"{what} must be float32 or {dtype}")
    return t.data_ptr(), _CODE[own]


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5, handle=None, stream=None):
    """Layer norm over the last dimension: ``(y, mean, rstd)``.

    x: [.., cols] fp32, bf16 or fp16, cols up to 16384; weight and bias:
    [cols], fp32 or x's type, or None (ones, zeros).  y has x's type and
    shape, mean and rstd (fp32, x.shape[:-1]) are what the backward pass
    takes."""
    if stream is not None:
        with torch.cuda.stream(stream):  # torch ties outputs and scratch to it
            return layer_norm(x, weight, bias, eps=eps, handle=handle)
    dev = _device("x, weight and bias", x, weight, bias)
    code = _code(x, "x")
    xr, rows, ldx = _rows(x, "x")
    shape, dtype = x.shape, x.dtype
    cols = shape[-1]
    wptr, wcode = _affine(weight, "weight", dtype, cols)
    bptr, bcode = _affine(bias, "bias", dtype, cols)
    if wptr is not None and bptr is not None and wcode != bcode:
        raise ValueError("weight and bias must have one type")
    h = _handle(dev, handle)
    where = x.device
    y = torch.empty(shape, dtype=dtype, device=where)
    mean = torch.empty(shape[:-1], dtype=torch.float32, device=where)
    rstd = torch.empty_like(mean)
    st = h._lib.muon_layer_norm_forward(h.ptr, xr.data_ptr(), ldx, wptr, bptr, y.data_ptr(), cols, mean.data_ptr(),
                                        rstd.data_ptr(), rows, cols, code, bcode if wptr is None else wcode, eps,
                                        _raw_stream(dev))
    if st:
        h._raise(st, "muon_layer_norm_forward")
    return y, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight=None, *, handle=None, stream=None):
    """``(dx, dweight, dbias)`` of layer_norm: dx in x's type, dweight and
    dbias fp32 [cols], summed over all rows in a fixed order."""
    if stream is not None:
        with torch.cuda.stream(stream):  # torch ties outputs and scratch to it
            return layer_norm_backward(dy, x, mean, rstd, weight, handle=handle)
    dev = _device("x, dy, mean, rstd and weight", x, dy, mean, rstd, weight)
    code = _code(x, "x")
    shape = x.shape
    if dy.shape != shape or dy.dtype != x.dtype:
        raise ValueError("dy must have x's shape and type")
    xr, rows, ldx = _rows(x, "x")
    gr, _, ldg = _rows(dy, "dy")
    outer = shape[:-1]
    for t, what in ((mean, "mean"), (rstd, "rstd")):
        if t.dtype is not torch.float32 or t.shape != outer or not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous float32 of shape {tuple(outer)}")
    cols = shape[-1]
    wptr, wcode = _affine(weight, "weight", x.dtype, cols)
    h = _handle(dev, handle)
    lib, need = h._lib, ctypes.c_uint64()
    st = lib.muon_layer_norm_workspace(h.ptr, rows, cols, ctypes.byref(need))
    if st:
        h._raise(st, "muon_layer_norm_workspace")
    need = need.value
    where = x.device
    ws = torch.empty(need, dtype=torch.uint8, device=where)
    dx = torch.empty(shape, dtype=x.dtype, device=where)
    dw = torch.empty(cols, dtype=torch.float32, device=where)
    db = torch.empty_like(dw)
    st = lib.muon_layer_norm_backward(h.ptr, gr.data_ptr(), ldg, xr.data_ptr(), ldx, mean.data_ptr(), rstd.data_ptr(),
                                      wptr, dx.data_ptr(), cols, dw.data_ptr(), db.data_ptr(), rows, cols, code,
                                      wcode, ws.data_ptr(), need, _raw_stream(dev))
    if st:
        h._raise(st, "muon_layer_norm_backward")
    return dx, dw, db


# ----------------------------------------------------------------- attention
def _strides(t, what, packed):
    """Strides (batch, token, head) of [batch, token, head, dim], or of
    [token, head, dim] when packed."""
    st = t.stride()
    if len(st) != (3 if packed else 4):
        raise ValueError(f"{what} must have {3 if packed else 4} dimensions")
    if st[-1] != 1 and t.shape[-1] != 1:
        raise ValueError(f"{what} must be contiguous in its last dimension")
    return (0, st[0], st[1]) if packed else st[:3]


# muon_attention_t: eleven pointers, eight times three strides, nine integers, the scale
_ATTENTION = struct.Struct("@11P24q9if")
assert _ATTENTION.size == ctypes.sizeof(MuonAttentionC)


class _Attention:
    """The checked arguments of an attention call."""

    __slots__ = ("packed", "strides", "ints", "scale", "cu", "like_q", "like_k", "lse_shape")

    def __init__(self, q, k, v, causal, window, scale, cu_q, cu_k):
        packed = self.packed = cu_q is not None or cu_k is not None
        code = _code(q, "q", _CODE16)
        if k.dtype is not q.dtype or v.dtype is not q.dtype:
            raise ValueError("q, k and v must have one type")
        self.strides = (*_strides(q, "q", packed), *_strides(k, "k", packed), *_strides(v, "v", packed))
        qs, ks = q.shape, k.shape
        if ks != v.shape or qs[-1] != ks[-1] or (not packed and qs[0] != ks[0]):
            raise ValueError(f"shapes do not go together: q {tuple(qs)}, k {tuple(ks)}, v {tuple(v.shape)}")
        if packed:
            if cu_q is None or cu_k is None:
                raise ValueError("cu_seqlens_q and cu_seqlens_k go together")
            for t, what in ((cu_q, "cu_seqlens_q"), (cu_k, "cu_seqlens_k")):
                if t.dtype != torch.int32 or t.dim() != 1 or t.shape[0] < 1 or not t.is_contiguous():
                    raise ValueError(f"{what} must be a contiguous int32 vector of at least one element")
            if cu_q.shape != cu_k.shape:
                raise ValueError("cu_seqlens_q and cu_seqlens_k must have one length")
            batch = cu_q.shape[0] - 1
            self.cu = (cu_q.data_ptr(), cu_k.data_ptr())
        else:
            batch = qs[0]
            self.cu = (0, 0)
        sq, heads, dim = qs[-3:]
        sk, kv_heads = ks[-3], ks[-2]
        # strides of contiguous outputs
        row = heads * dim
        self.like_q = (sq * row, row, dim)
        row = kv_heads * dim
        self.like_k = (sk * row, row, dim)
        self.lse_shape = (heads, sq) if packed else (batch, heads, sq)
        self.ints = (batch, sq, sk, heads, kv_heads, dim, 1 if causal else 0, int(window), code)
        if max(self.ints) >= 1 << 31 or min(self.ints) < 0:
            raise ValueError("negative or oversized shape or window")
        self.scale = float(scale) if scale is not None else 1.0 / math.sqrt(dim) if dim else 0.0

    def pack(self, pointers, strides):
        return _ATTENTION.pack(*pointers, *self.cu, *self.strides, *strides, *self.ints, self.scale)


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
    [batch, heads, sq] or [heads, tokens] (there: -inf)."""
    if stream is not None:
        with torch.cuda.stream(stream):  # torch ties outputs and scratch to it
            return attention(q, k, v, causal=causal, window=window, scale=scale, cu_seqlens_q=cu_seqlens_q,
                             cu_seqlens_k=cu_seqlens_k, handle=handle)
    dev = _device("q, k, v and the offsets", q, k, v, cu_seqlens_q, cu_seqlens_k)
    a = _Attention(q, k, v, causal, window, scale, cu_seqlens_q, cu_seqlens_k)
    h = _handle(dev, handle)
    where = q.device
    o = torch.empty(q.shape, dtype=q.dtype, device=where)
    lse = torch.empty(a.lse_shape, dtype=torch.float32, device=where)
    args = a.pack((q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), 0, 0, 0, 0),
                  a.like_q + _NO_STRIDES)
    st = h._lib.muon_attention_forward(h.ptr, args, _raw_stream(dev))
    if st:
        h._raise(st, "muon_attention_forward")
    return o, lse


_NO_STRIDES = (0,) * 12


def attention_backward(do, q, k, v, o, lse, *, causal: bool = False, window: int = 0, scale=None, cu_seqlens_q=None,
                       cu_seqlens_k=None, handle=None, stream=None):
    """``(dq, dk, dv)`` of attention, from its output and lse: the
    probabilities are recomputed, nothing of size sq x sk is kept.  dk and dv
    are summed over the query heads that share them, in a fixed order."""
    if stream is not None:
        with torch.cuda.stream(stream):  # torch ties outputs and scratch to it
            return attention_backward(do, q, k, v, o, lse, causal=causal, window=window, scale=scale,
                                      cu_seqlens_q=cu_seqlens_q, cu_seqlens_k=cu_seqlens_k, handle=handle)
    dev = _device("q, k, v, do, o, lse and the offsets", q, k, v, do, o, lse, cu_seqlens_q, cu_seqlens_k)
    a = _Attention(q, k, v, causal, window, scale, cu_seqlens_q, cu_seqlens_k)
    shape, dtype = q.shape, q.dtype
    if do.shape != shape or o.shape != shape or do.dtype is not dtype or o.dtype is not dtype:
        raise ValueError("do and o must have q's shape and type")
    if lse.dtype is not torch.float32 or lse.shape != a.lse_shape or not lse.is_contiguous():
        raise ValueError("lse must be the contiguous float32 tensor that attention returned")
    h = _handle(dev, handle)
    if not do.is_contiguous():
        st = do.stride()
        if st[-1] != 1 or 0 in st or any(s % 8 for s in st[:-1]):
            do = do.contiguous()         # autograd hands over expanded gradients
    where = q.device
    dq = torch.empty(shape, dtype=dtype, device=where)
    dk = torch.empty(k.shape, dtype=dtype, device=where)
    dv = torch.empty_like(dk)
    args = a.pack((q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), do.data_ptr(),
                   dq.data_ptr(), dk.data_ptr(), dv.data_ptr()),
                  (*_strides(o, "o", a.packed), *_strides(do, "do", a.packed), *a.like_q, *a.like_k, *a.like_k))
    lib = h._lib
    need = ctypes.c_uint64()
    st = lib.muon_attention_workspace(h.ptr, args, ctypes.byref(need))
    if st:
        h._raise(st, "muon_attention_workspace")
    need = need.value
    ws = torch.empty(need, dtype=torch.uint8, device=where)
    st = lib.muon_attention_backward(h.ptr, args, ws.data_ptr(), need, _raw_stream(dev))
    if st:
        h._raise(st, "muon_attention_backward")
    return dq, dk, dv


# --------------------------------------------------- activations in 8 bits
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
    dev = _device("x", x)
    code = _code(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    xr, rows, ldx = _rows(x, "x")
    cols = x.shape[1]
    h = _handle(dev, handle)
    blocks, lds = -(-cols // BLOCK), -(-rows // 16) * 16
    ldc = blocks * BLOCK
    where = x.device
    codes = torch.empty_strided((rows, cols), (ldc, 1), dtype=torch.float8_e4m3fn, device=where)
    scales = torch.empty_strided((blocks, rows), (lds, 1), dtype=torch.uint8, device=where)
    st = h._lib.muon_act8_store(h.ptr, xr.data_ptr(), ldx, codes.data_ptr(), ldc, scales.data_ptr(), lds, rows, cols,
                                code, _raw_stream(dev))
    if st:
        h._raise(st, "muon_act8_store")
    return codes, scales


def _act8_operands(codes, scales):
    """codes and scales as the kernels read them (padded rows), copied if
    they come in another layout, their shape and row strides."""
    if codes.dim() != 2 or (codes.dtype is not torch.float8_e4m3fn and codes.dtype is not torch.uint8):
        raise ValueError("codes must be 2-D float8_e4m3fn")
    rows, cols = codes.shape
    blocks = -(-cols // BLOCK)
    if scales.dtype is not torch.uint8 or scales.shape != (blocks, rows):
        raise ValueError(f"scales must be uint8 of shape {(blocks, rows)}")
    ldc, lds = codes.stride(), scales.stride()
    if rows and cols:
        if ldc[1] != 1 or ldc[0] % BLOCK or ldc[0] < cols or codes.data_ptr() % 16:
            wide = torch.zeros((rows, blocks * BLOCK), dtype=torch.uint8, device=codes.device)
            wide[:, :cols] = codes.view(torch.uint8) if codes.dtype is not torch.uint8 else codes
            codes, ldc = wide, wide.stride()
        if lds[1] != 1 or lds[0] % 16 or lds[0] < rows or scales.data_ptr() % 16:
            tall = torch.zeros((blocks, -(-rows // 16) * 16), dtype=torch.uint8, device=codes.device)
            tall[:, :rows] = scales
            scales, lds = tall, tall.stride()
    return codes, scales, rows, cols, ldc[0], lds[0]


def act8_restore(codes, scales, *, dtype=torch.bfloat16, handle=None, stream=None):
    """The values that act8_store kept, [rows, cols] in ``dtype``."""
    if stream is not None:
        with torch.cuda.stream(stream):  # torch ties outputs and scratch to it
            return act8_restore(codes, scales, dtype=dtype, handle=handle)
    dev = _device("codes and scales", codes, scales)
    code = _CODE.get(dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {dtype}")
    h = _handle(dev, handle)
    codes, scales, rows, cols, ldc, lds = _act8_operands(codes, scales)
    out = torch.empty((rows, cols), dtype=dtype, device=scales.device)
    st = h._lib.muon_act8_restore(h.ptr, codes.data_ptr(), ldc, scales.data_ptr(), lds, out.data_ptr(), cols, rows,
                                  cols, code, _raw_stream(dev))
    if st:
        h._raise(st, "muon_act8_restore")
    return out


def act8_weight_grad(dy, codes, scales, *, add=None, out=None, dtype=None, handle=None, stream=None):
    """dw [out, cols] = dy^T x (+ add) of a linear layer y = x w^T whose
    input x is kept in 8 bits.

    dy: bf16 [rows, out]; add: the gradient so far; out: where dw is written
    (``out=add`` adds in place); dtype: float32 (default) or bfloat16, that
    of add and out if they are given."""
    if stream is not None:
        with torch.cuda.stream(stream):  # torch ties outputs and scratch to it
            return act8_weight_grad(dy, codes, scales, add=add, out=out, dtype=dtype, handle=handle)
    dev = _device("dy, codes, scales, add and out", dy, codes, scales, add, out)
    _code(dy, "dy", _CODE_BF16)
    if dy.dim() != 2 or codes.dim() != 2 or dy.shape[0] != codes.shape[0]:
        raise ValueError("dy must be [rows, out] and codes [rows, cols]")
    shape = (dy.shape[1], codes.shape[1])
    ld = [shape[1], shape[1]]
    for i, (t, what) in enumerate(((add, "add"), (out, "out"))):
        if t is None:
            continue
        if t.shape != shape:
            raise ValueError(f"{what} must have shape {shape}")
        if dtype is not None and t.dtype is not dtype:
            raise ValueError(f"{what} must have type {dtype}")
        dtype = t.dtype
        st = t.stride()
        if st[1] != 1 and shape[1] > 1 or st[0] < shape[1] and shape[0] > 1:
            raise ValueError(f"{what} must have contiguous rows")
        ld[i] = max(st[0], shape[1])
    dtype = torch.float32 if dtype is None else dtype
    if dtype is not torch.float32 and dtype is not torch.bfloat16:
        raise ValueError("dtype must be float32 or bfloat16")
    h = _handle(dev, handle)
    dyr, _, ldy = _rows(dy, "dy")
    xc, sc, rows, cols, ldc, lds = _act8_operands(codes, scales)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dy.device)
    lib, need = h._lib, ctypes.c_uint64()
    st = lib.muon_act8_weight_grad_workspace(h.ptr, dyr.data_ptr(), ldy, rows, cols, shape[0], ctypes.byref(need))
    if st:
        h._raise(st, "muon_act8_weight_grad_workspace")
    ws = torch.empty(need.value, dtype=torch.uint8, device=dy.device) if need.value else None
    st = lib.muon_act8_weight_grad(h.ptr, dyr.data_ptr(), ldy, xc.data_ptr(), ldc, sc.data_ptr(), lds,
                                   add.data_ptr() if add is not None else None, ld[0], out.data_ptr(), ld[1], rows,
                                   cols, shape[0], _CODE[dtype], ws.data_ptr() if ws is not None else None,
                                   need.value, _raw_stream(dev))
    if st:
        h._raise(st, "muon_act8_weight_grad")
    return out
