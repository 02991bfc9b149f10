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

import torch

from . import _binding
from ._binding import MUON_BF16, MUON_F16, MUON_F32, MuonAttentionC

BLOCK = 128                       # columns that share one scale

_CODE = {torch.float32: MUON_F32, torch.bfloat16: MUON_BF16, torch.float16: MUON_F16}


def _code(t: torch.Tensor, what: str, allowed=(torch.float32, torch.bfloat16, torch.float16)) -> int:
    if t.dtype not in allowed:
        raise ValueError(f"{what} must be one of {', '.join(str(d) for d in allowed)}, not {t.dtype}")
    return _CODE[t.dtype]


def _cuda(what: str, *tensors):
    """Every tensor (None aside) on one CUDA device."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{what} must be CUDA tensors")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{what} must be on one device")
    return dev


class _Call:
    """The handle and the stream of one call; scratch and outputs are
    allocated inside it, so that torch ties them to that stream."""

    __slots__ = ("h", "lib", "stream", "_ctx")

    def __init__(self, dev, handle, stream):
        self.h = handle or _binding.default_handle(dev.index)
        if self.h.device != dev.index:
            raise ValueError(f"the handle is on device {self.h.device}, the tensors on {dev.index}")
        self.lib = self.h._lib
        self._ctx = None if stream is None else torch.cuda.stream(stream)
        self.stream = (torch.cuda.current_stream(dev) if stream is None else stream).cuda_stream

    def __enter__(self):
        if self._ctx is not None:
            self._ctx.__enter__()
        return self

    def __exit__(self, *exc):
        if self._ctx is not None:
            self._ctx.__exit__(*exc)

    def check(self, status: int, what: str):
        if status != 0:
            self.h._raise(status, what)


def _rows(t: torch.Tensor, what: str):
    """(tensor, rows, row stride) of [.., cols] seen as rows: the last
    dimension contiguous, the others with one stride between rows.  Anything
    else is copied once."""
    if t.dim() == 0:
        raise ValueError(f"{what} must have at least one dimension")
    cols = t.shape[-1]
    if t.dim() == 2 and (t.stride(1) == 1 or cols <= 1) and (t.stride(0) >= cols or t.shape[0] <= 1):
        return t, t.shape[0], max(t.stride(0), cols)
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
def _affine(t, what, x, cols):
    if t is None:
        return None
    if t.dim() != 1 or t.shape[0] != cols or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous vector of {cols} elements")
    if t.dtype not in (torch.float32, x.dtype):
        raise ValueError(f"{what} must be float32 or {x.dtype}")
    return t


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5, handle=None, stream=None):
    """Layer norm over the last dimension: ``(y, mean, rstd)``.

    x: [.., cols] fp32, bf16 or fp16, cols up to 16384; weight and bias:
    [cols], fp32 or x's type, or None (ones, zeros).  y has x's type and
    shape, mean and rstd (fp32, x.shape[:-1]) are what the backward pass
    takes."""
    dev = _cuda("x, weight and bias", x, weight, bias)
    code = _code(x, "x")
    cols = x.shape[-1] if x.dim() else 0
    weight, bias = _affine(weight, "weight", x, cols), _affine(bias, "bias", x, cols)
    w = weight if weight is not None else bias
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise ValueError("weight and bias must have one type")
    with _Call(dev, handle, stream) as c:
        xr, rows, ldx = _rows(x, "x")
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
        c.check(c.lib.muon_layer_norm_forward(
            c.h.ptr, xr.data_ptr(), ldx, weight.data_ptr() if weight is not None else None,
            bias.data_ptr() if bias is not None else None, y.data_ptr(), cols, mean.data_ptr(), rstd.data_ptr(), rows,
            cols, code, _CODE[w.dtype] if w is not None else MUON_F32, eps, c.stream), "muon_layer_norm_forward")
    return y, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight=None, *, handle=None, stream=None):
    """``(dx, dweight, dbias)`` of layer_norm: dx in x's type, dweight and
    dbias fp32 [cols], summed over all rows in a fixed order."""
    dev = _cuda("dy, x, mean, rstd and weight", dy, x, mean, rstd, weight)
    code = _code(x, "x")
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError("dy must have x's shape and type")
    for t, what in ((mean, "mean"), (rstd, "rstd")):
        if t.dtype != torch.float32 or t.shape != x.shape[:-1] or not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous float32 of shape {tuple(x.shape[:-1])}")
    cols = x.shape[-1]
    weight = _affine(weight, "weight", x, cols)
    with _Call(dev, handle, stream) as c:
        xr, rows, ldx = _rows(x, "x")
        gr, _, ldg = _rows(dy, "dy")
        need = ctypes.c_uint64()
        c.check(c.lib.muon_layer_norm_workspace(c.h.ptr, rows, cols, ctypes.byref(need)), "muon_layer_norm_workspace")
        ws = torch.empty(need.value, dtype=torch.uint8, device=dev)
        dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
        dwb = torch.empty((2, cols), dtype=torch.float32, device=dev)
        c.check(c.lib.muon_layer_norm_backward(
            c.h.ptr, gr.data_ptr(), ldg, xr.data_ptr(), ldx, mean.data_ptr(), rstd.data_ptr(),
            weight.data_ptr() if weight is not None else None, dx.data_ptr(), cols, dwb.data_ptr(),
            dwb.data_ptr() + 4 * cols, rows, cols, code, _CODE[weight.dtype] if weight is not None else MUON_F32,
            ws.data_ptr(), need.value, c.stream), "muon_layer_norm_backward")
    return dx, dwb[0], dwb[1]


# ----------------------------------------------------------------- attention
def _heads(t, what, packed):
    """Strides (batch, token, head) of [batch, token, head, dim], or of
    [token, head, dim] when packed."""
    want = 3 if packed else 4
    if t.dim() != want:
        raise ValueError(f"{what} must have {want} dimensions")
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] != 1:
        raise ValueError(f"{what} must be contiguous in its last dimension")
    return (0, st[0], st[1]) if packed else st[:3]


def _attention_args(q, k, v, causal, window, scale, cu_q, cu_k):
    packed = cu_q is not None or cu_k is not None
    code = _code(q, "q", (torch.bfloat16, torch.float16))
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k and v must have one type")
    a = MuonAttentionC()
    a.q_stride[:], a.k_stride[:], a.v_stride[:] = (_heads(t, n, packed) for t, n in ((q, "q"), (k, "k"), (v, "v")))
    if k.shape != v.shape or q.shape[-1] != k.shape[-1] or (not packed and q.shape[0] != k.shape[0]):
        raise ValueError(f"shapes do not go together: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    if packed:
        if cu_q is None or cu_k is None:
            raise ValueError("cu_seqlens_q and cu_seqlens_k go together")
        for t, what in ((cu_q, "cu_seqlens_q"), (cu_k, "cu_seqlens_k")):
            if t.dtype != torch.int32 or t.dim() != 1 or t.shape[0] < 1 or not t.is_contiguous():
                raise ValueError(f"{what} must be a contiguous int32 vector of at least one element")
        if cu_q.shape != cu_k.shape:
            raise ValueError("cu_seqlens_q and cu_seqlens_k must have one length")
        a.batch = cu_q.shape[0] - 1
        a.cu_seqlens_q, a.cu_seqlens_k = cu_q.data_ptr(), cu_k.data_ptr()
    else:
        a.batch = q.shape[0]
    a.sq, a.heads, a.dim = q.shape[-3:]
    a.sk, a.kv_heads = k.shape[-3:-1]
    a.q, a.k, a.v = q.data_ptr(), k.data_ptr(), v.data_ptr()
    a.causal, a.window, a.dtype = 1 if causal else 0, int(window), code
    a.scale = 1.0 / math.sqrt(a.dim) if scale is None and a.dim else float(scale or 0.0)
    return a, packed


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
    ``window`` of them.  scale: 1 / sqrt(dim) by default.
    o has q's shape and type (a query that sees no key: 0); lse is fp32
    [batch, heads, sq] or [heads, tokens] (there: -inf)."""
    dev = _cuda("q, k, v and the offsets", q, k, v, cu_seqlens_q, cu_seqlens_k)
    a, packed = _attention_args(q, k, v, causal, window, scale, cu_seqlens_q, cu_seqlens_k)
    with _Call(dev, handle, stream) as c:
        o = torch.empty(q.shape, dtype=q.dtype, device=dev)
        lse = torch.empty((a.heads, a.sq) if packed else (a.batch, a.heads, a.sq), dtype=torch.float32, device=dev)
        a.o, a.lse = o.data_ptr(), lse.data_ptr()
        a.o_stride[:] = _heads(o, "o", packed)
        c.check(c.lib.muon_attention_forward(c.h.ptr, ctypes.byref(a), c.stream), "muon_attention_forward")
    return o, lse


def attention_backward(do, q, k, v, o, lse, *, causal: bool = False, window: int = 0, scale=None, cu_seqlens_q=None,
                       cu_seqlens_k=None, handle=None, stream=None):
    """``(dq, dk, dv)`` of attention, from its output and lse: the
    probabilities are recomputed, nothing of size sq x sk is kept.  dk and dv
    are summed over the query heads that share them, in a fixed order."""
    dev = _cuda("do, q, k, v, o, lse and the offsets", do, q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k)
    a, packed = _attention_args(q, k, v, causal, window, scale, cu_seqlens_q, cu_seqlens_k)
    for t, what in ((do, "do"), (o, "o")):
        if t.shape != q.shape or t.dtype != q.dtype:
            raise ValueError(f"{what} must have q's shape and type")
    if lse.dtype != torch.float32 or lse.shape != ((a.heads, a.sq) if packed else (a.batch, a.heads, a.sq)) \
            or not lse.is_contiguous():
        raise ValueError("lse must be the contiguous float32 tensor that attention returned")
    with _Call(dev, handle, stream) as c:
        if do.stride(-1) != 1 or any(s % 8 for s in do.stride()[:-1]):
            do = do.contiguous()         # autograd hands over expanded gradients
        dq = torch.empty(q.shape, dtype=q.dtype, device=dev)
        dk = torch.empty(k.shape, dtype=q.dtype, device=dev)
        dv = torch.empty(v.shape, dtype=q.dtype, device=dev)
        a.o, a.lse, a.dout = o.data_ptr(), lse.data_ptr(), do.data_ptr()
        a.dq, a.dk, a.dv = dq.data_ptr(), dk.data_ptr(), dv.data_ptr()
        a.o_stride[:], a.dout_stride[:] = _heads(o, "o", packed), _heads(do, "do", packed)
        a.dq_stride[:], a.dk_stride[:], a.dv_stride[:] = (_heads(t, "", packed) for t in (dq, dk, dv))
        need = ctypes.c_uint64()
        c.check(c.lib.muon_attention_workspace(c.h.ptr, ctypes.byref(a), ctypes.byref(need)),
                "muon_attention_workspace")
        ws = torch.empty(need.value, dtype=torch.uint8, device=dev)
        c.check(c.lib.muon_attention_backward(c.h.ptr, ctypes.byref(a), ws.data_ptr(), need.value, c.stream),
                "muon_attention_backward")
    return dq, dk, dv


# --------------------------------------------------- activations in 8 bits
def _blocks(cols: int) -> int:
    return -(-cols // BLOCK)


def act8_store(x, *, handle=None, stream=None):
    """x [rows, cols] (fp32, bf16, fp16) in 8 bits: ``(codes, scales)``.

    codes: float8_e4m3fn [rows, cols]; scales: uint8 [ceil(cols / 128),
    rows], one exponent a row and 128 columns: the stored value is code times
    2^(scale - 127), with the smallest power of two that fits the block's
    largest value (at least 2^-111).  A block with a NaN or an infinity is
    stored as scale 255, codes 0 and stands for NaN.  Both are views of
    padded storage (whole blocks, 16 rows), which act8_weight_grad reads in
    place; copies in other layouts are taken too, at the cost of one more
    copy."""
    dev = _cuda("x", x)
    code = _code(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    with _Call(dev, handle, stream) as c:
        xr, rows, ldx = _rows(x, "x")
        cols = x.shape[1]
        ldc, lds = _blocks(cols) * BLOCK, -(-rows // 16) * 16
        codes = torch.empty((rows, ldc), dtype=torch.float8_e4m3fn, device=dev)
        scales = torch.empty((_blocks(cols), lds), dtype=torch.uint8, device=dev)
        c.check(c.lib.muon_act8_store(c.h.ptr, xr.data_ptr(), ldx, codes.data_ptr(), ldc, scales.data_ptr(), lds,
                                      rows, cols, code, c.stream), "muon_act8_store")
    return codes[:, :cols], scales[:, :rows]


def _act8_operands(codes, scales):
    """codes and scales as the kernels read them (padded rows), copied if
    they come in another layout, and their row strides."""
    if codes.dim() != 2 or codes.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise ValueError("codes must be 2-D float8_e4m3fn")
    rows, cols = codes.shape
    if scales.dtype != torch.uint8 or tuple(scales.shape) != (_blocks(cols), rows):
        raise ValueError(f"scales must be uint8 of shape {(_blocks(cols), rows)}")
    if rows and cols:
        if codes.stride(1) != 1 or codes.stride(0) % BLOCK or codes.stride(0) < cols or codes.data_ptr() % 16:
            wide = torch.zeros((rows, _blocks(cols) * BLOCK), dtype=torch.uint8, device=codes.device)
            wide[:, :cols] = codes.view(torch.uint8) if codes.dtype != torch.uint8 else codes
            codes = wide
        if scales.stride(1) != 1 or scales.stride(0) % 16 or scales.stride(0) < rows or scales.data_ptr() % 16:
            tall = torch.zeros((scales.shape[0], -(-rows // 16) * 16), dtype=torch.uint8, device=codes.device)
            tall[:, :rows] = scales
            scales = tall
    return codes, scales, rows, cols, codes.stride(0), scales.stride(0) if scales.dim() == 2 else 0


def act8_restore(codes, scales, *, dtype=torch.bfloat16, handle=None, stream=None):
    """The values that act8_store kept, [rows, cols] in ``dtype``."""
    dev = _cuda("codes and scales", codes, scales)
    if dtype not in _CODE:
        raise ValueError(f"unsupported dtype {dtype}")
    with _Call(dev, handle, stream) as c:
        codes, scales, rows, cols, ldc, lds = _act8_operands(codes, scales)
        out = torch.empty((rows, cols), dtype=dtype, device=dev)
        c.check(c.lib.muon_act8_restore(c.h.ptr, codes.data_ptr(), ldc, scales.data_ptr(), lds, out.data_ptr(), cols,
                                        rows, cols, _CODE[dtype], c.stream), "muon_act8_restore")
    return out


def act8_weight_grad(dy, codes, scales, *, add=None, out=None, dtype=None, handle=None, stream=None):
    """dw [out, cols] = dy^T x (+ add) of a linear layer y = x w^T whose
    input x is kept in 8 bits.

    dy: bf16 [rows, out]; add: the gradient so far; out: where dw is written
    (``out=add`` adds in place); dtype: float32 (default) or bfloat16, that
    of add and out if they are given."""
    dev = _cuda("dy, codes, scales, add and out", dy, codes, scales, add, out)
    _code(dy, "dy", (torch.bfloat16,))
    if dy.dim() != 2 or codes.dim() != 2 or dy.shape[0] != codes.shape[0]:
        raise ValueError("dy must be [rows, out] and codes [rows, cols]")
    shape = (dy.shape[1], codes.shape[1])
    for t, what in ((add, "add"), (out, "out")):
        if t is None:
            continue
        if tuple(t.shape) != shape:
            raise ValueError(f"{what} must have shape {shape}")
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"{what} must have type {dtype}")
        dtype = t.dtype
        if t.stride(1) != 1 and shape[1] > 1 or t.stride(0) < shape[1] and shape[0] > 1:
            raise ValueError(f"{what} must have contiguous rows")
    dtype = torch.float32 if dtype is None else dtype
    if dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("dtype must be float32 or bfloat16")
    with _Call(dev, handle, stream) as c:
        dyr, _, ldy = _rows(dy, "dy")
        xc, sc, rows, cols, ldc, lds = _act8_operands(codes, scales)
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=dev)
        need = ctypes.c_uint64()
        c.check(c.lib.muon_act8_weight_grad_workspace(c.h.ptr, dyr.data_ptr(), ldy, rows, cols, shape[0],
                                                      ctypes.byref(need)),
                "muon_act8_weight_grad_workspace")
        ws = torch.empty(need.value, dtype=torch.uint8, device=dev) if need.value else None
        c.check(c.lib.muon_act8_weight_grad(
            c.h.ptr, dyr.data_ptr(), ldy, xc.data_ptr(), ldc, sc.data_ptr(), lds,
            add.data_ptr() if add is not None else None, max(add.stride(0), cols) if add is not None else cols,
            out.data_ptr(), max(out.stride(0), cols), rows, cols, shape[0], _CODE[dtype],
            ws.data_ptr() if ws is not None else None, need.value, c.stream), "muon_act8_weight_grad")
    return out
