"""Weights in 4 bits with a scale per group of 32, 64 or 128 values of a row, and products of few rows with them.

  int4_quantize(W, group)                           (q, s, zeros): W is about (q - zero) s
  int4_dequantize(q, s, zeros)                      W again, for the products of many rows
  dp_gemm_fwd_int4(X, q, s, zeros)                  Y = X W^T
  dp_gemm_fwd_int4_grouped(X, q, s, offsets, zeros) Y[t] = X[t] W_e^T for the rows t of expert e

q [N, K/2] (uint8) holds two codes 0..15 a byte, the even column in the low half; s [N, K/group] is
bf16 or fp32; zeros [N, K/group] (uint8, 0..15) or None (8).  Experts add a dimension in front.  All
three are contiguous, as int4_quantize makes them; the group's size follows from their shapes.
"""
from __future__ import annotations

import torch

from . import _call as c

_U8 = torch.uint8
_BITS = {torch.int32: 32, torch.int64: 64}
_fn = {}


def _bind(L):
    P, I, S = c.P, c.I, c.S
    L.dp_int4_quantize.argtypes = [P, I, S, I, I, I, P, P, S, P, P]
    L.dp_int4_dequantize.argtypes = [P, P, S, P, I, I, I, P, I, S, P]
    L.dp_gemm_fwd_int4.argtypes = [P, I, P, P, S, P, I, P, I, I, I, I, S, P]
    L.dp_gemm_fwd_int4_grouped.argtypes = [P, I, P, P, S, P, I, P, S, P, I, I, I, I, I, S, P]
    names = ("dp_int4_quantize", "dp_int4_dequantize", "dp_gemm_fwd_int4", "dp_gemm_fwd_int4_grouped")
    _fn.update({name: getattr(L, name) for name in names})


def _row_stride(w, name, what, shape):
    """Leading dimension of [N, K] or [E, N, K], the rows of all experts equally far apart."""
    if len(shape) == 2:
        return c.ld(w, name, what, shape)
    if not w.is_contiguous():
        raise ValueError(f"{name}: {what} with experts must be contiguous")
    return shape[-1]


def int4_quantize(W, group=128, zeros=False, scale_dtype=c.BF16, stream=None):
    """(q, s, zeros or None) of W [N,K] or [E,N,K] (bf16 or fp32; K a multiple of the group): a symmetric
    range per group, or with ``zeros`` the group's own, which includes 0."""
    name = "int4_quantize"
    index = W.get_device()
    if index < 0:
        c.refuse_devices(name, {"W": W})
    f32 = W.dtype is c.F32
    if not f32 and W.dtype is not c.BF16:
        raise TypeError(f"{name}: W must be bfloat16 or float32")
    if scale_dtype is not c.BF16 and scale_dtype is not c.F32:
        raise TypeError(f"{name}: scale_dtype must be bfloat16 or float32")
    shape = W.shape
    if len(shape) not in (2, 3):
        raise ValueError(f"{name}: W must be [N, K] or [E, N, K]")
    if group not in (32, 64, 128) or shape[-1] % group or shape[-1] == 0:
        raise ValueError(f"{name}: group must be 32, 64 or 128 and divide K")
    ld, K, front = _row_stride(W, name, "W", shape), shape[-1], shape[:-1]
    if not _fn:
        c.load()

    def work(st):
        q = c.new((*front, K // 2), _U8)
        s = c.new((*front, K // group), scale_dtype)
        z = c.new((*front, K // group), _U8) if zeros else None
        code = _fn["dp_int4_quantize"](W.data_ptr(), ld, f32, front.numel(), K, group, q.data_ptr(), s.data_ptr(),
                                       scale_dtype is c.F32, None if z is None else z.data_ptr(), st)
        if code:
            c.check(code, name)
        return q, s, z

    return c.on_stream(index, stream, (W,), work)


def _weights(q, s, zeros, dims, name):
    """(N, K, group, whether the scales are fp32) of contiguous codes, scales and zero points."""
    front, width = q.shape[:-1], s.shape[-1] if s.dim() else 0
    K = 2 * q.shape[-1] if q.dim() else 0
    if q.dtype is not _U8 or (zeros is not None and zeros.dtype is not _U8):
        raise TypeError(f"{name}: codes and zeros must be uint8")
    f32 = s.dtype is c.F32
    if not f32 and s.dtype is not c.BF16:
        raise TypeError(f"{name}: scales must be bfloat16 or float32")
    if q.dim() not in dims or s.shape[:-1] != front or (zeros is not None and zeros.shape != s.shape):
        raise ValueError(f"{name}: codes [..., K/2], scales and zeros [..., K/group] must have the same rows")
    if not (q.is_contiguous() and s.is_contiguous() and (zeros is None or zeros.is_contiguous())):
        raise ValueError(f"{name}: codes, scales and zeros must be contiguous")
    group = K // width if width else 0
    if group not in (32, 64, 128) or group * width != K:
        raise ValueError(f"{name}: the scales' shape makes no groups of 32, 64 or 128")
    return front, K, group, f32


def int4_dequantize(q, s, zeros=None, out=None, out_dtype=c.BF16, stream=None):
    """W = (q - zero) s, [N,K] or [E,N,K]."""
    name = "int4_dequantize"
    index = q.get_device()
    if index < 0 or s.get_device() != index or (zeros is not None and zeros.get_device() != index):
        c.refuse_devices(name, {what: t for what, t in (("codes", q), ("scales", s), ("zeros", zeros)) if t is not None})
    front, K, group, f32 = _weights(q, s, zeros, (2, 3), name)
    if not _fn:
        c.load()

    def work(st):
        shape = (*front, K)
        w, code = c.output(out, shape, out_dtype, index, q.device, name)
        code = _fn["dp_int4_dequantize"](q.data_ptr(), s.data_ptr(), f32, None if zeros is None else zeros.data_ptr(), front.numel(), K,
                                         group, w.data_ptr(), _row_stride(w, name, "out", shape), code, st)
        if code:
            c.check(code, name)
        return w

    return c.on_stream(index, stream, (q, s, zeros, out), work)


def _rows(X, K, name):
    if X.dtype is not c.BF16:
        raise TypeError(f"{name}: X must be bfloat16")
    if X.dim() != 2 or X.shape[1] != K:
        raise ValueError(f"{name}: X must be [T, K] with the weights' K")
    return X.shape[0], c.ld(X, name, "X")


def dp_gemm_fwd_int4(X, q, s, zeros=None, out=None, out_dtype=c.BF16, stream=None):
    """Y[T,N] = X W^T: X [T,K] bf16; q [N,K/2], s and zeros [N,K/group].  For few rows (decoding)."""
    name = "dp_gemm_fwd_int4"
    index = X.get_device()
    if index < 0 or q.get_device() != index or s.get_device() != index or (zeros is not None and zeros.get_device() != index):
        tensors = (("X", X), ("codes", q), ("scales", s), ("zeros", zeros))
        c.refuse_devices(name, {what: t for what, t in tensors if t is not None})
    (N,), K, group, f32 = _weights(q, s, zeros, (2,), name)
    T, ldx = _rows(X, K, name)
    if not _fn:
        c.load()

    def work(st):
        y, code, ldy = c.output_rows(out, (T, N), out_dtype, index, X.device, name)
        code = _fn[name](X.data_ptr(), ldx, q.data_ptr(), s.data_ptr(), f32, None if zeros is None else zeros.data_ptr(), group,
                         y.data_ptr(), ldy, T, N, K, code, st)
        if code:
            c.check(code, name)
        return y

    return c.on_stream(index, stream, (X, q, s, zeros, out), work)


def dp_gemm_fwd_int4_grouped(X, q, s, offsets, zeros=None, out=None, out_dtype=c.BF16, stream=None):
    """Y[t] = X[t] W_e^T for the rows t of expert e: X [T,K] bf16; q [E,N,K/2], s and zeros [E,N,K/group];
    offsets [E + 1] as in dp_gemm_fwd_grouped (rows outside all groups give zero rows)."""
    name = "dp_gemm_fwd_int4_grouped"
    index = X.get_device()
    if (index < 0 or q.get_device() != index or s.get_device() != index or offsets.get_device() != index or
            (zeros is not None and zeros.get_device() != index)):
        tensors = (("X", X), ("codes", q), ("scales", s), ("zeros", zeros), ("offsets", offsets))
        c.refuse_devices(name, {what: t for what, t in tensors if t is not None})
    (E, N), K, group, f32 = _weights(q, s, zeros, (3,), name)
    T, ldx = _rows(X, K, name)
    bits = _BITS.get(offsets.dtype)
    if bits is None:
        raise TypeError(f"{name}: offsets must be int32 or int64")
    if offsets.dim() != 1 or not offsets.is_contiguous() or offsets.numel() != E + 1:
        raise ValueError(f"{name}: offsets must be a contiguous vector of E + 1 values")
    if not _fn:
        c.load()

    def work(st):
        y, code, ldy = c.output_rows(out, (T, N), out_dtype, index, X.device, name)
        code = _fn[name](X.data_ptr(), ldx, q.data_ptr(), s.data_ptr(), f32, None if zeros is None else zeros.data_ptr(), group,
                         offsets.data_ptr(), bits, y.data_ptr(), ldy, E, T, N, K, code, st)
        if code:
            c.check(code, name)
        return y

    return c.on_stream(index, stream, (X, q, s, zeros, offsets, out), work)
