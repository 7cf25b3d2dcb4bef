"""Products of rows sorted by expert with their expert's weights (BF16).

  dp_gemm_fwd_grouped(X, W, offsets)      Y[t]  = X[t] W_e^T
  dp_gemm_dgrad_grouped(dY, W, offsets)   dX[t] = dY[t] W_e
  dp_gemm_wgrad_grouped(dY, X, offsets)   dW_e  = sum over the expert's rows of dY[t]^T X[t]

Expert e owns the rows offsets[e] .. offsets[e + 1] (E + 1 values, int32 or int64, on the
device).  The host never reads them, so a call neither waits for the router nor changes
with its choice.  Rows outside all groups give zero rows; experts without rows give zero
weight gradients.  W and dW are [E, N, K] ("nk") or [E, K, N] ("kn").
"""
from __future__ import annotations

import torch

from . import _call as c

_BITS = {torch.int32: 32, torch.int64: 64}
_LAYOUTS = {"nk": 0, "kn": 1}
_fn = {}


def _bind(L):
    P, I, S = c.P, c.I, c.S
    for name in ("dp_gemm_fwd_grouped", "dp_gemm_dgrad_grouped"):
        getattr(L, name).argtypes = [P, I, P, I, I, S, P, S, P, I, I, I, I, I, S, P]
    L.dp_gemm_wgrad_grouped.argtypes = [P, I, P, I, P, S, P, I, I, S, I, I, I, I, S, P]
    _fn.update({name: getattr(L, name) for name in ("dp_gemm_fwd_grouped", "dp_gemm_dgrad_grouped", "dp_gemm_wgrad_grouped")})


def _experts(w: torch.Tensor, name: str, what: str, shape):
    """(leading dimension, expert stride) of an [E, rows, columns] view of that shape."""
    strides = w.stride()
    if len(shape) != 3 or (strides[2] != 1 and shape[2] > 1):
        raise ValueError(f"{name}: {what} must be [E, rows, columns] with unit column stride")
    if (strides[1] == 0 and shape[1] > 1) or (strides[0] == 0 and shape[0] > 1):  # (0 means packed to the library)
        raise ValueError(f"{name}: {what} must not be expanded over experts or rows (stride 0)")
    ld = strides[1] if shape[1] > 1 else max(shape[2], 1)
    return ld, strides[0] if shape[0] > 1 else shape[1] * ld


def _layout(weight_layout):
    kn = _LAYOUTS.get(weight_layout)
    if kn is None:
        raise ValueError('weight_layout must be "nk" ([N, K] weights) or "kn" ([K, N])')
    return kn


def _check(name, a, b, b_name, offsets, E):
    """Devices, types and the offsets' form; the offsets' width and the device's index."""
    index = a.get_device()
    if index < 0 or b.get_device() != index or offsets.get_device() != index:
        c.refuse_devices(name, {"rows": a, b_name: b, "offsets": offsets})
    if a.dtype is not c.BF16 or b.dtype is not c.BF16:
        raise TypeError(f"{name}: rows and {b_name} must be bfloat16")
    bits = _BITS.get(offsets.dtype)
    if bits is None:
        raise TypeError(f"{name}: offsets must be int32 or int64")
    if offsets.dim() != 1 or not offsets.is_contiguous() or offsets.numel() != E + 1:
        raise ValueError(f"{name}: offsets must be a contiguous vector of E + 1 values")
    return index, bits


def _rows_by_experts(name, forward, a, W, offsets, out, out_dtype, weight_layout, stream):
    kn = _layout(weight_layout)
    rows, weights = a.shape, W.shape
    if len(rows) != 2 or len(weights) != 3:
        raise ValueError(f"{name}: rows must be 2-D and weights 3-D")
    T, width = rows
    E, N, K = weights
    if kn:
        N, K = K, N
    if width != (K if forward else N):
        raise ValueError(f"{name}: the rows' length does not match the weights")
    index, bits = _check(name, a, W, "weights", offsets, E)
    ldw, bsw = _experts(W, name, "weights", weights)
    lda = c.ld(a, name, "rows", rows)
    if not _fn:
        c.load()

    def work(st):
        shape = (T, N if forward else K)
        y, code = c.output(out, shape, out_dtype, index, a.device, name)
        code = _fn[name](a.data_ptr(), lda, W.data_ptr(), ldw, bsw, kn, offsets.data_ptr(), bits, y.data_ptr(),
                         c.ld(y, name, "out", shape), E, T, N, K, code, st)
        if code:
            c.check(code, name)
        return y

    return c.on_stream(index, stream, (a, W, offsets, out), work)


def dp_gemm_fwd_grouped(X, W, offsets, out=None, out_dtype=c.BF16, weight_layout="nk", stream=None):
    """Y[t] = X[t] W_e^T for the rows t of expert e: X [T,K]; W [E,N,K] ("nk") or [E,K,N] ("kn"); Y [T,N]."""
    return _rows_by_experts("dp_gemm_fwd_grouped", True, X, W, offsets, out, out_dtype, weight_layout, stream)


def dp_gemm_dgrad_grouped(dY, W, offsets, out=None, out_dtype=c.BF16, weight_layout="nk", stream=None):
    """dX[t] = dY[t] W_e for the rows t of expert e: dY [T,N]; W as in the forward pass; dX [T,K]."""
    return _rows_by_experts("dp_gemm_dgrad_grouped", False, dY, W, offsets, out, out_dtype, weight_layout, stream)


def dp_gemm_wgrad_grouped(dY, X, offsets, out=None, out_dtype=c.BF16, weight_layout="nk", stream=None):
    """dW_e = sum over expert e's rows of dY[t]^T X[t]: dY [T,N]; X [T,K]; dW [E,N,K] ("nk") or [E,K,N] ("kn")."""
    name = "dp_gemm_wgrad_grouped"
    kn = _layout(weight_layout)
    if dY.dim() != 2 or X.dim() != 2 or dY.shape[0] != X.shape[0]:
        raise ValueError(f"{name}: dY[T,N] and X[T,K] must have the same rows")
    (T, N), K = dY.shape, X.shape[1]
    E = offsets.numel() - 1
    index, bits = _check(name, dY, X, "X", offsets, max(E, 0))
    ldg, ldx = c.ld(dY, name, "dY"), c.ld(X, name, "X")
    if not _fn:
        c.load()

    def work(st):
        shape = (E, K, N) if kn else (E, N, K)
        dW, code = c.output(out, shape, out_dtype, index, dY.device, name)
        ldw, bsw = _experts(dW, name, "out", shape)
        code = _fn[name](dY.data_ptr(), ldg, X.data_ptr(), ldx, offsets.data_ptr(), bits, dW.data_ptr(), ldw, bsw, kn, E, T,
                         N, K, code, st)
        if code:
            c.check(code, name)
        return dW

    return c.on_stream(index, stream, (dY, X, offsets, out), work)
