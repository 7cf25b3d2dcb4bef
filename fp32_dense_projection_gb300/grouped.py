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

_BF16, _F32 = torch.bfloat16, torch.float32


def _bind(L):
    P, I, S = c.P, c.I, c.S
    for name in ("dp_gemm_fwd_grouped", "dp_gemm_dgrad_grouped"):
        getattr(L, name).argtypes = [P, I, P, I, I, S, P, S, P, I, I, I, I, I, S, P]
    L.dp_gemm_wgrad_grouped.argtypes = [P, I, P, I, P, S, P, I, I, S, I, I, I, I, S, P]


def _experts(w: torch.Tensor, name: str, what: str):
    """(leading dimension, expert stride) of an [E, rows, columns] view."""
    c.need(w.dim() == 3 and (w.size(2) <= 1 or w.stride(2) == 1), f"{name}: {what} must be [E, rows, columns] with unit column stride")
    ld = w.stride(1) if w.size(1) > 1 else max(w.size(2), 1)
    bs = w.stride(0) if w.size(0) > 1 else w.size(1) * ld
    return ld, bs


def _check(name, rows: dict, weights, offsets, E):
    device = c.one_device(name, {**rows, "weights": weights, "offsets": offsets} if weights is not None else {**rows, "offsets": offsets})
    for what, t in rows.items():
        c.need(t.dtype == _BF16, f"{name}: {what} must be bfloat16", TypeError)
    if weights is not None:
        c.need(weights.dtype == _BF16, f"{name}: weights must be bfloat16", TypeError)
    c.need(offsets.dtype in (torch.int32, torch.int64), f"{name}: offsets must be int32 or int64", TypeError)
    c.need(offsets.dim() == 1 and offsets.is_contiguous() and offsets.numel() >= 1 and (E is None or offsets.numel() == E + 1),
           f"{name}: offsets must be a contiguous vector of E + 1 values")
    return device


def _rows_by_experts(name, op, a, W, offsets, out, out_dtype, weight_layout, stream):
    from . import DP_OUT_BF16, DP_OUT_F32, _check as status, _layout, _ptr, lib
    kn = _layout(weight_layout)
    c.need(a.dim() == 2 and W.dim() == 3, f"{name}: rows must be 2-D and weights 3-D")
    T, width = a.shape
    E = W.shape[0]
    N, K = (W.shape[2], W.shape[1]) if kn else (W.shape[1], W.shape[2])
    c.need(width == (K if op == "fwd" else N), f"{name}: the rows' length does not match the weights")
    device = _check(name, {"rows": a}, W, offsets, E)
    ldw, bsw = _experts(W, name, "weights")
    with c.on_stream(device, stream, (a, W, offsets, out)) as st:
        out = c.output(out, (T, N if op == "fwd" else K), out_dtype, device, name, (_BF16, _F32))
        code = DP_OUT_F32 if out.dtype == _F32 else DP_OUT_BF16
        status(getattr(lib(), name)(_ptr(a), c.matrix(a, name, "rows"), _ptr(W), ldw, bsw, int(kn), _ptr(offsets),
                                    offsets.element_size() * 8, _ptr(out), c.matrix(out, name, "out"), E, T, N, K, code, st), name)
    return out


def dp_gemm_fwd_grouped(X, W, offsets, out=None, out_dtype=_BF16, weight_layout="nk", stream=None):
    """Y[t] = X[t] W_e^T for the rows t of expert e: X [T,K]; W [E,N,K] ("nk") or [E,K,N] ("kn"); Y [T,N]."""
    return _rows_by_experts("dp_gemm_fwd_grouped", "fwd", X, W, offsets, out, out_dtype, weight_layout, stream)


def dp_gemm_dgrad_grouped(dY, W, offsets, out=None, out_dtype=_BF16, weight_layout="nk", stream=None):
    """dX[t] = dY[t] W_e for the rows t of expert e: dY [T,N]; W as in the forward pass; dX [T,K]."""
    return _rows_by_experts("dp_gemm_dgrad_grouped", "dgrad", dY, W, offsets, out, out_dtype, weight_layout, stream)


def dp_gemm_wgrad_grouped(dY, X, offsets, out=None, out_dtype=_BF16, weight_layout="nk", stream=None):
    """dW_e = sum over expert e's rows of dY[t]^T X[t]: dY [T,N]; X [T,K]; dW [E,N,K] ("nk") or [E,K,N] ("kn")."""
    from . import DP_OUT_BF16, DP_OUT_F32, _check as status, _layout, _ptr, lib
    name = "dp_gemm_wgrad_grouped"
    kn = _layout(weight_layout)
    c.need(dY.dim() == 2 and X.dim() == 2 and dY.shape[0] == X.shape[0], f"{name}: dY[T,N] and X[T,K] must have the same rows")
    (T, N), K = dY.shape, X.shape[1]
    device = _check(name, {"dY": dY, "X": X}, None, offsets, None)
    E = offsets.numel() - 1
    with c.on_stream(device, stream, (dY, X, offsets, out)) as st:
        out = c.output(out, (E, K, N) if kn else (E, N, K), out_dtype, device, name, (_BF16, _F32))
        ldo, bso = _experts(out, name, "out")
        code = DP_OUT_F32 if out.dtype == _F32 else DP_OUT_BF16
        status(lib().dp_gemm_wgrad_grouped(_ptr(dY), c.matrix(dY, name, "dY"), _ptr(X), c.matrix(X, name, "X"), _ptr(offsets),
                                           offsets.element_size() * 8, _ptr(out), ldo, bso, int(kn), E, T, N, K, code, st), name)
    return out
