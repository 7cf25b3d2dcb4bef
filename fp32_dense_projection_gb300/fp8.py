"""8-bit floating point with one FP32 scale per 128 values: quantisation and products.

  fp8_quantize(x, scaling)               "row": (q, s[T, ceil(C/128)])    blocks of 128 in a row
                                         "col": (q, s[ceil(T/128), C])    blocks of 128 in a column
                                         "block": (q, s[ceil(T/128), ceil(C/128)])
                                         "both": the row pair and the column pair, one read of x
  dp_gemm_fwd_fp8(Xq, Xs, Wq, Ws)        Y  = X W^T   X "row", W "block"
  dp_gemm_dgrad_fp8(dYq, dYs, Wq, Ws)    dX = dY W    dY "row", W "block" (the forward pass's)
  dp_gemm_wgrad_fp8(dYq, dYs, Xq, Xs)    dW = dY^T X  dY and X "col"

q is torch.float8_e4m3fn or float8_e5m2 and x is about q * s.  Scales may have any strides;
fp8_quantize lays row scales out with a column in one piece, as the products read them.
"""
from __future__ import annotations

import torch

from . import _call as c

_BF16, _F32 = torch.bfloat16, torch.float32
_FORMATS = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}
_SCALINGS = {"row": 0, "col": 1, "block": 2, "both": 3}


def _bind(L):
    P, I, S = c.P, c.I, c.S
    L.dp_fp8_quantize.argtypes = [P, I, S, I, I, S, S, P, I, P, I, I, P, I, P, I, P]
    for name in ("dp_gemm_fwd_fp8", "dp_gemm_dgrad_fp8", "dp_gemm_wgrad_fp8"):
        getattr(L, name).argtypes = [P, I, S, P, I, I, P, I, S, P, I, I, P, I, I, I, I, S, P]


def fp8_quantize(x, scaling="row", dtype=torch.float8_e4m3fn, stream=None):
    """Quantise x [T, C] (bf16 or fp32; C a multiple of 16) with a scale per 128 values:
    (q, scales), or (q_row, scales_row, q_col, scales_col) with scaling="both"."""
    from . import _check as status, _ptr, lib
    name = "fp8_quantize"
    c.need(scaling in _SCALINGS, f"{name}: scaling must be one of {tuple(_SCALINGS)}")
    c.need(dtype in _FORMATS, f"{name}: dtype must be one of {tuple(_FORMATS)}", TypeError)
    device = c.one_device(name, {"x": x})
    c.need(x.dtype in (_BF16, _F32), f"{name}: x must be bfloat16 or float32", TypeError)
    ldx = c.matrix(x, name, "x")
    T, C = x.shape
    tb, cb = -(-T // 128), -(-C // 128)
    q = s = qc = sc = None
    s_row = s_col = 0
    with c.on_stream(device, stream, (x,)) as st:
        if scaling in ("row", "both"):
            q = torch.empty((T, C), dtype=dtype, device=device)
            s = torch.empty((cb, T), dtype=_F32, device=device).t()
            s_row, s_col = 1, T
        elif scaling == "block":
            q = torch.empty((T, C), dtype=dtype, device=device)
            s = torch.empty((tb, cb), dtype=_F32, device=device)
            s_row, s_col = cb, 1
        if scaling in ("col", "both"):
            qc = torch.empty((T, C), dtype=dtype, device=device)
            sc = torch.empty((tb, C), dtype=_F32, device=device)
        status(lib().dp_fp8_quantize(_ptr(x), ldx, int(x.dtype == _F32), T, C, _SCALINGS[scaling], _FORMATS[dtype],
                                     _ptr(q), C, _ptr(s), s_row, s_col, _ptr(qc), C, _ptr(sc), C, st), name)
    if scaling == "both":
        return q, s, qc, sc
    return (qc, sc) if scaling == "col" else (q, s)


def _scales(s, shape, name, what):
    c.need(s.dtype == _F32, f"{name}: {what} must be float32", TypeError)
    c.need(tuple(s.shape) == shape, f"{name}: {what} must have shape {shape}")
    return s.stride(0), s.stride(1)


def _product(name, a, sa, a_shape, b, sb, b_shape, out, out_shape, out_dtype, sizes, stream):
    from . import DP_OUT_BF16, DP_OUT_F32, _check as status, _ptr, lib
    device = c.one_device(name, {"first operand": a, "its scales": sa, "second operand": b, "its scales": sb})
    for what, t in (("first operand", a), ("second operand", b)):
        c.need(t.dtype in _FORMATS, f"{name}: the {what} must be float8_e4m3fn or float8_e5m2", TypeError)
    ra, ca = _scales(sa, a_shape, name, "the first operand's scales")
    rb, cb = _scales(sb, b_shape, name, "the second operand's scales")
    lda, ldb = c.matrix(a, name, "the first operand"), c.matrix(b, name, "the second operand")
    with c.on_stream(device, stream, (a, sa, b, sb, out)) as st:
        out = c.output(out, out_shape, out_dtype, device, name, (_BF16, _F32))
        status(getattr(lib(), name)(_ptr(a), lda, _FORMATS[a.dtype], _ptr(sa), ra, ca, _ptr(b), ldb, _FORMATS[b.dtype],
                                    _ptr(sb), rb, cb, _ptr(out), c.matrix(out, name, "out"), *sizes,
                                    DP_OUT_F32 if out.dtype == _F32 else DP_OUT_BF16, st), name)
    return out


def _blocks(n: int) -> int:
    return -(-n // 128)


def dp_gemm_fwd_fp8(Xq, Xs, Wq, Ws, out=None, out_dtype=_BF16, stream=None):
    """Y[T,N] = X W^T: Xq [T,K] with row scales Xs [T, ceil(K/128)], Wq [N,K] with Ws [ceil(N/128), ceil(K/128)]."""
    name = "dp_gemm_fwd_fp8"
    c.need(Xq.dim() == 2 and Wq.dim() == 2 and Xq.shape[1] == Wq.shape[1], f"{name}: X[T,K] and W[N,K] must share K")
    (T, K), N = Xq.shape, Wq.shape[0]
    return _product(name, Xq, Xs, (T, _blocks(K)), Wq, Ws, (_blocks(N), _blocks(K)), out, (T, N), out_dtype, (T, N, K), stream)


def dp_gemm_dgrad_fp8(dYq, dYs, Wq, Ws, out=None, out_dtype=_BF16, stream=None):
    """dX[T,K] = dY W: dYq [T,N] with row scales dYs [T, ceil(N/128)], Wq and Ws as in the forward pass."""
    name = "dp_gemm_dgrad_fp8"
    c.need(dYq.dim() == 2 and Wq.dim() == 2 and dYq.shape[1] == Wq.shape[0], f"{name}: dY[T,N] and W[N,K] must share N")
    (T, N), K = dYq.shape, Wq.shape[1]
    return _product(name, dYq, dYs, (T, _blocks(N)), Wq, Ws, (_blocks(N), _blocks(K)), out, (T, K), out_dtype, (T, N, K), stream)


def dp_gemm_wgrad_fp8(dYq, dYs, Xq, Xs, out=None, out_dtype=_BF16, stream=None):
    """dW[N,K] = dY^T X: dYq [T,N] and Xq [T,K] with column scales dYs [ceil(T/128), N], Xs [ceil(T/128), K]."""
    name = "dp_gemm_wgrad_fp8"
    c.need(dYq.dim() == 2 and Xq.dim() == 2 and dYq.shape[0] == Xq.shape[0], f"{name}: dY[T,N] and X[T,K] must share T")
    (T, N), K = dYq.shape, Xq.shape[1]
    return _product(name, dYq, dYs, (_blocks(T), N), Xq, Xs, (_blocks(T), K), out, (N, K), out_dtype, (T, N, K), stream)
