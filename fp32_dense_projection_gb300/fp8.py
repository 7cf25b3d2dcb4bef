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

_FORMATS = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}
_SCALINGS = {"row": 0, "col": 1, "block": 2, "both": 3}
_fn = {}


def _bind(L):
    P, I, S = c.P, c.I, c.S
    products = ("dp_gemm_fwd_fp8", "dp_gemm_dgrad_fp8", "dp_gemm_wgrad_fp8")
    L.dp_fp8_quantize.argtypes = [P, I, S, I, I, S, S, P, I, P, I, I, P, I, P, I, P]
    for name in products:
        getattr(L, name).argtypes = [P, I, S, P, I, I, P, I, S, P, I, I, P, I, I, I, I, S, P]
    _fn.update({name: getattr(L, name) for name in ("dp_fp8_quantize", *products)})


def fp8_quantize(x, scaling="row", dtype=torch.float8_e4m3fn, stream=None):
    """Quantise x [T, C] (bf16 or fp32; C a multiple of 16) with a scale per 128 values:
    (q, scales), or (q_row, scales_row, q_col, scales_col) with scaling="both"."""
    name = "fp8_quantize"
    mode, fmt = _SCALINGS.get(scaling), _FORMATS.get(dtype)
    if mode is None:
        raise ValueError(f"{name}: scaling must be one of {tuple(_SCALINGS)}")
    if fmt is None:
        raise TypeError(f"{name}: dtype must be one of {tuple(_FORMATS)}")
    index = x.get_device()
    if index < 0:
        c.refuse_devices(name, {"x": x})
    f32 = x.dtype is c.F32
    if not f32 and x.dtype is not c.BF16:
        raise TypeError(f"{name}: x must be bfloat16 or float32")
    ldx = c.ld(x, name, "x")
    T, C = x.shape
    tb, cb, device = -(-T // 128), -(-C // 128), x.device
    if not _fn:
        c.load()

    def work(st):
        q = s = qc = sc = None
        s_row = s_col = 0
        if mode != 1:
            q = torch.empty((T, C), dtype=dtype, device=device)
            if mode == 2:
                s = torch.empty((tb, cb), dtype=c.F32, device=device)
                s_row, s_col = cb, 1
            else:
                s = torch.empty((cb, T), dtype=c.F32, device=device).t()
                s_row, s_col = 1, T
        if mode & 1:
            qc = torch.empty((T, C), dtype=dtype, device=device)
            sc = torch.empty((tb, C), dtype=c.F32, device=device)
        code = _fn["dp_fp8_quantize"](x.data_ptr(), ldx, f32, T, C, mode, fmt, None if q is None else q.data_ptr(), C,
                                      None if s is None else s.data_ptr(), s_row, s_col,
                                      None if qc is None else qc.data_ptr(), C, None if sc is None else sc.data_ptr(), C, st)
        if code:
            c.check(code, name)
        return (q, s, qc, sc) if mode == 3 else (qc, sc) if mode == 1 else (q, s)

    return c.on_stream(index, stream, (x,), work)


def _refuse(name, a, sa, a_shape, b, sb, b_shape):
    """Say what is wrong with the operands (something is)."""
    c.refuse_devices(name, {"the first operand": a, "its scales": sa, "the second operand": b, "its scales ": sb})
    for what, q, s, shape in (("first", a, sa, a_shape), ("second", b, sb, b_shape)):
        if q.dtype not in _FORMATS:
            raise TypeError(f"{name}: the {what} operand must be float8_e4m3fn or float8_e5m2")
        if s.dtype is not c.F32:
            raise TypeError(f"{name}: the {what} operand's scales must be float32")
        if s.shape != shape:
            raise ValueError(f"{name}: the {what} operand's scales must have shape {shape}")
    raise AssertionError(name)


def _product(name, a, a_shape, sa, sa_shape, b, b_shape, sb, sb_shape, out, out_shape, out_dtype, T, N, K, stream):
    index, fa, fb = a.get_device(), _FORMATS.get(a.dtype), _FORMATS.get(b.dtype)
    if (index < 0 or sa.get_device() != index or b.get_device() != index or sb.get_device() != index or fa is None or
            fb is None or sa.dtype is not c.F32 or sb.dtype is not c.F32 or sa.shape != sa_shape or sb.shape != sb_shape):
        _refuse(name, a, sa, sa_shape, b, sb, sb_shape)
    lda, ldb = c.ld(a, name, "the first operand", a_shape), c.ld(b, name, "the second operand", b_shape)
    (ra, ca), (rb, cb) = sa.stride(), sb.stride()
    if not _fn:
        c.load()

    def work(st):
        y, code = c.output(out, out_shape, out_dtype, index, a.device, name)
        code = _fn[name](a.data_ptr(), lda, fa, sa.data_ptr(), ra, ca, b.data_ptr(), ldb, fb, sb.data_ptr(), rb, cb,
                         y.data_ptr(), c.ld(y, name, "out", out_shape), T, N, K, code, st)
        if code:
            c.check(code, name)
        return y

    return c.on_stream(index, stream, (a, sa, b, sb, out), work)


def _shapes(name, a, b, dim_a, dim_b, what):
    sa, sb = a.shape, b.shape
    if len(sa) != 2 or len(sb) != 2 or sa[dim_a] != sb[dim_b]:
        raise ValueError(f"{name}: {what}")
    return sa, sb


def dp_gemm_fwd_fp8(Xq, Xs, Wq, Ws, out=None, out_dtype=c.BF16, stream=None):
    """Y[T,N] = X W^T: Xq [T,K] with row scales Xs [T, ceil(K/128)], Wq [N,K] with Ws [ceil(N/128), ceil(K/128)]."""
    name = "dp_gemm_fwd_fp8"
    x, w = _shapes(name, Xq, Wq, 1, 1, "X[T,K] and W[N,K] must share K")
    (T, K), N = x, w[0]
    kb = -(-K // 128)
    return _product(name, Xq, x, Xs, (T, kb), Wq, w, Ws, (-(-N // 128), kb), out, (T, N), out_dtype, T, N, K, stream)


def dp_gemm_dgrad_fp8(dYq, dYs, Wq, Ws, out=None, out_dtype=c.BF16, stream=None):
    """dX[T,K] = dY W: dYq [T,N] with row scales dYs [T, ceil(N/128)], Wq and Ws as in the forward pass."""
    name = "dp_gemm_dgrad_fp8"
    g, w = _shapes(name, dYq, Wq, 1, 0, "dY[T,N] and W[N,K] must share N")
    (T, N), K = g, w[1]
    nb = -(-N // 128)
    return _product(name, dYq, g, dYs, (T, nb), Wq, w, Ws, (nb, -(-K // 128)), out, (T, K), out_dtype, T, N, K, stream)


def dp_gemm_wgrad_fp8(dYq, dYs, Xq, Xs, out=None, out_dtype=c.BF16, stream=None):
    """dW[N,K] = dY^T X: dYq [T,N] and Xq [T,K] with column scales dYs [ceil(T/128), N], Xs [ceil(T/128), K]."""
    name = "dp_gemm_wgrad_fp8"
    g, x = _shapes(name, dYq, Xq, 0, 0, "dY[T,N] and X[T,K] must share T")
    (T, N), K = g, x[1]
    tb = -(-T // 128)
    return _product(name, dYq, g, dYs, (tb, N), Xq, x, Xs, (tb, K), out, (N, K), out_dtype, T, N, K, stream)
