"""Layer norm in front of the projections, and its gradients.

  layer_norm_fwd(x, weight, bias)                   (y, mean, rstd): y = (x - mean) rstd weight + bias over each row
  layer_norm_bwd(dY, x, mean, rstd, weight)         (dX, dW, dB): the gradients of rows, weight and bias

Rows and their gradients are bf16 or fp32, weight and bias fp32 or bf16 (both alike); mean, rstd and
the gradients of weight and bias are fp32.  Sums over tokens are deterministic.
"""
from __future__ import annotations

import ctypes

import torch

from . import _call as c

_fn = {}


def _bind(L):
    P, I, S = c.P, c.I, c.S
    L.dp_layer_norm_fwd.argtypes = [P, I, S, P, P, S, ctypes.c_double, P, I, S, P, P, I, I, P]
    L.dp_layer_norm_bwd.argtypes = [P, I, S, P, I, S, P, P, P, S, P, I, S, P, P, I, I, P, ctypes.c_size_t, P]
    L.dp_layer_norm_workspace_size.argtypes = [I, I, S, ctypes.POINTER(ctypes.c_size_t)]
    _fn.update({name: getattr(L, name) for name in ("dp_layer_norm_fwd", "dp_layer_norm_bwd", "dp_layer_norm_workspace_size")})


def _rows(t, name, what):
    """Whether the rows are fp32 (else bf16)."""
    if t.dtype is c.F32:
        return 1
    if t.dtype is c.BF16:
        return 0
    raise TypeError(f"{name}: {what} must be bfloat16 or float32")


def _vector(t, n, dtypes, name, what):
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: {what} must be {' or '.join(str(d).removeprefix('torch.') for d in dtypes)}")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name}: {what} must be a contiguous vector of {n} values")


_PARAMS, _STATS = (c.F32, c.BF16), (c.F32,)


def layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, out=None, out_dtype=c.BF16, stream=None):
    """(y [T,C], mean [T], rstd [T]) of x [T,C] (C a multiple of 8, at most 16384)."""
    name = "layer_norm_fwd"
    index = x.get_device()
    if index < 0 or (weight is not None and weight.get_device() != index) or (bias is not None and bias.get_device() != index):
        c.refuse_devices(name, {k: t for k, t in (("x", x), ("weight", weight), ("bias", bias)) if t is not None})
    f32, ldx = _rows(x, name, "x"), c.ld(x, name, "x")
    T, C = shape = x.shape
    w32 = 0
    for what, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _vector(t, C, _PARAMS, name, what)
            w32 = t.dtype is c.F32
    if weight is not None and bias is not None and weight.dtype is not bias.dtype:
        raise TypeError(f"{name}: weight and bias must have the same type")
    if not _fn:
        c.load()

    def work(st):
        y, code, ldy = c.output_rows(out, shape, out_dtype, index, x.device, name)
        mean = c.new_vector(T, c.F32)
        rstd = c.new_vector(T, c.F32)
        code = _fn["dp_layer_norm_fwd"](x.data_ptr(), ldx, f32, None if weight is None else weight.data_ptr(),
                                        None if bias is None else bias.data_ptr(), w32, eps, y.data_ptr(), ldy,
                                        code, mean.data_ptr(), rstd.data_ptr(), T, C, st)
        if code:
            c.check(code, name)
        return y, mean, rstd

    return c.on_stream(index, stream, (x, weight, bias, out), work)


_last_size = (None, 0)  # the last call's sizes and what they need


def _workspace_size(index, T, C):
    """Of the current device (asked again only where the sizes change)."""
    global _last_size
    key, size = _last_size
    if key != (index, T, C):
        n = ctypes.c_size_t(0)
        status = _fn["dp_layer_norm_workspace_size"](T, C, 0, ctypes.byref(n))
        if status:
            c.check(status, "layer_norm_bwd")
        size = n.value
        _last_size = (index, T, C), size
    return size


def layer_norm_bwd(dY, x, mean, rstd, weight=None, dX=None, dx_dtype=c.BF16, workspace=None, stream=None, param_grads=None):
    """(dX [T,C], dW [C], dB [C]) from dY [T,C] and what the forward pass read and returned.
    dW and dB are made where there is a weight, or as ``param_grads`` says (True: also without one, for a
    bias alone, dW as of a weight of ones; False: None)."""
    name = "layer_norm_bwd"
    index = dY.get_device()
    if (index < 0 or x.get_device() != index or mean.get_device() != index or rstd.get_device() != index or
            (weight is not None and weight.get_device() != index) or (workspace is not None and workspace.get_device() != index)):
        tensors = {"dY": dY, "x": x, "mean": mean, "rstd": rstd, "weight": weight, "workspace": workspace}
        c.refuse_devices(name, {k: t for k, t in tensors.items() if t is not None})
    g32, ldg, x32, ldx = _rows(dY, name, "dY"), c.ld(dY, name, "dY"), _rows(x, name, "x"), c.ld(x, name, "x")
    T, C = shape = dY.shape
    if x.shape != shape:
        raise ValueError(f"{name}: dY and x must have the same shape")
    _vector(mean, T, _STATS, name, "mean")
    _vector(rstd, T, _STATS, name, "rstd")
    if weight is not None:
        _vector(weight, C, _PARAMS, name, "weight")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError(f"{name}: workspace must be contiguous")
    if param_grads is None:
        param_grads = weight is not None
    if not _fn:
        c.load()

    def work(st):
        d, code, ld_dx = c.output_rows(dX, shape, dx_dtype, index, dY.device, name, "dX")
        dW = dB = buf = None
        size = 0
        if param_grads:
            dW = c.new_vector(C, c.F32)
            dB = c.new_vector(C, c.F32)
            if workspace is None:
                size = _workspace_size(index, T, C)
                buf = c.new_vector(size, torch.uint8)
            else:
                buf, size = workspace, workspace.nbytes
        status = _fn["dp_layer_norm_bwd"](dY.data_ptr(), ldg, g32, x.data_ptr(), ldx, x32, mean.data_ptr(), rstd.data_ptr(),
                                          None if weight is None else weight.data_ptr(), weight is not None and weight.dtype is c.F32,
                                          d.data_ptr(), ld_dx, code, None if dW is None else dW.data_ptr(),
                                          None if dB is None else dB.data_ptr(), T, C, None if buf is None else buf.data_ptr(), size, st)
        if status:
            c.check(status, name)
        return d, dW, dB

    return c.on_stream(index, stream, (dY, x, mean, rstd, weight, dX, workspace), work)
