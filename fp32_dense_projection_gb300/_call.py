"""Marshalling shared by the grouped, 8-bit and AdamW bindings.

A call of a few microseconds on the GPU is bound by what the host does before it, so checks
are plain comparisons, and their messages are put together only when one of them fails.
"""
from __future__ import annotations

import ctypes

import torch

P, I, S = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
BF16, F32 = torch.bfloat16, torch.float32
OUT_CODES = {BF16: 0, F32: 1}  # dp_out_dtype

_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def load():
    """Load the library: a module's first call (it fills the module's table of functions, at once)."""
    from . import lib
    lib()


def check(code: int, what: str):
    """Raise the status of a call that did not succeed."""
    from . import _check
    _check(code, what)


def refuse_devices(name: str, tensors: dict):
    """Say which of the tensors is not on the first one's CUDA device (one of them is not)."""
    first = None
    for what, t in tensors.items():
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name}: {what} must be a CUDA tensor")
        first = t.device if first is None else first
        if t.device != first:
            raise ValueError(f"{name}: {what} is on {t.device}, the first operand on {first}")


def ld(t: torch.Tensor, name: str, what: str, shape=None) -> int:
    """Leading dimension of a 2-D view (of that shape) with unit column stride.  Rows that share
    their memory (an expanded row) are refused: to the library a stride of 0 means packed rows."""
    strides, shape = t.stride(), t.shape if shape is None else shape
    if len(shape) != 2 or (strides[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name}: {what} must be 2-D with unit column stride")
    if shape[0] <= 1:
        return max(strides[0], shape[1])
    if strides[0] == 0:
        raise ValueError(f"{name}: {what} must not be expanded over its rows (stride 0)")
    return strides[0]


def output(out, shape, dtype, index: int, device, name: str):
    """The given output, checked, or a new one; and its type's code."""
    if out is None:
        code = OUT_CODES.get(dtype)
        if code is None:
            raise TypeError(f"{name}: out_dtype must be bfloat16 or float32")
        return torch.empty(shape, dtype=dtype, device=device), code
    code = OUT_CODES.get(out.dtype)
    if code is None:
        raise TypeError(f"{name}: out must be bfloat16 or float32")
    if out.shape != shape:
        raise ValueError(f"{name}: out must have shape {tuple(shape)}")
    if out.get_device() != index:
        raise ValueError(f"{name}: out must be on {device}")
    return out, code


def on_stream(index: int, stream, tensors, work):
    """work(raw stream) with the device current and, if one is given, on that stream: memory
    that the call allocates belongs to it, and its operands' memory is not handed out again
    before the stream's work on them is done."""
    if stream is None:
        if _current_device() == index:
            return work(_raw_stream(index))
        with torch.cuda.device(index):
            return work(_raw_stream(index))
    with torch.cuda.device(index), torch.cuda.stream(stream):
        result = work(stream.cuda_stream)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return result
