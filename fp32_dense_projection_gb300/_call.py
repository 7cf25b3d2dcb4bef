"""Marshalling shared by the bindings of the grouped, 8-bit and 4-bit products, AdamW, layer norm and the experts' operators.

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
_deterministic = torch.are_deterministic_algorithms_enabled


def _public(shape, strides, dtype):
    return torch.empty_strided(shape, strides, dtype=dtype, device="cuda")


def _choose(found):
    """The function found if it makes what the public one makes (without dispatch: 0.9 for 1.5 us by itself, a call of layer norm
    13.8 for 17.6, of the choice 8.8 for 12.6)."""
    try:
        t = found((2, 3), (3, 1), BF16)
        ok = t.shape == (2, 3) and t.stride() == (3, 1) and t.dtype is BF16 and t.get_device() == _current_device()
    except Exception:  # something else has its name
        ok = False
    return found if ok else _public


def _direct(shape, strides, dtype):
    """An uninitialised tensor on the current device.  (The first one; from then on, what _choose gives.)"""
    global _direct
    _direct = _choose(_found)
    return _direct(shape, strides, dtype)


try:
    from torch._C import _len_torch_dispatch_stack as _modes
    from torch._C._dynamo.guards import _empty_strided_cuda as _found
    _modes()
except Exception:  # not in this torch: the public function alone
    _modes, _direct = int, _public


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


def new(shape, dtype):
    """A new contiguous tensor on the current device.  What watches torch's allocations (dispatch modes, the filling of new
    memory that goes with deterministic algorithms) gets the public function's."""
    empty = _public if _deterministic() or _modes() else _direct
    if len(shape) == 2:
        rows, cols = shape
        return empty((rows, cols), (cols, 1), dtype)
    strides, step = [], 1
    for n in reversed(shape):
        strides.append(step)
        step *= max(n, 1)
    return empty(tuple(shape), tuple(reversed(strides)), dtype)


def new_vector(n, dtype):
    return (_public if _deterministic() or _modes() else _direct)((n,), (1,), dtype)


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


def output_rows(out, shape, dtype, index: int, device, name: str, what: str = "out"):
    """The given 2-D output, checked, or a new one; its type's code; its leading dimension."""
    if out is None:
        code = OUT_CODES.get(dtype)
        if code is not None:
            return new(shape, dtype), code, shape[1]
    y, code = output(out, shape, dtype, index, device, name)
    return y, code, ld(y, name, what, shape)


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
