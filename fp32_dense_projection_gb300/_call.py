"""Marshalling shared by the grouped, 8-bit and AdamW bindings."""
from __future__ import annotations

import contextlib
import ctypes

import torch

P, I, S = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int


def need(ok: bool, what: str, kind=ValueError):
    if not ok:
        raise kind(what)


def one_device(name: str, tensors: dict) -> torch.device:
    """The CUDA device that every given tensor is on."""
    device = None
    for what, t in tensors.items():
        need(isinstance(t, torch.Tensor) and t.is_cuda, f"{name}: {what} must be a CUDA tensor")
        if device is None:
            device = t.device
        need(t.device == device, f"{name}: {what} is on {t.device}, the first operand on {device}")
    return device


@contextlib.contextmanager
def on_stream(device: torch.device, stream, tensors=()):
    """The device and, if one is given, the stream of a call: memory that the call
    allocates belongs to that stream, and its operands' memory is not handed out again
    before the stream's work on them is done."""
    if stream is None and device.index == torch.cuda.current_device():
        yield ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)
        return
    with torch.cuda.device(device):
        if stream is None:
            yield ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)
            return
        with torch.cuda.stream(stream):
            yield ctypes.c_void_p(stream.cuda_stream)
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def matrix(t: torch.Tensor, name: str, what: str):
    """Leading dimension of a 2-D view with unit column stride."""
    need(t.dim() == 2 and (t.size(1) <= 1 or t.stride(1) == 1), f"{name}: {what} must be 2-D with unit column stride")
    return t.stride(0) if t.size(0) > 1 else max(t.stride(0), t.size(1))


def output(out, shape, dtype, device, name: str, allowed):
    if out is None:
        need(dtype in allowed, f"{name}: out_dtype must be one of {allowed}", TypeError)
        return torch.empty(shape, dtype=dtype, device=device)
    need(tuple(out.shape) == tuple(shape), f"{name}: out must have shape {tuple(shape)}")
    need(out.dtype in allowed, f"{name}: out must be one of {allowed}", TypeError)
    need(out.is_cuda and out.device == device, f"{name}: out must be on {device}")
    return out
