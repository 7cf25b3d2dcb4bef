"""AdamW over many tensors in one launch, moments in 32 or 8 bits.

  opt = AdamW(params, lr=1e-3, state_bits=8, copies=bf16_weights)
  opt.step(grads, grad_scale=clip)

params are dense fp32 or bf16 CUDA tensors, updated in place; grads fp32 or bf16, one per
parameter (None: that parameter is left as it is).  copies are optional bf16 tensors that
receive the updated parameter: the working weights of the GEMMs beside fp32 master weights.
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import _call as c

_BLOCK = 128
_ENTRY = np.dtype([("param", "u8"), ("grad", "u8"), ("exp_avg", "u8"), ("exp_avg_sq", "u8"), ("exp_avg_scale", "u8"),
                   ("exp_avg_sq_scale", "u8"), ("copy", "u8"), ("numel", "i8"), ("param_bf16", "i4"), ("grad_bf16", "i4")])


class _Hyper(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay", "grad_scale")] + [
        ("grad_scale_ptr", ctypes.c_void_p), ("step", ctypes.c_int64)]


def _bind(L):
    L.dp_adamw_step.argtypes = [c.P, c.I, c.S, ctypes.POINTER(_Hyper), c.P]


class AdamW:
    """AdamW with decoupled weight decay over a list of tensors.

    state_bits=32 keeps both moments in fp32.  state_bits=8 keeps them as float8_e4m3fn
    codes with an fp32 scale per 128 consecutive elements: ``exp_avg`` holds m / scale,
    ``exp_avg_sq`` holds sqrt(v) / scale.  The moments are attributes (lists of tensors) and
    may be passed in, with ``step`` the updates already done, to resume a run.
    """

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2, state_bits=32, copies=None,
                 exp_avg=None, exp_avg_sq=None, exp_avg_scale=None, exp_avg_sq_scale=None, step=0):
        self.params = list(params)
        c.need(state_bits in (8, 32), "AdamW: state_bits must be 8 or 32")
        c.need(len(betas) == 2 and all(0.0 <= b < 1.0 for b in betas), "AdamW: betas must lie in [0, 1)")
        c.need(lr >= 0 and eps >= 0 and weight_decay >= 0, "AdamW: lr, eps and weight_decay must not be negative")
        c.need(step >= 0, "AdamW: step must not be negative")
        self.lr, self.betas, self.eps, self.weight_decay = lr, tuple(betas), eps, weight_decay
        self.state_bits, self.step_count = state_bits, int(step)
        self.device = c.one_device("AdamW", {f"params[{i}]": p for i, p in enumerate(self.params)})
        for i, p in enumerate(self.params):
            c.need(p.dtype in (torch.float32, torch.bfloat16), f"AdamW: params[{i}] must be float32 or bfloat16", TypeError)
            c.need(p.is_contiguous(), f"AdamW: params[{i}] must be contiguous")
        n = len(self.params)
        self._shapes = [p.shape for p in self.params]
        kind = torch.float8_e4m3fn if state_bits == 8 else torch.float32
        self.exp_avg = self._state("exp_avg", exp_avg, kind, False)
        self.exp_avg_sq = self._state("exp_avg_sq", exp_avg_sq, kind, False)
        self.exp_avg_scale = self.exp_avg_sq_scale = None
        if state_bits == 8:
            self.exp_avg_scale = self._state("exp_avg_scale", exp_avg_scale, torch.float32, True)
            self.exp_avg_sq_scale = self._state("exp_avg_sq_scale", exp_avg_sq_scale, torch.float32, True)
        else:
            c.need(exp_avg_scale is None and exp_avg_sq_scale is None, "AdamW: scales belong to state_bits=8")
        self.copies = None
        if copies is not None:
            self.copies = list(copies)
            c.need(len(self.copies) == n, "AdamW: copies must have one entry (a tensor or None) per parameter")
            for i, (t, p) in enumerate(zip(self.copies, self.params)):
                if t is not None:
                    self._alike(f"copies[{i}]", t, p.shape, torch.bfloat16)
        self._table = np.zeros(n, _ENTRY)
        self._table["numel"] = [p.numel() for p in self.params]
        self._table["param_bf16"] = [p.dtype == torch.bfloat16 for p in self.params]

    def _alike(self, what, t, shape, dtype):
        c.need(isinstance(t, torch.Tensor) and t.device == self.device, f"AdamW: {what} must be on {self.device}")
        c.need(t.dtype == dtype, f"AdamW: {what} must be {dtype}", TypeError)
        c.need(t.shape == shape and t.is_contiguous(), f"AdamW: {what} must be contiguous with shape {tuple(shape)}")

    def _state(self, what, given, dtype, scales):
        shapes = [torch.Size((-(-p.numel() // _BLOCK),)) if scales else p.shape for p in self.params]
        if given is None:
            return [torch.zeros(s, dtype=dtype, device=self.device) for s in shapes]
        given = list(given)
        c.need(len(given) == len(shapes), f"AdamW: {what} must have one tensor per parameter")
        for i, (t, s) in enumerate(zip(given, shapes)):
            self._alike(f"{what}[{i}]", t, s, dtype)
        return given

    def step(self, grads, lr=None, grad_scale=1.0, stream=None):
        """One update.  lr overrides the constructor's for this step (a schedule); the
        gradients are multiplied by grad_scale, a number or a one-element fp32 CUDA tensor (a
        clipping coefficient computed on the device, read without synchronising)."""
        from . import _check as status, lib
        grads = list(grads)
        c.need(len(grads) == len(self.params), "AdamW.step: grads must have one entry (a tensor or None) per parameter")
        t = self._table
        for g, shape in zip(grads, self._shapes):
            if g is not None and not (
                    g.shape == shape and g.is_contiguous() and g.device == self.device and
                    (g.dtype is torch.bfloat16 or g.dtype is torch.float32)):
                raise ValueError(f"AdamW.step: a gradient must be contiguous, float32 or bfloat16, on {self.device}, of its "
                                 f"parameter's shape {tuple(shape)}")
        t["grad"] = [0 if g is None else g.data_ptr() for g in grads]
        t["grad_bf16"] = [g is not None and g.dtype is torch.bfloat16 for g in grads]
        t["param"] = [p.data_ptr() for p in self.params]
        t["exp_avg"] = [x.data_ptr() for x in self.exp_avg]
        t["exp_avg_sq"] = [x.data_ptr() for x in self.exp_avg_sq]
        if self.state_bits == 8:
            t["exp_avg_scale"] = [x.data_ptr() for x in self.exp_avg_scale]
            t["exp_avg_sq_scale"] = [x.data_ptr() for x in self.exp_avg_sq_scale]
        if self.copies is not None:
            t["copy"] = [0 if x is None else x.data_ptr() for x in self.copies]
        h = _Hyper(self.lr if lr is None else lr, self.betas[0], self.betas[1], self.eps, self.weight_decay, 1.0, None,
                   self.step_count + 1)
        if isinstance(grad_scale, torch.Tensor):
            c.need(grad_scale.numel() == 1 and grad_scale.dtype == torch.float32 and grad_scale.device == self.device,
                   "AdamW.step: a grad_scale tensor must hold one float32 on the parameters' device")
            h.grad_scale_ptr = grad_scale.data_ptr()
        else:
            h.grad_scale = float(grad_scale)
        used = () if stream is None else (*(g for g in grads if g is not None), *self.params, *self.exp_avg, *self.exp_avg_sq,
                                          *(self.exp_avg_scale or ()), *(self.exp_avg_sq_scale or ()),
                                          *(x for x in self.copies or () if x is not None))
        with c.on_stream(self.device, stream, used) as st:
            status(lib().dp_adamw_step(t.ctypes.data_as(c.P), len(self.params), self.state_bits, ctypes.byref(h), st), "dp_adamw_step")
        self.step_count += 1
