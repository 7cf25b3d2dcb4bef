"""AdamW over many tensors in one launch, moments in 32 or 8 bits.

  opt = AdamW(params, lr=1e-3, state_bits=8, copies=bf16_weights)
  opt.step(grads, grad_scale=clip)

params are dense fp32 or bf16 CUDA tensors, updated in place; grads fp32 or bf16, one per
parameter (None: that parameter, its moments and its count of updates are left as they are).
copies are optional bf16 tensors that
receive the updated parameter: the working weights of the GEMMs beside fp32 master weights.
"""
from __future__ import annotations

import ctypes
from operator import attrgetter

import numpy as np
import torch

from . import _call as c

_BLOCK = 128
_ENTRY = np.dtype([("param", "u8"), ("grad", "u8"), ("exp_avg", "u8"), ("exp_avg_sq", "u8"), ("exp_avg_scale", "u8"),
                   ("exp_avg_sq_scale", "u8"), ("copy", "u8"), ("numel", "i8"), ("param_bf16", "i4"), ("grad_bf16", "i4")])


class _Hyper(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay", "grad_scale")] + [
        ("grad_scale_ptr", ctypes.c_void_p), ("step", ctypes.c_int64)]


_fn = {}


def _bind(L):
    L.dp_adamw_step.argtypes = [c.P, c.I, c.S, ctypes.POINTER(_Hyper), c.P]
    _fn["step"] = L.dp_adamw_step


_increment_version = torch.autograd.graph.increment_version
_capturing = torch._C._cuda_isCurrentStreamCapturing
_data_ptr, _is_contiguous, _get_device = torch.Tensor.data_ptr, torch.Tensor.is_contiguous, torch.Tensor.get_device
_numel = torch.Tensor.numel
_shape, _dtype = attrgetter("shape"), attrgetter("dtype")
_F32, _BF16 = torch.float32, torch.bfloat16


def _need(ok, what, kind=ValueError):
    if not ok:
        raise kind(f"AdamW: {what}")


def _scale_shape(shape):
    return torch.Size((-(-shape.numel() // _BLOCK),))


class AdamW:
    """AdamW with decoupled weight decay over a list of tensors.

    state_bits=32 keeps both moments in fp32.  state_bits=8 keeps them as float8_e4m3fn
    codes with an fp32 scale per 128 consecutive elements: ``exp_avg`` holds m / scale,
    ``exp_avg_sq`` holds sqrt(v) / scale.  Codes of moments with a long memory (sqrt(v) above
    beta2 = 0.95, m above beta1 = 0.98) are rounded stochastically, by a hash of element and
    step (a run repeats bit for bit): rounded to nearest they would not follow small changes.

    The moments are attributes (tuples of tensors) and may be passed in, with ``step`` the
    updates already done (a number, or one per parameter as in ``steps``), to resume a run.
    ``step_count`` counts the calls of ``step``; a parameter's bias corrections go by the
    updates that it had.

    The updates are made in place, outside autograd; they raise the versions of parameters
    and copies, so that a backward pass that has saved one of them refuses to use what it has
    become.  The lists of tensors are fixed at construction; the tensors may get new memory
    between steps (``.data``), of their shape, but not share it.  A step cannot be captured
    into a CUDA graph: its count and rate are arguments of the launch.
    """

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2, state_bits=32, copies=None,
                 exp_avg=None, exp_avg_sq=None, exp_avg_scale=None, exp_avg_sq_scale=None, step=0):
        _need(state_bits in (8, 32), "state_bits must be 8 or 32")
        _need(len(betas) == 2 and all(0.0 <= b < 1.0 for b in betas), "betas must lie in [0, 1)")
        _need(lr >= 0 and eps >= 0 and weight_decay >= 0, "lr, eps and weight_decay must not be negative")
        self.params = tuple(params)
        steps = [int(x) for x in step] if isinstance(step, (list, tuple)) else [int(step)] * len(self.params)
        _need(len(steps) == len(self.params), "step must be a number or have one entry per parameter")
        _need(min(steps, default=0) >= 0, "step must not be negative")
        self.lr, self.betas, self.eps, self.weight_decay = lr, tuple(betas), eps, weight_decay
        self.state_bits, self.step_count = state_bits, max(steps, default=0)
        self._missed = [self.step_count - x for x in steps] if len(set(steps)) > 1 else None  # per parameter; None: none
        n = len(self.params)
        self.device = None
        for i, p in enumerate(self.params):
            _need(isinstance(p, torch.Tensor) and p.is_cuda, f"params[{i}] must be a CUDA tensor")
            self.device = self.device or p.device
            _need(p.device == self.device, f"params[{i}] is on {p.device}, params[0] on {self.device}")
        self.copies = None if copies is None else tuple(copies)
        _need(copies is None or len(self.copies) == n, "copies must have one entry (a tensor or None) per parameter")
        self._table = np.zeros(n, _ENTRY)
        self._shapes = [p.shape for p in self.params]
        kind = torch.float8_e4m3fn if state_bits == 8 else _F32
        m = self._moments = {"exp_avg": self._state(exp_avg, kind, False), "exp_avg_sq": self._state(exp_avg_sq, kind, False),
                             "exp_avg_scale": None, "exp_avg_sq_scale": None}
        if state_bits == 8:
            m["exp_avg_scale"] = self._state(exp_avg_scale, _F32, True)
            m["exp_avg_sq_scale"] = self._state(exp_avg_sq_scale, _F32, True)
        else:
            _need(exp_avg_scale is None and exp_avg_sq_scale is None, "scales belong to state_bits=8")
        self._held = tuple(x for t in (self.params, self.copies, *m.values()) for x in t or () if x is not None)
        # tensors that someone else may hold: all, until then without the moments made here
        given = any(x is not None for x in (exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale))
        self._watched = self._held if given else self._held[:len(self._held) - sum(len(t) for t in m.values() if t is not None)]
        self._enter()

    def _moment(name):
        def get(self):
            if self._watched is not self._held:
                self._watched = self._held
                self._note()
            return self._moments[name]
        return property(get)

    exp_avg, exp_avg_sq = _moment("exp_avg"), _moment("exp_avg_sq")
    exp_avg_scale, exp_avg_sq_scale = _moment("exp_avg_scale"), _moment("exp_avg_sq_scale")
    del _moment

    def _alike(self, what, t, shape, dtypes):
        _need(isinstance(t, torch.Tensor) and t.device == self.device, f"{what} must be on {self.device}")
        _need(t.dtype in dtypes, f"{what} must be {' or '.join(map(str, dtypes))}", TypeError)
        _need(t.shape == shape and t.is_contiguous(), f"{what} must be contiguous with shape {tuple(shape)}")

    def _changed(self):
        """Whether a parameter, copy or moment is not what was entered: its .data may have been
        replaced, also by another view or type at the same address.  (As many elements of the same
        type in one piece there are the same elements; a shape is four times as dear to read as their number.)"""
        watched = self._watched
        return (list(map(_data_ptr, self._held)) != self._pointers or list(map(_dtype, watched)) != self._dtypes or
                list(map(_numel, watched)) != self._numels or False in map(_is_contiguous, watched))

    def _note(self):
        """What later steps compare with."""
        self._pointers = list(map(_data_ptr, self._held))
        self._dtypes, self._numels = list(map(_dtype, self._watched)), list(map(_numel, self._watched))

    def _enter(self):
        """Check the tensors and then enter them in the table (all of them or, if one is refused, none)."""
        kind = torch.float8_e4m3fn if self.state_bits == 8 else _F32
        columns = {}
        for what, tensors in {"param": self.params, "copy": self.copies, **self._moments}.items():
            if tensors is None:
                continue
            name = {"param": "params", "copy": "copies"}.get(what, what)
            _need(len(tensors) == len(self._shapes), f"{name} must have one tensor per parameter")
            dtypes = {"param": (_F32, _BF16), "copy": (_BF16,)}.get(what, (_F32,) if "scale" in what else (kind,))
            for i, (x, shape) in enumerate(zip(tensors, self._shapes)):
                if x is not None or what != "copy":
                    self._alike(f"{name}[{i}]", x, _scale_shape(shape) if "scale" in what else shape, dtypes)
            columns[what] = [0 if x is None else x.data_ptr() for x in tensors]
        # (blocks of one launch write each tensor without regard to the others; a BF16 parameter may be its own copy)
        own = {id(q) for p, q in zip(self.params, self.copies or ()) if q is not None and q.data_ptr() == p.data_ptr() and
               q.nbytes == p.nbytes}
        spans = sorted((x.data_ptr(), x.nbytes) for i, x in enumerate(self._held)
                       if x.numel() and (i < len(self.params) or id(x) not in own))
        for (a, size), (b, _) in zip(spans, spans[1:]):
            _need(a + size <= b, "params, copies and moments must not share memory (a tied weight is one parameter)")
        for what, column in columns.items():
            self._table[what] = column
        self._table["numel"] = [p.numel() for p in self.params]
        self._table["param_bf16"] = [p.dtype is _BF16 for p in self.params]
        # (inference tensors have no version)
        self._versioned = [tuple(x for x in (p, q) if x is not None and not x.is_inference())
                           for p, q in zip(self.params, self.copies or [None] * len(self.params))]
        self._all_versioned = tuple(x for group in self._versioned for x in group)
        self._grad_dtypes = None
        self._note()

    def _state(self, given, dtype, scales):
        if given is None:
            given = (torch.zeros(_scale_shape(p.shape) if scales else p.shape, dtype=dtype, device=self.device)
                     for p in self.params)
        return tuple(given)

    @property
    def steps(self):
        """Updates that each parameter had."""
        return tuple(self.step_count - x for x in self._missed or [0] * len(self.params))

    def step(self, grads, lr=None, grad_scale=1.0, stream=None):
        """One update.  lr overrides the constructor's for this step (a schedule); the
        gradients are multiplied by grad_scale, a number or a one-element fp32 CUDA tensor (a
        clipping coefficient computed on the device, read without synchronising)."""
        grads = list(grads)
        _need(len(grads) == len(self.params), "grads must have one entry (a tensor or None) per parameter")
        if not grads:
            self.step_count += 1
            return
        if self._changed():
            self._enter()
        index = self.device.index
        some = [g for g in grads if g is not None]
        shapes = self._shapes if len(some) == len(grads) else [s for g, s in zip(grads, self._shapes) if g is not None]
        dtypes = list(map(_dtype, some))
        if (list(map(_shape, some)) != shapes or False in map(_is_contiguous, some) or set(map(_get_device, some)) - {index} or
                set(dtypes) - {_F32, _BF16}):
            raise ValueError(f"AdamW.step: every gradient must be contiguous, float32 or bfloat16, on {self.device} and of its "
                             "parameter's shape")
        t = self._table
        at = list(map(_data_ptr, some)) if len(some) == len(grads) else [0 if g is None else g.data_ptr() for g in grads]
        if len(some) != len(grads):
            t["grad_bf16"] = [g is not None and g.dtype is _BF16 for g in grads]
            self._grad_dtypes = None
        elif dtypes != self._grad_dtypes:
            t["grad_bf16"] = [d is _BF16 for d in dtypes]
            self._grad_dtypes = dtypes
        h = _Hyper(self.lr if lr is None else lr, self.betas[0], self.betas[1], self.eps, self.weight_decay, 1.0, None, 0)
        if isinstance(grad_scale, torch.Tensor):
            if grad_scale.numel() != 1 or grad_scale.dtype is not _F32 or grad_scale.get_device() != index:
                raise ValueError("AdamW.step: a grad_scale tensor must hold one float32 on the parameters' device")
            h.grad_scale_ptr = grad_scale.data_ptr()
        else:
            h.grad_scale = float(grad_scale)
        used = () if stream is None else (*some, *self._held, *((grad_scale,) if isinstance(grad_scale, torch.Tensor) else ()))
        if not _fn:
            c.load()

        def work(st):
            if _capturing():  # (a replay would repeat this step's corrections and rate)
                raise RuntimeError("AdamW.step: a step cannot be captured: its count and rate are arguments of its launch")
            # one call for the parameters that have had the same number of updates
            for missed in (0,) if self._missed is None else {x for x, a in zip(self._missed, at) if a}:
                t["grad"] = at if self._missed is None else [a if x == missed else 0 for x, a in zip(self._missed, at)]
                h.step = self.step_count + 1 - missed
                code = _fn["step"](t.ctypes.data, len(grads), self.state_bits, ctypes.byref(h), st)
                if code:
                    return code
            return 0
        code = c.on_stream(index, stream, used, work)
        if code:
            c.check(code, "dp_adamw_step")
        self.step_count += 1
        if len(some) == len(grads):
            _increment_version(self._all_versioned)
        else:
            _increment_version([x for group, g in zip(self._versioned, grads) if g is not None for x in group])
            self._missed = [x + (g is None) for x, g in zip(self._missed or [0] * len(grads), grads)]
