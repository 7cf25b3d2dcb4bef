"""The way of tokens to their experts and back, around the products grouped by expert.

  route_topk(logits, k)                             (gates, choice): the k experts of each token
  route_topk_bwd(d_gates, logits, gates, choice)    d_logits
  expert_sort(choice, E)                            (offsets, row_of, order): the pairs sorted by expert
  expert_gather(x, row_of)                          the tokens' rows in that order
  expert_combine(y, row_of, gates)                  the experts' rows back, weighted; without gates the
                                                    gradient of expert_gather
  expert_combine_bwd(d_out, y, row_of, gates)       (d_y, d_gates)

A pair is a token and one of its k choices.  ``offsets`` is what the grouped products read; nothing
is read back to the host.  Pairs without an expert (choice outside [0, E), as route_topk gives
where experts are closed by logits of -infinity) stand behind the last group, with zero rows.
"""
from __future__ import annotations

import ctypes

import torch

from . import _call as c

_I32 = torch.int32
_BITS = {torch.int32: 32, torch.int64: 64}
_ROW_TYPES = {c.BF16: 0, c.F32: 1}
_NO_WORKSPACE = 4  # DP_ERR_WORKSPACE
_fn = {}


def _bind(L):
    P, I, S, Z = c.P, c.I, c.S, ctypes.c_size_t
    L.dp_route_topk.argtypes = [P, I, P, P, I, I, I, S, P]
    L.dp_route_topk_bwd.argtypes = [P, P, I, P, P, P, I, I, I, I, S, P]
    L.dp_expert_sort.argtypes = [P, S, I, I, P, P, P, P, Z, P]
    L.dp_expert_sort_workspace_size.argtypes = [I, I, ctypes.POINTER(Z)]
    L.dp_expert_gather.argtypes = [P, I, S, P, P, I, I, I, I, P]
    L.dp_expert_combine.argtypes = [P, I, S, P, P, P, I, P, I, S, I, I, I, P]
    L.dp_expert_combine_bwd.argtypes = [P, I, S, P, I, S, P, P, P, I, S, P, I, I, I, P]
    names = ("dp_route_topk", "dp_route_topk_bwd", "dp_expert_sort", "dp_expert_sort_workspace_size", "dp_expert_gather",
             "dp_expert_combine", "dp_expert_combine_bwd")
    _fn.update({name: getattr(L, name) for name in names})


def _need(t, shape, dtype, name, what):
    if t.dtype is not dtype:
        raise TypeError(f"{name}: {what} must be {str(dtype).removeprefix('torch.')}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: {what} must be contiguous with shape {tuple(shape)}")


def _kind(t, name, what):
    kind = _ROW_TYPES.get(t.dtype)
    if kind is None:
        raise TypeError(f"{name}: {what} must be bfloat16 or float32")
    return kind


def route_topk(logits, k, renormalize=True, stream=None):
    """(gates [T,k] fp32, choice [T,k] int32) from logits [T,E] (fp32; E at most 1024, k at most 32): the
    largest first, the lowest index first among equals.  Gates are the softmax over the chosen
    (renormalize) or over all experts.  Experts with logits of -infinity are closed: where fewer
    than k are open, choice is -1 and the gate 0."""
    name = "route_topk"
    index = logits.get_device()
    if index < 0:
        c.refuse_devices(name, {"logits": logits})
    if logits.dtype is not c.F32:
        raise TypeError(f"{name}: logits must be float32")
    ld = c.ld(logits, name, "logits")
    T, E = logits.shape
    if not 1 <= k <= E:
        raise ValueError(f"{name}: k must lie in 1 .. E")
    if not _fn:
        c.load()

    def work(st):
        gates = c.new((T, k), c.F32)
        choice = c.new((T, k), _I32)
        code = _fn["dp_route_topk"](logits.data_ptr(), ld, gates.data_ptr(), choice.data_ptr(), T, E, k, bool(renormalize), st)
        if code:
            c.check(code, name)
        return gates, choice

    return c.on_stream(index, stream, (logits,), work)


def route_topk_bwd(d_gates, logits, gates, choice, renormalize=True, out=None, stream=None):
    """d_logits [T,E] (fp32) from d_gates [T,k] (fp32) and what route_topk read and returned."""
    name = "route_topk_bwd"
    index = d_gates.get_device()
    if index < 0 or logits.get_device() != index or gates.get_device() != index or choice.get_device() != index:
        c.refuse_devices(name, {"d_gates": d_gates, "logits": logits, "gates": gates, "choice": choice})
    if logits.dtype is not c.F32:
        raise TypeError(f"{name}: logits must be float32")
    ld = c.ld(logits, name, "logits")
    T, E = shape = logits.shape
    if gates.dim() != 2:
        raise ValueError(f"{name}: gates must be [T, k]")
    k = gates.shape[1]
    _need(gates, (T, k), c.F32, name, "gates")
    _need(d_gates, (T, k), c.F32, name, "d_gates")
    _need(choice, (T, k), _I32, name, "choice")
    if out is not None and out.dtype is not c.F32:
        raise TypeError(f"{name}: out must be float32")
    if not _fn:
        c.load()

    def work(st):
        d, _, ldd = c.output_rows(out, shape, c.F32, index, logits.device, name)
        code = _fn["dp_route_topk_bwd"](d_gates.data_ptr(), logits.data_ptr(), ld, gates.data_ptr(), choice.data_ptr(), d.data_ptr(),
                                        ldd, T, E, k, bool(renormalize), st)
        if code:
            c.check(code, name)
        return d

    return c.on_stream(index, stream, (d_gates, logits, gates, choice, out), work)


def expert_sort(choice, E, workspace=None, stream=None):
    """(offsets [E + 1], row_of like choice, order [pairs]), all int32, from choice (int32 or int64, [T,k]).
    Pair p goes to row row_of[p] of the sorted buffer, expert e has the rows offsets[e] .. offsets[e + 1],
    and row r comes from pair order[r].  A pair without an expert has ~row (below zero) in row_of."""
    name = "expert_sort"
    index = choice.get_device()
    if index < 0 or (workspace is not None and workspace.get_device() != index):
        c.refuse_devices(name, {"choice": choice} if workspace is None else {"choice": choice, "workspace": workspace})
    bits = _BITS.get(choice.dtype)
    if bits is None:
        raise TypeError(f"{name}: choice must be int32 or int64")
    if not choice.is_contiguous():
        raise ValueError(f"{name}: choice must be contiguous")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError(f"{name}: workspace must be contiguous")
    pairs, device = choice.numel(), choice.device
    if not _fn:
        c.load()

    def work(st):
        offsets = c.new_vector(E + 1 if E > 0 else 1, _I32)
        row_of = c.new(choice.shape, _I32)
        order = c.new_vector(pairs, _I32)
        buf, size = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
        args = (choice.data_ptr(), bits, pairs, E, offsets.data_ptr(), row_of.data_ptr(), order.data_ptr())
        code = _fn["dp_expert_sort"](*args, buf, size, st)
        if code == _NO_WORKSPACE and workspace is None:  # (very many pairs: nothing has been launched)
            n = ctypes.c_size_t(0)
            code = _fn["dp_expert_sort_workspace_size"](pairs, E, ctypes.byref(n))
            if not code:
                buf = c.new_vector(n.value, torch.uint8)
                code = _fn["dp_expert_sort"](*args, buf.data_ptr(), n.value, st)
        if code:
            c.check(code, name)
        return offsets, row_of, order

    return c.on_stream(index, stream, (choice, workspace), work)


def _pairs(row_of, name):
    """(T, k) of the pairs' rows."""
    if row_of.dtype is not _I32:
        raise TypeError(f"{name}: row_of must be int32")
    if row_of.dim() != 2 or not row_of.is_contiguous():
        raise ValueError(f"{name}: row_of must be contiguous [T, k]")
    return row_of.shape


def _matrix(t, shape, name, what):
    if t.shape != shape:
        raise ValueError(f"{name}: {what} must have shape {tuple(shape)}")
    return c.ld(t, name, what, shape)


def expert_gather(x, row_of, out=None, stream=None):
    """rows [T k, C] with rows[row_of[t, j]] = x[t] (bf16 or fp32, as x), zero for pairs without an expert."""
    name = "expert_gather"
    index = x.get_device()
    if index < 0 or row_of.get_device() != index:
        c.refuse_devices(name, {"x": x, "row_of": row_of})
    f32, ldx = _kind(x, name, "x"), c.ld(x, name, "x")
    T, k = _pairs(row_of, name)
    C = x.shape[1]
    if x.shape[0] != T:
        raise ValueError(f"{name}: x and row_of must have the same tokens")
    if out is not None and out.dtype is not x.dtype:
        raise TypeError(f"{name}: out must have x's type")
    if not _fn:
        c.load()

    def work(st):
        shape = (T * k, C)
        rows, _, ldr = c.output_rows(out, shape, x.dtype, index, x.device, name)
        code = _fn["dp_expert_gather"](x.data_ptr(), ldx, f32, row_of.data_ptr(), rows.data_ptr(), ldr, T, k, C, st)
        if code:
            c.check(code, name)
        return rows

    return c.on_stream(index, stream, (x, row_of, out), work)


def expert_combine(y, row_of, gates=None, add=None, out=None, out_dtype=c.BF16, stream=None):
    """out [T,C] = add + sum_j gates[t, j] y[row_of[t, j]] over the pairs that have an expert: y [T k, C]
    bf16 or fp32, gates [T,k] fp32 or None (1), add [T,C] of out's type or None (0)."""
    name = "expert_combine"
    index = y.get_device()
    if (index < 0 or row_of.get_device() != index or (gates is not None and gates.get_device() != index) or
            (add is not None and add.get_device() != index)):
        tensors = {"y": y, "row_of": row_of, "gates": gates, "add": add}
        c.refuse_devices(name, {what: t for what, t in tensors.items() if t is not None})
    f32 = _kind(y, name, "y")
    T, k = _pairs(row_of, name)
    if y.dim() != 2:
        raise ValueError(f"{name}: y must be [T k, C]")
    C = y.shape[1]
    ldy = _matrix(y, (T * k, C), name, "y")
    shape, lda = (T, C), 0
    if gates is not None:
        _need(gates, (T, k), c.F32, name, "gates")
    if add is not None:
        if add.dtype is not (out_dtype if out is None else out.dtype):
            raise TypeError(f"{name}: add must have out's type")
        lda = _matrix(add, shape, name, "add")
    if not _fn:
        c.load()

    def work(st):
        o, code, ldo = c.output_rows(out, shape, out_dtype, index, y.device, name)
        code = _fn["dp_expert_combine"](y.data_ptr(), ldy, f32, row_of.data_ptr(), None if gates is None else gates.data_ptr(),
                                        None if add is None else add.data_ptr(), lda, o.data_ptr(), ldo, code, T, k, C, st)
        if code:
            c.check(code, name)
        return o

    return c.on_stream(index, stream, (y, row_of, gates, add, out), work)


def expert_combine_bwd(d_out, y, row_of, gates, d_y=None, dy_dtype=c.BF16, stream=None):
    """(d_y [T k, C], d_gates [T,k] fp32) from d_out [T,C] (the gradient of ``add`` is d_out itself)."""
    name = "expert_combine_bwd"
    index = d_out.get_device()
    if index < 0 or y.get_device() != index or row_of.get_device() != index or gates.get_device() != index:
        c.refuse_devices(name, {"d_out": d_out, "y": y, "row_of": row_of, "gates": gates})
    d32, y32 = _kind(d_out, name, "d_out"), _kind(y, name, "y")
    T, k = _pairs(row_of, name)
    if d_out.dim() != 2:
        raise ValueError(f"{name}: d_out must be [T, C]")
    C = d_out.shape[1]
    shape = (T * k, C)
    ldd, ldy = _matrix(d_out, (T, C), name, "d_out"), _matrix(y, shape, name, "y")
    _need(gates, (T, k), c.F32, name, "gates")
    if not _fn:
        c.load()

    def work(st):
        d, code, ld_dy = c.output_rows(d_y, shape, dy_dtype, index, y.device, name, "d_y")
        d_gates = c.new((T, k), c.F32)
        code = _fn["dp_expert_combine_bwd"](d_out.data_ptr(), ldd, d32, y.data_ptr(), ldy, y32, row_of.data_ptr(), gates.data_ptr(),
                                            d.data_ptr(), ld_dy, code, d_gates.data_ptr(), T, k, C, st)
        if code:
            c.check(code, name)
        return d, d_gates

    return c.on_stream(index, stream, (d_out, y, row_of, gates, d_y), work)
