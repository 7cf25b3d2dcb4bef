"""Refusals of the grouped, 8-bit and AdamW entry points, on a host without a GPU: argument
checks come before any device call."""
import ctypes

import pytest
import torch

import fp32_dense_projection_gb300 as dp
from fp32_dense_projection_gb300 import build as dpbuild
from fp32_dense_projection_gb300.adamw import _ENTRY, _Hyper

OK, INVALID, ALIGNMENT, UNSUPPORTED = 0, 1, 2, 3
A = 1 << 20  # an aligned, never dereferenced address


@pytest.fixture(scope="module")
def L():
    dpbuild.build()
    return dp.lib()


def grouped(L, op="fwd", a=A, lda=0, w=A, ldw=0, bsw=0, kn=0, offs=A, bits=32, out=A, ldo=0, bso=0, E=4, T=64, N=64, K=64, code=0):
    if op == "wgrad":
        return L.dp_gemm_wgrad_grouped(a, lda, w, ldw, offs, bits, out, ldo, bso, kn, E, T, N, K, code, None)
    return getattr(L, f"dp_gemm_{op}_grouped")(a, lda, w, ldw, bsw, kn, offs, bits, out, ldo, E, T, N, K, code, None)


@pytest.mark.parametrize("op", ["fwd", "dgrad", "wgrad"])
@pytest.mark.parametrize("kw,want", [
    (dict(code=2), INVALID), (dict(kn=2), INVALID), (dict(E=-1), INVALID), (dict(T=-1), INVALID), (dict(N=0), INVALID),
    (dict(K=0), INVALID), (dict(bits=16), INVALID), (dict(offs=None), INVALID), (dict(a=None), INVALID), (dict(w=None), INVALID),
    (dict(out=None), INVALID), (dict(lda=8), INVALID), (dict(ldw=8), INVALID), (dict(ldo=8), INVALID),
    (dict(N=60), UNSUPPORTED), (dict(K=12), UNSUPPORTED), (dict(E=1025), UNSUPPORTED), (dict(T=2 ** 31), UNSUPPORTED),
    (dict(a=A + 8), ALIGNMENT), (dict(w=A + 2), ALIGNMENT), (dict(out=A + 8), ALIGNMENT), (dict(offs=A + 2), ALIGNMENT),
    (dict(offs=A + 4, bits=64), ALIGNMENT), (dict(lda=67), ALIGNMENT), (dict(ldw=67), ALIGNMENT),
])
def test_grouped_refusals(L, op, kw, want):
    assert grouped(L, op, **kw) == want


def test_grouped_expert_strides(L):
    assert grouped(L, "fwd", bsw=-8) == INVALID and grouped(L, "fwd", bsw=4097) == ALIGNMENT
    assert grouped(L, "wgrad", bso=-8) == INVALID and grouped(L, "wgrad", bso=4097) == ALIGNMENT


def fp8(L, op="fwd", a=A, lda=0, fa=0, sa=A, sa1=1, sa2=1, b=A, ldb=0, fb=0, sb=A, sb1=1, sb2=1, out=A, ldo=0, T=64, N=64, K=64, code=0):
    return getattr(L, f"dp_gemm_{op}_fp8")(a, lda, fa, sa, sa1, sa2, b, ldb, fb, sb, sb1, sb2, out, ldo, T, N, K, code, None)


@pytest.mark.parametrize("op", ["fwd", "dgrad", "wgrad"])
@pytest.mark.parametrize("kw,want", [
    (dict(code=-1), INVALID), (dict(fa=2), INVALID), (dict(fb=-1), INVALID), (dict(T=-1), INVALID), (dict(N=0), INVALID),
    (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(out=None), INVALID), (dict(sa=None), INVALID), (dict(sb=None), INVALID),
    (dict(sa1=-1), INVALID), (dict(sb2=-1), INVALID), (dict(lda=16), INVALID), (dict(ldb=16), INVALID), (dict(ldo=16), INVALID),
    (dict(N=72), UNSUPPORTED), (dict(K=8), UNSUPPORTED), (dict(T=2 ** 31), UNSUPPORTED), (dict(a=A + 8), ALIGNMENT),
    (dict(b=A + 8), ALIGNMENT), (dict(out=A + 4), ALIGNMENT), (dict(sa=A + 2), ALIGNMENT), (dict(lda=72), ALIGNMENT),
])
def test_fp8_refusals(L, op, kw, want):
    assert fp8(L, op, **kw) == want


def quantize(L, x=A, ldx=0, f32=0, rows=64, cols=64, scaling=3, fmt=0, q=A, ldq=0, s=A, s_row=1, s_col=64, qc=A, ldqc=0, sc=A, sc_row=64):
    return L.dp_fp8_quantize(x, ldx, f32, rows, cols, scaling, fmt, q, ldq, s, s_row, s_col, qc, ldqc, sc, sc_row, None)


@pytest.mark.parametrize("kw,want", [
    (dict(scaling=4), INVALID), (dict(fmt=2), INVALID), (dict(f32=2), INVALID), (dict(rows=-1), INVALID), (dict(cols=0), INVALID),
    (dict(cols=40), UNSUPPORTED), (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID), (dict(qc=None), INVALID),
    (dict(sc=None), INVALID), (dict(sc_row=60), INVALID), (dict(sc_row=66), ALIGNMENT), (dict(sc=A + 4), ALIGNMENT),
    (dict(s=A + 2), ALIGNMENT), (dict(x=A + 8), ALIGNMENT), (dict(q=A + 4), ALIGNMENT), (dict(s_row=-1), INVALID),
    (dict(scaling=0, q=None), INVALID), (dict(scaling=1, sc=None), INVALID), (dict(ldx=32), INVALID), (dict(ldq=72), ALIGNMENT),
])
def test_quantize_refusals(L, kw, want):
    assert quantize(L, **kw) == want


def adamw(L, bits=32, count=1, table=True, hyper=None, **fields):
    import numpy as np
    t = np.zeros(1, _ENTRY)
    for k, v in dict(param=A, grad=A, exp_avg=A, exp_avg_sq=A, exp_avg_scale=A, exp_avg_sq_scale=A, numel=64, **{}).items():
        t[k] = fields.get(k, v)
    for k in ("copy", "param_bf16", "grad_bf16"):
        t[k] = fields.get(k, 0)
    h = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, grad_scale=1.0, grad_scale_ptr=None, step=1)
    h.update(hyper or {})
    return L.dp_adamw_step(t.ctypes.data if table else None, count, bits, ctypes.byref(_Hyper(**h)), None)


@pytest.mark.parametrize("kw,want", [
    (dict(bits=16), INVALID), (dict(count=-1), INVALID), (dict(table=False), INVALID), (dict(numel=-1), INVALID), (dict(param=0), INVALID),
    (dict(exp_avg=0), INVALID), (dict(exp_avg_sq=0), INVALID), (dict(bits=8, exp_avg_scale=0), INVALID),
    (dict(bits=8, exp_avg_sq_scale=0), INVALID), (dict(param=A + 2), ALIGNMENT), (dict(grad=A + 1, grad_bf16=1), ALIGNMENT),
    (dict(exp_avg=A + 2), ALIGNMENT), (dict(copy=A + 1), ALIGNMENT), (dict(exp_avg_scale=A + 2), ALIGNMENT),
    (dict(hyper=dict(lr=-1.0)), INVALID), (dict(hyper=dict(lr=float("nan"))), INVALID), (dict(hyper=dict(beta1=1.0)), INVALID),
    (dict(hyper=dict(beta2=-0.1)), INVALID), (dict(hyper=dict(eps=-1.0)), INVALID), (dict(hyper=dict(weight_decay=-1.0)), INVALID),
    (dict(hyper=dict(step=0)), INVALID), (dict(hyper=dict(grad_scale_ptr=A + 2)), ALIGNMENT),
])
def test_adamw_refusals(L, kw, want):
    assert adamw(L, **kw) == want


def test_python_refusals():
    x, w, o = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(2, 64, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    for f in (lambda: dp.dp_gemm_fwd_grouped(x, w, o), lambda: dp.dp_gemm_dgrad_grouped(x, w, o), lambda: dp.dp_gemm_wgrad_grouped(x, x, o),
              lambda: dp.fp8_quantize(x), lambda: dp.AdamW([x])):
        with pytest.raises(ValueError, match="CUDA tensor"):
            f()
    with pytest.raises(ValueError, match="weight_layout"):
        dp.dp_gemm_fwd_grouped(x, w, o, weight_layout="kk")
    with pytest.raises(ValueError, match="does not match"):
        dp.dp_gemm_fwd_grouped(x[:, :32], w, o)
    with pytest.raises(ValueError, match="scaling"):
        dp.fp8_quantize(x, scaling="tile")
    with pytest.raises(TypeError, match="dtype"):
        dp.fp8_quantize(x, dtype=torch.int8)
    with pytest.raises(ValueError, match="state_bits"):
        dp.AdamW([x], state_bits=16)
