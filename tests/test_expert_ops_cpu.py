"""Refusals of the layer norm, expert and 4-bit entry points, on a host without a GPU: argument checks come before any
device call."""
import ctypes

import pytest
import torch

import fp32_dense_projection_gb300 as dp
from fp32_dense_projection_gb300 import build as dpbuild

OK, INVALID, ALIGNMENT, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4
A = 1 << 20  # an aligned, never dereferenced address


@pytest.fixture(scope="module")
def L():
    dpbuild.build()
    return dp.lib()


def norm_fwd(L, x=A, ldx=0, x32=0, w=A, b=A, w32=0, eps=1e-5, y=A, ldy=0, out=0, mean=A, rstd=A, T=4, C=64):
    return L.dp_layer_norm_fwd(x, ldx, x32, w, b, w32, eps, y, ldy, out, mean, rstd, T, C, None)


def norm_bwd(L, g=A, ldg=0, g32=0, x=A, ldx=0, x32=0, mean=A, rstd=A, w=A, w32=0, y=A, ldy=0, out=0, dw=A, db=A, T=4, C=64, ws=A, size=1 << 30):
    return L.dp_layer_norm_bwd(g, ldg, g32, x, ldx, x32, mean, rstd, w, w32, y, ldy, out, dw, db, T, C, ws, size, None)


SHARED = [
    (dict(x32=2), INVALID), (dict(w32=2), INVALID), (dict(out=2), INVALID), (dict(T=-1), INVALID), (dict(C=0), INVALID), (dict(x=None), INVALID),
    (dict(y=None), INVALID), (dict(mean=None), INVALID), (dict(rstd=None), INVALID), (dict(ldx=32), INVALID), (dict(ldy=32), INVALID),
    (dict(C=60), UNSUPPORTED), (dict(C=16392), UNSUPPORTED), (dict(T=2 ** 31), UNSUPPORTED), (dict(x=A + 8), ALIGNMENT), (dict(y=A + 8), ALIGNMENT),
    (dict(w=A + 4), ALIGNMENT), (dict(mean=A + 2), ALIGNMENT), (dict(rstd=A + 1), ALIGNMENT), (dict(ldx=68), ALIGNMENT), (dict(ldy=68), ALIGNMENT),
]


@pytest.mark.parametrize("kw,want", SHARED + [(dict(b=A + 8), ALIGNMENT), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID)])
def test_layer_norm_fwd_refusals(L, kw, want):
    assert norm_fwd(L, **kw) == want


@pytest.mark.parametrize("kw,want", SHARED + [(dict(g=None), INVALID), (dict(g=A + 8), ALIGNMENT), (dict(ldg=8), INVALID), (dict(g32=-1), INVALID),
                                              (dict(dw=None), INVALID), (dict(db=None), INVALID), (dict(dw=A + 2), ALIGNMENT)])
def test_layer_norm_bwd_refusals(L, kw, want):
    assert norm_bwd(L, **kw) == want


def test_layer_norm_workspace(L):
    n = ctypes.c_size_t(0)
    assert L.dp_layer_norm_workspace_size(16384, 4096, 152, ctypes.byref(n)) == OK and 0 < n.value <= 64 << 20
    assert L.dp_layer_norm_workspace_size(1, 64, 152, ctypes.byref(n)) == OK and 0 < n.value <= 4096
    assert L.dp_layer_norm_workspace_size(0, 64, 152, ctypes.byref(n)) == OK and n.value == 0
    assert L.dp_layer_norm_workspace_size(4, 60, 152, ctypes.byref(n)) == UNSUPPORTED
    assert L.dp_layer_norm_workspace_size(4, 64, 152, None) == INVALID


def route(L, l=A, ld=0, gates=A, choice=A, T=4, E=16, k=2, norm=1):
    return L.dp_route_topk(l, ld, gates, choice, T, E, k, norm, None)


def route_bwd(L, dg=A, l=A, ld=0, gates=A, choice=A, d=A, ldd=0, T=4, E=16, k=2, norm=0):
    return L.dp_route_topk_bwd(dg, l, ld, gates, choice, d, ldd, T, E, k, norm, None)


ROUTE = [(dict(l=None), INVALID), (dict(gates=None), INVALID), (dict(choice=None), INVALID), (dict(T=-1), INVALID), (dict(E=0), INVALID),
         (dict(k=0), INVALID), (dict(k=17), INVALID), (dict(norm=2), INVALID), (dict(ld=15), INVALID), (dict(E=1025), UNSUPPORTED),
         (dict(E=64, k=33), UNSUPPORTED), (dict(T=2 ** 31), UNSUPPORTED), (dict(l=A + 2), ALIGNMENT), (dict(gates=A + 2), ALIGNMENT),
         (dict(choice=A + 1), ALIGNMENT)]


@pytest.mark.parametrize("kw,want", ROUTE)
def test_route_refusals(L, kw, want):
    assert route(L, **kw) == want


@pytest.mark.parametrize("kw,want", ROUTE + [(dict(dg=None), INVALID), (dict(d=None), INVALID), (dict(d=None, norm=1), INVALID), (dict(ldd=8), INVALID),
                                             (dict(d=A + 2), ALIGNMENT), (dict(dg=A + 3), ALIGNMENT)])
def test_route_bwd_refusals(L, kw, want):
    assert route_bwd(L, **kw) == want


def sort(L, choice=A, bits=32, pairs=64, E=8, offsets=A, row_of=A, order=A, ws=A, size=1 << 30):
    return L.dp_expert_sort(choice, bits, pairs, E, offsets, row_of, order, ws, size, None)


@pytest.mark.parametrize("kw,want", [
    (dict(bits=16), INVALID), (dict(pairs=-1), INVALID), (dict(E=0), INVALID), (dict(E=1025), UNSUPPORTED), (dict(pairs=2 ** 31), UNSUPPORTED),
    (dict(choice=None), INVALID), (dict(offsets=None), INVALID), (dict(row_of=None), INVALID), (dict(order=None), INVALID),
    (dict(choice=A + 2), ALIGNMENT), (dict(choice=A + 4, bits=64), ALIGNMENT), (dict(order=A + 1), ALIGNMENT),
    (dict(pairs=1 << 22, ws=None), WORKSPACE), (dict(pairs=1 << 22, size=64), WORKSPACE),
])
def test_sort_refusals(L, kw, want):
    assert sort(L, **kw) == want


def test_sort_workspace(L):
    n = ctypes.c_size_t(1)
    assert L.dp_expert_sort_workspace_size(64, 8, ctypes.byref(n)) == OK and n.value == 0
    assert L.dp_expert_sort_workspace_size(1 << 22, 1024, ctypes.byref(n)) == OK and 0 < n.value <= 4 << 20
    assert L.dp_expert_sort_workspace_size(-1, 8, ctypes.byref(n)) == INVALID
    assert L.dp_expert_sort_workspace_size(4, 2000, ctypes.byref(n)) == UNSUPPORTED


def gather(L, x=A, ldx=0, f32=0, row_of=A, out=A, ldo=0, T=4, k=2, C=64):
    return L.dp_expert_gather(x, ldx, f32, row_of, out, ldo, T, k, C, None)


def combine(L, x=A, ldx=0, f32=0, row_of=A, gates=A, add=None, ld_add=0, out=A, ldo=0, code=0, T=4, k=2, C=64):
    return L.dp_expert_combine(x, ldx, f32, row_of, gates, add, ld_add, out, ldo, code, T, k, C, None)


def combine_bwd(L, d=A, ldd=0, d32=0, x=A, ldx=0, f32=0, row_of=A, gates=A, out=A, ldo=0, code=0, dg=A, T=4, k=2, C=64):
    return L.dp_expert_combine_bwd(d, ldd, d32, x, ldx, f32, row_of, gates, out, ldo, code, dg, T, k, C, None)


ROWS = [(dict(x=None), INVALID), (dict(out=None), INVALID), (dict(row_of=None), INVALID), (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(C=0), INVALID),
        (dict(f32=2), INVALID), (dict(ldx=32), INVALID), (dict(ldo=32), INVALID), (dict(C=60), UNSUPPORTED), (dict(T=1 << 30, k=4), UNSUPPORTED),
        (dict(x=A + 8), ALIGNMENT), (dict(out=A + 8), ALIGNMENT), (dict(row_of=A + 2), ALIGNMENT), (dict(ldx=68), ALIGNMENT)]


@pytest.mark.parametrize("kw,want", ROWS)
def test_gather_refusals(L, kw, want):
    assert gather(L, **kw) == want


@pytest.mark.parametrize("kw,want", ROWS + [(dict(code=2), INVALID), (dict(gates=A + 2), ALIGNMENT), (dict(add=A + 8), ALIGNMENT),
                                            (dict(add=A, ld_add=8), INVALID)])
def test_combine_refusals(L, kw, want):
    assert combine(L, **kw) == want


@pytest.mark.parametrize("kw,want", ROWS + [(dict(code=2), INVALID), (dict(d=None), INVALID), (dict(d32=2), INVALID), (dict(gates=None), INVALID),
                                            (dict(dg=None), INVALID), (dict(dg=A + 2), ALIGNMENT), (dict(ldd=8), INVALID)])
def test_combine_bwd_refusals(L, kw, want):
    assert combine_bwd(L, **kw) == want


@pytest.mark.parametrize("C", [0x7FFFF808, 0x7FFFFF00])
def test_columns_that_a_counter_of_32_bits_would_pass(L, C):
    """Threads go over a row up to 2048 columns at a time: from a last column C - 8 on the next must still fit."""
    assert gather(L, C=C, T=1) == combine(L, C=C, T=1) == combine_bwd(L, C=C, T=1) == UNSUPPORTED


def product(L, x=A, ldx=0, q=A, s=A, s32=0, z=None, group=32, offs=None, bits=32, y=A, ldy=0, E=1, T=4, N=64, K=128, out=0, grouped=False):
    if grouped:
        return L.dp_gemm_fwd_int4_grouped(x, ldx, q, s, s32, z, group, offs, bits, y, ldy, E, T, N, K, out, None)
    return L.dp_gemm_fwd_int4(x, ldx, q, s, s32, z, group, y, ldy, T, N, K, out, None)


PRODUCT = [(dict(x=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID), (dict(y=None), INVALID), (dict(s32=2), INVALID), (dict(out=2), INVALID),
           (dict(T=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(ldx=64), INVALID), (dict(ldy=32), INVALID), (dict(group=16), UNSUPPORTED),
           (dict(K=144), UNSUPPORTED), (dict(N=60), UNSUPPORTED), (dict(K=32768 + 32), UNSUPPORTED), (dict(T=2 ** 31), UNSUPPORTED), (dict(x=A + 8), ALIGNMENT),
           (dict(q=A + 8), ALIGNMENT), (dict(s=A + 1), ALIGNMENT), (dict(s=A + 2, s32=1), ALIGNMENT), (dict(y=A + 8), ALIGNMENT), (dict(ldx=132), ALIGNMENT)]


@pytest.mark.parametrize("kw,want", PRODUCT)
@pytest.mark.parametrize("grouped", [False, True])
def test_int4_product_refusals(L, kw, want, grouped):
    assert product(L, grouped=grouped, offs=A, **kw) == want


def test_int4_grouped_refusals(L):
    assert product(L, grouped=True) == INVALID and product(L, grouped=True, offs=A, bits=16) == INVALID
    assert product(L, grouped=True, offs=A, E=-1) == INVALID and product(L, grouped=True, offs=A, E=1025) == UNSUPPORTED
    assert product(L, grouped=True, offs=A + 2) == ALIGNMENT and product(L, grouped=True, offs=A + 4, bits=64) == ALIGNMENT


@pytest.mark.parametrize("E,N", [(1 << 33, 1 << 30), (1 << 40, 1 << 30), (1 << 62, 8), (4, 1 << 61), ((1 << 63) - 1, 64)])
def test_int4_rows_that_leave_64_bits(L, E, N):
    """Experts times rows are counted after each of them has been held to its range."""
    assert product(L, grouped=True, offs=A, E=E, N=N) == UNSUPPORTED
    assert product(L, grouped=True, offs=A, E=E, N=N, q=None) == UNSUPPORTED  # (which asks whether there are rows)


def test_int4_code_refusals(L):
    def quantize(w=A, ldw=0, w32=0, rows=4, K=128, group=32, q=A, s=A, s32=0, z=None):
        return L.dp_int4_quantize(w, ldw, w32, rows, K, group, q, s, s32, z, None)

    def expand(q=A, s=A, s32=0, z=None, rows=4, K=128, group=32, w=A, ldw=0, out=0):
        return L.dp_int4_dequantize(q, s, s32, z, rows, K, group, w, ldw, out, None)
    for f in (quantize, expand):
        assert f(w=None) == INVALID and f(q=None) == INVALID and f(s=None) == INVALID and f(rows=-1) == INVALID and f(K=0) == INVALID
        assert f(s32=2) == INVALID and f(ldw=64) == INVALID and f(group=256) == UNSUPPORTED and f(K=100) == UNSUPPORTED
        assert f(q=A + 4) == ALIGNMENT and f(s=A + 1) == ALIGNMENT and f(w=A + 8) == ALIGNMENT and f(ldw=130) == ALIGNMENT
    assert quantize(w32=2) == INVALID and expand(out=2) == INVALID


def test_python_refusals():
    x, row_of = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32)
    l, q = torch.zeros(4, 8), torch.zeros(8, 32, dtype=torch.uint8)
    s = torch.zeros(8, 2, dtype=torch.bfloat16)
    for f in (lambda: dp.layer_norm_fwd(x), lambda: dp.layer_norm_bwd(x, x, l[:, 0], l[:, 0]), lambda: dp.route_topk(l, 2),
              lambda: dp.route_topk_bwd(l, l, l, row_of), lambda: dp.expert_sort(row_of, 8), lambda: dp.expert_gather(x, row_of),
              lambda: dp.expert_combine(x, row_of), lambda: dp.expert_combine_bwd(x, x, row_of, l), lambda: dp.int4_quantize(x),
              lambda: dp.int4_dequantize(q, s), lambda: dp.dp_gemm_fwd_int4(x, q, s), lambda: dp.dp_gemm_fwd_int4_grouped(x, q, s, row_of)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            f()
