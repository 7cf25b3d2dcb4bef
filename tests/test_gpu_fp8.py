"""8-bit quantisation and products against the definitions.

Quantisation: scales within one rounding of the 64-bit value; q s within half a code of x
(E4M3: 2^-4 |x|, E5M2: 2^-3 |x|, and half the smallest code below the normal range), and the
very codes that the same FP32 operations give in plain torch.
Products: a block's sum of 128 products takes four tensor-core steps, each within a few
units of 2^-23 of the sum of magnitudes S = sum |a||b|; the scaled block sums are added in
FP32, two roundings each.  So |got - ref| <= (24 + 2 blocks) 2^-23 S (FP32 out), and
2^-8 |ref| more for BF16.
"""
import pytest
import torch

import fp32_dense_projection_gb300 as dp
from gpu_common import DEV

pytestmark = pytest.mark.gpu

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
TOP = {E4: 448.0, E5: 57344.0}
HALF = {E4: 2.0 ** -4, E5: 2.0 ** -3}          # half a code, relative, in the normal range
LEAST = {E4: 2.0 ** -10, E5: 2.0 ** -17}       # half the smallest code


def blocks(n):
    return -(-n // 128)


def spread(s, scaling, shape):
    if scaling in ("row", "block"):
        s = s.repeat_interleave(128, 1)[:, :shape[1]]
    if scaling in ("col", "block"):
        s = s.repeat_interleave(128, 0)[:shape[0]]
    return s


def plain(x, scaling, dtype):
    """The same FP32 operations in torch (quotients of tensors: torch turns those with a
    Python number into products with a reciprocal)."""
    T, C = x.shape
    rows, cols = (128 if scaling in ("col", "block") else 1), (128 if scaling in ("row", "block") else 1)
    a = torch.nn.functional.pad(x.float().abs(), (0, -C % cols, 0, -T % rows))
    a = a.view(-(-T // rows), rows, -(-C // cols), cols).amax((1, 3)).clamp_min(1e-30)
    top = torch.full_like(a, TOP[dtype])
    f = (top / a).repeat_interleave(rows, 0)[:T].repeat_interleave(cols, 1)[:, :C]
    return (x.float() * f).clamp(-TOP[dtype], TOP[dtype]).to(dtype), a / top


def values(T, C, seed, kind="normal", dtype=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((T, C), device=DEV, generator=g)
    if kind == "wide":  # magnitudes over many octaves, zeros among them
        x = x * torch.exp2(torch.randint(-40, 40, (T, C), device=DEV, generator=g).float())
        x[torch.rand((T, C), device=DEV, generator=g) < 0.1] = 0
    return x.to(dtype)


@pytest.mark.parametrize("T,C", [(1, 16), (3, 128), (127, 144), (128, 256), (129, 16), (500, 1040), (260, 2064)])
@pytest.mark.parametrize("scaling", ["row", "col", "block", "both"])
@pytest.mark.parametrize("dtype", [E4, E5])
@pytest.mark.parametrize("src", [torch.bfloat16, torch.float32])
def test_quantize(T, C, scaling, dtype, src):
    for kind in ("normal", "wide"):
        x = values(T, C, T + C, kind, src)
        got = dp.fp8_quantize(x, scaling, dtype)
        pairs = [("row", got[:2]), ("col", got[2:])] if scaling == "both" else [(scaling, got)]
        for how, (q, s) in pairs:
            want_q, want_s = plain(x, how, dtype)
            assert q.dtype == dtype and q.shape == x.shape and s.shape == want_s.shape
            assert torch.equal(s, want_s)
            assert torch.equal(q.view(torch.uint8), want_q.view(torch.uint8))
            wide = spread(s.double(), how, x.shape)
            off = (q.double() * wide - x.double()).abs()
            assert bool((off <= HALF[dtype] * (1 + 1e-5) * x.double().abs() + LEAST[dtype] * (1 + 1e-5) * wide).all())


@pytest.mark.parametrize("scaling", ["row", "col", "block", "both"])
def test_quantize_strided_source(scaling):
    x = values(70, 272, 1)
    wide = torch.full((70, 320), float("inf"), device=DEV).bfloat16()
    wide[:, 16:288] = x
    for a, b in zip(dp.fp8_quantize(wide[:, 16:288], scaling), dp.fp8_quantize(x, scaling)):
        assert torch.equal(a.float(), b.float())


def test_quantize_zeros_and_non_finite_blocks():
    x = values(256, 256, 2)
    x[:128, :128] = 0
    x[128, 5], x[200, 130] = float("nan"), float("inf")
    for how in ("row", "col", "block"):
        q, s = dp.fp8_quantize(x, how)
        d = q.double() * spread(s.double(), how, x.shape)
        bad = {"row": ((128, slice(0, 128)), (200, slice(128, 256))),
               "col": ((slice(128, 256), 5), (slice(128, 256), 130)),
               "block": ((slice(128, 256), slice(0, 128)), (slice(128, 256), slice(128, 256)))}[how]
        fine = torch.ones_like(d, dtype=torch.bool)
        for b in bad:  # the whole block says so
            assert not bool(torch.isfinite(d[b]).any())
            fine[b] = False
        assert bool(torch.isfinite(d[fine]).all()) and bool((d[:128, :128] == 0).all())


def test_quantize_beyond_32_bit_offsets():
    T, C = 131_201, 16_384
    x = torch.zeros((T, C), dtype=torch.bfloat16, device=DEV)
    x[-200:] = values(200, C, 3)
    for how in ("row", "col"):
        q, s = dp.fp8_quantize(x, how)
        lo = T - T % 128 - 128
        want_q, want_s = plain(x[lo:], how, E4)
        assert torch.equal(q[lo:].view(torch.uint8), want_q.view(torch.uint8))
        assert torch.equal(s[lo:] if how == "row" else s[lo // 128:], want_s)


def operands(op, T, N, K, seed, fa=E4, fb=E4, ints=False):
    """(quantised pair, dequantised in 64 bits) of both operands."""
    shapes = {"fwd": ((T, K), (N, K)), "dgrad": ((T, N), (N, K)), "wgrad": ((T, N), (T, K))}[op]
    hows = {"fwd": ("row", "block"), "dgrad": ("row", "block"), "wgrad": ("col", "col")}[op]
    out = []
    for i, (shape, how, f) in enumerate(zip(shapes, hows, (fa, fb))):
        if ints:  # integer codes and power-of-two scales: every sum is exact in FP32
            g = torch.Generator(device=DEV).manual_seed(seed + i)
            q = torch.randint(-3, 4, shape, device=DEV, generator=g).float().to(f)
            s_shape = {"row": (shape[0], blocks(shape[1])), "col": (blocks(shape[0]), shape[1]),
                       "block": (blocks(shape[0]), blocks(shape[1]))}[how]
            s = torch.exp2(torch.randint(-2, 3, s_shape, device=DEV, generator=g).float())
        else:
            q, s = dp.fp8_quantize(values(*shape, seed + i), how, f)
        out.append(((q, s), q.double() * spread(s.double(), how, shape)))
    return out


def product(op, a, b):
    return a @ b.T if op == "fwd" else a @ b if op == "dgrad" else a.T @ b


def call(op, a, b, **kw):
    return {"fwd": dp.dp_gemm_fwd_fp8, "dgrad": dp.dp_gemm_dgrad_fp8, "wgrad": dp.dp_gemm_wgrad_fp8}[op](*a, *b, **kw)


OPS = ("fwd", "dgrad", "wgrad")
SHAPES = [(1, 16, 16), (1, 512, 1040), (2, 144, 128), (17, 272, 400), (127, 128, 256), (129, 1040, 144), (300, 528, 2064),
          (1000, 272, 528), (64, 12288, 144), (5000, 256, 384)]


@pytest.mark.parametrize("T,N,K", SHAPES)
@pytest.mark.parametrize("op", OPS)
def test_exact_products(op, T, N, K):
    (a, da), (b, db) = operands(op, T, N, K, T + N, ints=True)
    ref = product(op, da, db)
    assert torch.equal(call(op, a, b, out_dtype=torch.float32), ref.float())
    assert torch.equal(call(op, a, b), ref.to(torch.bfloat16))
    assert dp.device_error() == 0


@pytest.mark.parametrize("T,N,K", [(2500, 2064, 2064), (2305, 2320, 2576), (4096, 2048, 1664)])
@pytest.mark.parametrize("op", OPS)
def test_exact_products_on_many_tiles(op, T, N, K):
    """Sizes whose tiles fill the device: two SMs share a tile of 256 x 256, ragged at its edges."""
    (a, da), (b, db) = operands(op, T, N, K, T + N, ints=True)
    ref = product(op, da, db)
    assert torch.equal(call(op, a, b, out_dtype=torch.float32), ref.float())
    assert torch.equal(call(op, a, b), ref.to(torch.bfloat16))
    assert dp.device_error() == 0


@pytest.mark.parametrize("T,N,K", [(16, 4096, 4096), (130, 272, 4112), (3000, 144, 272), (128, 128, 16384), (7, 1040, 656)])
@pytest.mark.parametrize("op", OPS)
def test_exact_products_of_few_tiles(op, T, N, K):
    """Sizes whose tiles do not fill the device: clusters of SMs share a tile's contraction, the
    shares uneven, rows and columns ragged."""
    (a, da), (b, db) = operands(op, T, N, K, T + K, ints=True)
    ref = product(op, da, db)
    assert torch.equal(call(op, a, b, out_dtype=torch.float32), ref.float())
    assert torch.equal(call(op, a, b), ref.to(torch.bfloat16))
    assert dp.device_error() == 0


@pytest.mark.parametrize("fa,fb", [(E4, E4), (E5, E4), (E4, E5), (E5, E5)])
@pytest.mark.parametrize("op", OPS)
def test_real_products(op, fa, fb):
    for T, N, K in ((1, 272, 528), (333, 1040, 656), (2000, 256, 4112), (2600, 2064, 2192)):
        (a, da), (b, db) = operands(op, T, N, K, T, fa, fb)
        ref, mag = product(op, da, db), product(op, da.abs(), db.abs())
        tol = (24 + 2 * blocks({"fwd": K, "dgrad": N, "wgrad": T}[op])) * 2.0 ** -23 * mag
        assert bool(((call(op, a, b, out_dtype=torch.float32).double() - ref).abs() <= tol).all())
        assert bool(((call(op, a, b).double() - ref).abs() <= tol + 2.0 ** -8 * ref.abs()).all())


@pytest.mark.parametrize("op", OPS)
def test_strides(op):
    """Operands and outputs inside wider buffers; scales transposed, strided or broadcast."""
    T, N, K = 200, 272, 400
    (a, da), (b, db) = operands(op, T, N, K, 5, ints=True)
    ref = product(op, da, db).float()

    def inside(q):
        big = torch.full((q.shape[0], q.shape[1] + 48), 448.0, device=DEV).to(E4)
        big[:, 16:16 + q.shape[1]] = q
        return big[:, 16:16 + q.shape[1]]

    def every_other(s):
        big = torch.full((2 * s.shape[0], 3 * s.shape[1]), float("nan"), device=DEV)
        big[::2, ::3] = s
        return big[::2, ::3]
    for f in (lambda s: s.t().contiguous().t(), lambda s: s.contiguous(), every_other):
        big = torch.full((ref.shape[0], ref.shape[1] + 32), 5.0, device=DEV)
        out = big[:, 16:16 + ref.shape[1]]
        assert call(op, (inside(a[0]), f(a[1])), (inside(b[0]), f(b[1])), out=out) is out
        assert torch.equal(out, ref)
        assert bool((big[:, :16] == 5).all()) and bool((big[:, 16 + ref.shape[1]:] == 5).all())
    one = torch.ones(1, 1, device=DEV)
    got = call(op, (a[0], one.expand(a[1].shape)), (b[0], one.expand(b[1].shape)), out_dtype=torch.float32)
    assert torch.equal(got, product(op, a[0].double(), b[0].double()).float())


@pytest.mark.parametrize("op", OPS)
def test_non_finite_rows_stay_in_their_rows(op):
    (a, da), (b, _) = operands(op, 150, 144, 272, 6, ints=True)
    q = a[0].clone()
    q[70, 3] = float("nan")
    clean, got = call(op, a, b, out_dtype=torch.float32), call(op, (q, a[1]), b, out_dtype=torch.float32)
    hit = 3 if op == "wgrad" else 70
    keep = torch.arange(got.shape[0], device=DEV) != hit
    assert torch.equal(got[keep], clean[keep]) and bool(torch.isnan(got[hit]).all())


@pytest.mark.parametrize("op", OPS)
def test_no_rows_streams_graph_and_repeats(op):
    (a, _), (b, _) = operands(op, 0, 144, 272, 7, ints=True)
    out = call(op, a, b, out_dtype=torch.float32)
    assert out.numel() == 0 or bool((out == 0).all())
    (a, _), (b, _) = operands(op, 700, 528, 656, 8)
    first = call(op, a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = call(op, a, b, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out = call(op, a, b)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(other, first) and torch.equal(out, first) and torch.equal(call(op, a, b), first)


def test_gradients_against_differences():
    """L = sum(Y G) with Y = X W^T is linear: integer differences are exact."""
    T, N, K = 140, 144, 272
    g = torch.Generator(device=DEV).manual_seed(1)

    def ints(*shape):
        return torch.randint(-2, 3, shape, device=DEV, generator=g).float()
    x, w, grad = ints(T, K), ints(N, K), ints(T, N)
    ux, uw = ints(T, K).clamp(-1, 1), ints(N, K).clamp(-1, 1)

    def pair(v, shape):
        return v.to(E4), torch.ones(shape, device=DEV)

    def loss(x, w):
        y = dp.dp_gemm_fwd_fp8(*pair(x, (T, blocks(K))), *pair(w, (blocks(N), blocks(K))), out_dtype=torch.float32)
        return float((y.double() * grad.double()).sum())
    dX = dp.dp_gemm_dgrad_fp8(*pair(grad, (T, blocks(N))), *pair(w, (blocks(N), blocks(K))), out_dtype=torch.float32)
    dW = dp.dp_gemm_wgrad_fp8(*pair(grad, (blocks(T), N)), *pair(x, (blocks(T), K)), out_dtype=torch.float32)
    assert (loss(x + ux, w) - loss(x - ux, w)) / 2 == float((dX.double() * ux.double()).sum())
    assert (loss(x, w + uw) - loss(x, w - uw)) / 2 == float((dW.double() * uw.double()).sum())
