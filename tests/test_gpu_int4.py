"""Weights in 4 bits with group scales: quantisation, expansion and products, against plain forms.

Quantisation follows its FP32 formulas bit for bit.  Products on small integers with scales that are powers of two are
exact in FP32, so outputs must be equal.  On real operands, S = sum |x||w| in 64 bits: each tensor-core step (16
products and the running sum) loses at most a few units of 2^-23 of the group's magnitudes, a group has
group / 16 steps, its sum meets the scale (one FP32 step), and the sums of groups, warps and CTAs are added one after
the other:  |got - ref| <= (4 (group / 16 + 2) + K / group + 16) 2^-23 S;  BF16 outputs add 2^-8 |ref|.
"""
import pytest
import torch

import fp32_dense_projection_gb300 as dp
from gpu_common import DEV

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(shape, seed, dtype=BF16, scale=1.0):
    return (torch.randn(shape, device=DEV, generator=gen(seed)) * scale).to(dtype)


def codes_of(q):
    return torch.stack((q & 15, q >> 4), -1).flatten(-2)


def expand(q, s, z, group):
    """The weights that are meant, in 64 bits."""
    c = codes_of(q).double().unflatten(-1, (-1, group))
    zero = 8.0 if z is None else z.double()[..., None]
    return ((c - zero) * s.double()[..., None]).flatten(-2)


def plain_quantize(W, group, zeros, kind):
    g = W.float().unflatten(-1, (-1, group))
    if zeros:
        lo, hi = g.amin(-1).clamp_max(0.0), g.amax(-1).clamp_min(0.0)
        s = ((hi - lo) / torch.full_like(hi, 15.0)).clamp_min(1e-30).to(kind)
        z = (-lo / s.float()).round().clamp(0, 15)
    else:
        s = (g.abs().amax(-1) / torch.full_like(g[..., 0], 7.0)).clamp_min(1e-30).to(kind)
        z = torch.full_like(s, 8.0, dtype=F32)
    q = ((g / s.float()[..., None]).round() + z[..., None]).clamp(0, 15).to(torch.uint8).flatten(-2)
    return q[..., 0::2] | (q[..., 1::2] << 4), s, z.to(torch.uint8) if zeros else None


@pytest.mark.parametrize("shape", [(1, 32), (8, 128), (3, 96), (40, 4096), (1000, 640), (5, 24, 256), (4096, 1024)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("wt,st", [(BF16, BF16), (F32, F32), (F32, BF16), (BF16, F32)])
def test_quantize_and_dequantize(shape, group, zeros, wt, st):
    if shape[-1] % group:
        with pytest.raises(ValueError, match="divide K"):
            dp.int4_quantize(normal(shape, 1), group)
        return
    W = normal(shape, sum(shape), wt, 0.05)
    W.view(-1)[::7] = 0
    W.view(-1, group)[0] = 0                 # a group of zeros
    W.view(-1, group)[-1] = W.view(-1, group)[-1].abs() + 1  # a group of one sign
    q, s, z = dp.int4_quantize(W, group, zeros=zeros, scale_dtype=st)
    want = plain_quantize(W, group, zeros, st)
    assert torch.equal(q, want[0]) and torch.equal(s, want[1]) and (z is None if not zeros else torch.equal(z, want[2]))
    for out in (BF16, F32):
        got = dp.int4_dequantize(q, s, zeros=z, out_dtype=out)
        ref = expand(q, s, z, group)
        assert got.dtype is out and got.shape == W.shape
        if st is BF16 and out is F32:  # (4 or 5 bits times 8)
            assert torch.equal(got.double(), ref)
        else:
            assert bool(((got.double() - ref).abs() <= (torch.finfo(out).eps / 2 + 2.0 ** -24) * ref.abs()).all())
    # a code is off by half a step at most; where a scale was rounded down to BF16 the ends of the range by 7 (15) such roundings
    step = s.float().repeat_interleave(group, -1)
    assert bool(((dp.int4_dequantize(q, s, zeros=z, out_dtype=F32) - W.float()).abs() <= step * (0.5 + 2e-6 + (15 * 2.0 ** -8 if st is BF16 else 0))).all())


def test_quantize_padded_rows_and_bad_values():
    W = normal((50, 256 + 64), 1)[:, :256]
    got, want = dp.int4_quantize(W, 64), dp.int4_quantize(W.contiguous(), 64)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    buf = torch.full((50, 256 + 8), 7.0, device=DEV, dtype=BF16)
    dp.int4_dequantize(*want, out=buf[:, :256])
    assert torch.equal(buf[:, :256], dp.int4_dequantize(*want)) and bool((buf[:, 256:] == 7).all())
    bad = W.contiguous().clone()
    bad[3, 70], bad[9, 10] = float("nan"), float("inf")
    for zeros in (False, True):
        q, s, z = dp.int4_quantize(bad, 64, zeros=zeros)
        clean = dp.int4_quantize(W, 64, zeros=zeros)
        keep = torch.ones(50, 4, dtype=torch.bool, device=DEV)
        keep[3, 1] = keep[9, 0] = False
        assert s[3, 1].isnan() and s[9, 0].isinf() and torch.equal(s[keep], clean[1][keep])
        rows = keep.repeat_interleave(32, 1)
        assert torch.equal(q[rows], clean[0][rows])


@pytest.mark.parametrize("rows", ["1", "3", "16", "50"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("wt,st", [(BF16, BF16), (F32, F32), (F32, BF16), (BF16, F32)])
def test_quantize_and_dequantize_in_parts(rows, group, zeros, wt, st, monkeypatch):
    """More rows than a launch counts (here: a few): each part's pointers, of padded rows too, follow the last one's."""
    K, pad = 640 if group < 128 else 384, 24
    W = normal((50, K + pad), 1, wt, 0.05)[:, :K]
    want = dp.int4_quantize(W, group, zeros=zeros, scale_dtype=st)
    wide = [dp.int4_dequantize(*want, out_dtype=out) for out in (BF16, F32)]
    monkeypatch.setenv("DP_FORCE_INT4_ROWS", rows)
    got = dp.int4_quantize(W, group, zeros=zeros, scale_dtype=st)
    assert all(torch.equal(a, b) if zeros or i < 2 else a is None for i, (a, b) in enumerate(zip(got, want)))
    assert torch.equal(dp.int4_quantize(W.contiguous().view(5, 10, K), group, zeros=zeros, scale_dtype=st)[0], want[0].view(5, 10, K // 2))
    for w in wide:
        buf = torch.full((50, K + pad), 7.0, device=DEV, dtype=w.dtype)
        dp.int4_dequantize(*want, out=buf[:, :K])
        assert torch.equal(buf[:, :K], w) and bool((buf[:, K:] == 7).all())
        assert torch.equal(dp.int4_dequantize(*want, out_dtype=w.dtype), w)


def problem(E, N, K, group, zeros, st, seed, exact):
    """Codes, scales and zero points of E experts (0: none)."""
    front = (E, N) if E else (N,)
    q = torch.randint(0, 256, (*front, K // 2), device=DEV, generator=gen(seed), dtype=torch.uint8)
    if exact:
        s = (2.0 ** torch.randint(-2, 2, (*front, K // group), device=DEV, generator=gen(seed + 1)).float()).to(st)
    else:
        s = ((torch.rand((*front, K // group), device=DEV, generator=gen(seed + 1)) + 0.2) / K ** 0.5).to(st)
    z = torch.randint(0, 16, s.shape, device=DEV, generator=gen(seed + 2), dtype=torch.uint8) if zeros else None
    return q, s, z


def rows(T, K, seed, exact):
    if exact:
        return torch.randint(-2, 3, (T, K), device=DEV, generator=gen(seed)).bfloat16()
    return normal((T, K), seed)


def check(got, ref, mag, group, K, exact):
    out = got.dtype
    if exact:
        assert torch.equal(got, ref.float().to(out))
        return
    tol = (4 * (group / 16 + 2) + K / group + 16) * 2.0 ** -23 * mag
    tol = tol + (2.0 ** -8 * (ref.abs() + tol) if out is BF16 else 0)
    off = (got.double() - ref).abs()
    assert got.isfinite().all() and bool((off <= tol).all()), float((off / tol.clamp_min(1e-300)).max())


SIZES = [(1, 8, 128), (1, 16, 32), (2, 24, 96), (8, 64, 256), (1, 4096, 4096), (9, 40, 160), (16, 136, 1024), (17, 1000, 640), (31, 264, 2176),
         (33, 128, 4096), (64, 72, 1056), (65, 512, 2048), (200, 48, 320), (3, 16, 32768), (40, 24, 20480), (1, 12288, 1024), (5, 8, 8192)]


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_products(T, N, K, group, zeros):
    if K % group:
        return
    for exact in (True, False):
        for st in (BF16, F32):
            q, s, z = problem(0, N, K, group, zeros, st, T + N, exact)
            X = rows(T, K, 3, exact)
            W = expand(q, s, z, group)
            ref, mag = X.double() @ W.T, X.double().abs() @ W.abs().T
            for out in (BF16, F32):
                check(dp.dp_gemm_fwd_int4(X, q, s, zeros=z, out_dtype=out), ref, mag, group, K, exact)
    assert dp.device_error() == 0


GROUPS = {
    "one_row": (0, [1], 0),
    "one_row_of_many": (0, [0, 0, 1, 0], 0),
    "decode": (0, [i % 3 for i in range(40)], 0),
    "ragged": (3, [5, 0, 9, 17, 1, 33, 0, 8], 6),
    "all_empty": (10, [0, 0, 0], 3),
    "one_expert": (0, [70], 0),
    "many_rows": (0, [100, 1, 60], 5),
    "most_experts": (0, [(i * 7) % 2 for i in range(1024)], 1),
}


@pytest.mark.parametrize("groups", sorted(GROUPS))
@pytest.mark.parametrize("group", [32, 64, 128])
def test_grouped(groups, group):
    front, counts, back = GROUPS[groups]
    E, T = len(counts), front + sum(counts) + back
    edges = [front]
    for n in counts:
        edges.append(edges[-1] + n)
    for N, K in ((24, 128), (136, 1152), (64, 4096)) if E < 100 else ((16, 256),):
        for exact, zeros, st, bits in ((True, True, BF16, torch.int32), (False, False, F32, torch.int64)):
            q, s, z = problem(E, N, K, group, zeros, st, E + N, exact)
            X = rows(T, K, 3, exact)
            ref = torch.zeros(T, N, dtype=torch.float64, device=DEV)
            mag = torch.zeros_like(ref)
            for e in range(E):
                a, b = edges[e], edges[e + 1]
                if b > a:
                    W = expand(q[e], s[e], None if z is None else z[e], group)
                    ref[a:b], mag[a:b] = X[a:b].double() @ W.T, X[a:b].double().abs() @ W.abs().T
            offsets = torch.tensor(edges, dtype=bits, device=DEV)
            for out in (BF16, F32):
                buf = torch.full((T, N), 7.0, device=DEV, dtype=out)
                check(dp.dp_gemm_fwd_int4_grouped(X, q, s, offsets, zeros=z, out=buf), ref, mag, group, K, exact)
    assert dp.device_error() == 0


@pytest.mark.parametrize("teams", ["1", "4"])
@pytest.mark.parametrize("tokens", ["1", "3", "8", "16"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_forms(teams, tokens, group, monkeypatch):
    """Each cut of the work over warps and passes, where a CTA's range holds several experts, passes and odd tiles."""
    monkeypatch.setenv("DP_FORCE_INT4_TEAMS", teams)
    monkeypatch.setenv("DP_FORCE_INT4_TOKENS", tokens)
    counts = [3, 0, 21, 1, 16, 17, 0, 8, 9, 33, 2, 2]
    edges = [2]
    for n in counts:
        edges.append(edges[-1] + n)
    E, T = len(counts), edges[-1] + 5
    for N, K in ((1000, 384), (424, 4096), (2056, 2304), (264, 5120)):
        q, s, z = problem(E, N, K, group, True, BF16, N, True)
        X = rows(T, K, 3, True)
        ref = torch.zeros(T, N, dtype=torch.float64, device=DEV)
        for e in range(E):
            ref[edges[e]:edges[e + 1]] = X[edges[e]:edges[e + 1]].double() @ expand(q[e], s[e], z[e], group).T
        got = dp.dp_gemm_fwd_int4_grouped(X, q, s, torch.tensor(edges, dtype=torch.int32, device=DEV), zeros=z, out_dtype=F32)
        assert torch.equal(got, ref.float())
        got = dp.dp_gemm_fwd_int4(X[:37], q[0], s[0], zeros=z[0], out_dtype=F32)
        assert torch.equal(got, (X[:37].double() @ expand(q[0], s[0], z[0], group).T).float())
    assert dp.device_error() == 0


def test_bad_offsets_are_clamped_and_reported():
    E, T, N, K = 6, 40, 32, 128
    q, s, z = problem(E, N, K, 32, True, BF16, 1, True)
    X = rows(T, K, 2, True)
    dp.device_error()
    for given, meant in (([0, 5, 3, 20, 90, 10, 40], [0, 5, 5, 20, 40, 40, 40]), ([-4, 5, 9, 20, 30, 35, 39], [0, 5, 9, 20, 30, 35, 39]),
                         ([0, 0, 0, 0, 0, 0, 2 ** 31 - 1], [0, 0, 0, 0, 0, 0, 40])):
        got = dp.dp_gemm_fwd_int4_grouped(X, q, s, torch.tensor(given, dtype=torch.int32, device=DEV), zeros=z)
        assert dp.device_error() == 1
        assert torch.equal(got, dp.dp_gemm_fwd_int4_grouped(X, q, s, torch.tensor(meant, dtype=torch.int32, device=DEV), zeros=z))
        assert dp.device_error() == 0


def test_bad_rows_stay_by_themselves():
    """Infinities and NaN in a token reach its own outputs only: of the tokens beside it, of the next expert, and of
    padding rows."""
    E, T, N, K = 4, 30, 40, 256
    q, s, z = problem(E, N, K, 64, True, BF16, 1, False)
    offsets = torch.tensor([2, 9, 9, 20, 27], dtype=torch.int32, device=DEV)
    X = rows(T, K, 2, False)
    clean = dp.dp_gemm_fwd_int4_grouped(X, q, s, offsets, zeros=z)
    bad = X.clone()
    bad[0], bad[8], bad[20, 5], bad[29] = float("nan"), float("inf"), float("nan"), float("inf")
    got = dp.dp_gemm_fwd_int4_grouped(bad, q, s, offsets, zeros=z)
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[[8, 20]] = False
    assert torch.equal(got[keep], clean[keep]) and not got[8].isfinite().any() and bool(got[20].isnan().all())
    dense = dp.dp_gemm_fwd_int4(bad[7:12], q[0], s[0], zeros=z[0])
    want = dp.dp_gemm_fwd_int4(X[7:12], q[0], s[0], zeros=z[0])
    assert torch.equal(dense[[0, 2, 3, 4]], want[[0, 2, 3, 4]]) and not dense[1].isfinite().any()


def test_zero_points_are_four_bits():
    q, s, z = problem(0, 16, 128, 32, True, F32, 1, True)
    X = rows(3, 128, 2, True)
    assert torch.equal(dp.dp_gemm_fwd_int4(X, q, s, zeros=z | 0xF0), dp.dp_gemm_fwd_int4(X, q, s, zeros=z))
    assert torch.equal(dp.int4_dequantize(q, s, zeros=z | 0xF0), dp.int4_dequantize(q, s, zeros=z))


def test_padded_rows_and_repeats():
    T, N, K = 20, 72, 1024
    q, s, z = problem(0, N, K, 128, False, BF16, 1, False)
    X = normal((T, K + 8), 2)[:, :K]
    buf = torch.full((T, N + 24), 7.0, device=DEV)
    got = dp.dp_gemm_fwd_int4(X, q, s, out=buf[:, :N])
    for _ in range(5):
        assert torch.equal(got, dp.dp_gemm_fwd_int4(X.contiguous(), q, s, out_dtype=F32))
    assert bool((buf[:, N:] == 7).all())


def test_no_rows():
    q, s, _ = problem(0, 16, 128, 32, False, BF16, 1, False)
    assert dp.dp_gemm_fwd_int4(torch.empty(0, 128, device=DEV, dtype=BF16), q, s).shape == (0, 16)
    e = torch.empty(0, 16, 64, dtype=torch.uint8, device=DEV), torch.empty(0, 16, 4, dtype=BF16, device=DEV)
    got = dp.dp_gemm_fwd_int4_grouped(rows(5, 128, 1, False), *e, torch.zeros(1, dtype=torch.int32, device=DEV))
    assert got.shape == (5, 16) and not got.any()
    assert [t.shape for t in dp.int4_quantize(torch.empty(0, 128, device=DEV), 32)[:2]] == [(0, 64), (0, 4)]


@pytest.mark.parametrize("K,group", [(4096, 32), (1088, 32), (192, 32), (2176, 64), (320, 64), (4096, 128), (384, 128)])
@pytest.mark.parametrize("st", [BF16, F32])
def test_scales_anywhere(K, group, st):
    """Scales and zero points at any address of their type, and any number of groups, give the same bits."""
    N, E = 72, 3
    q, s, z = (torch.stack(t) for t in zip(*(problem(0, N, K, group, True, st, e, False) for e in range(E))))
    X = rows(9, K, 3, False)
    offsets = torch.tensor([0, 4, 4, 9], device=DEV, dtype=torch.int32)
    want = dp.dp_gemm_fwd_int4(X, q[0], s[0], zeros=z[0]), dp.dp_gemm_fwd_int4_grouped(X, q, s, offsets, zeros=z)
    for shift in (1, 2, 3, 8):
        buf, bufz = torch.zeros(s.numel() + shift, device=DEV, dtype=st), torch.zeros(z.numel() + shift, device=DEV, dtype=torch.uint8)
        s2, z2 = buf[shift:].view(s.shape), bufz[shift:].view(z.shape)
        s2.copy_(s)
        z2.copy_(z)
        for sc, ze in ((s2, z), (s, z2), (s2, z2)):
            assert torch.equal(dp.dp_gemm_fwd_int4(X, q[0], sc[0], zeros=ze[0]), want[0])
            assert torch.equal(dp.dp_gemm_fwd_int4_grouped(X, q, sc, offsets, zeros=ze), want[1])
    ref = X[:4].double() @ expand(q[0], s[0], z[0], group).T
    check(want[1][:4], ref, X[:4].double().abs() @ expand(q[0], s[0], z[0], group).abs().T, group, K, False)
    assert dp.device_error() == 0


def test_experts_past_32_bits():
    """Codes of 2^31 bytes and more: the last expert's are read."""
    E, N, K = 260, 4096, 4096
    q = torch.zeros(E, N, K // 2, dtype=torch.uint8, device=DEV)
    s = torch.ones(E, N, K // 128, dtype=BF16, device=DEV)
    one, sone, _ = problem(0, N, K, 128, False, BF16, 1, True)
    q[-1], s[-1] = one, sone
    X = rows(3, K, 2, True)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[-1] = 3
    got = dp.dp_gemm_fwd_int4_grouped(X, q, s, offsets, out_dtype=F32)
    assert torch.equal(got, dp.dp_gemm_fwd_int4(X, one, sone, out_dtype=F32))
    assert torch.equal(dp.int4_dequantize(q, s)[-1], dp.int4_dequantize(one, sone))


def test_streams_and_graphs():
    """On another stream, and captured: a replay follows new inputs and offsets; two graphs side by side."""
    E, T, N, K = 8, 24, 128, 1024
    q, s, z = problem(E, N, K, 64, True, BF16, 1, False)
    dense = problem(0, 256, K, 128, False, F32, 2, False)
    X = [rows(T, K, 3, False), rows(T, K, 3, False)]
    offsets = torch.tensor([0, 3, 3, 9, 10, 12, 20, 21, 24], dtype=torch.int32, device=DEV)

    def step(x):
        return dp.dp_gemm_fwd_int4_grouped(x, q, s, offsets, zeros=z), dp.dp_gemm_fwd_int4(x, *dense[:2])
    want = step(X[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dp.dp_gemm_fwd_int4_grouped(X[0], q, s, offsets, zeros=z, stream=side), dp.dp_gemm_fwd_int4(X[0], *dense[:2], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graphs, outs = [torch.cuda.CUDAGraph() for _ in X], []
    for g, x in zip(graphs, X):
        with torch.cuda.graph(g):
            outs.append(step(x))
    X[0].copy_(rows(T, K, 5, False))
    offsets.copy_(torch.tensor([1, 1, 4, 4, 4, 15, 16, 20, 23], dtype=torch.int32))
    want = [step(x) for x in X]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in X]
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert dp.device_error() == 0


def test_the_same_layer_expanded():
    """Products of the 4-bit weights, and the BF16 products of the weights expanded: the expansion rounds (q - z) s to BF16 once."""
    N, K = 256, 1024
    W = normal((N, K), 1, BF16, K ** -0.5)
    q, s, z = dp.int4_quantize(W, 64, zeros=True)
    X = normal((12, K), 2)
    got, wide = dp.dp_gemm_fwd_int4(X, q, s, zeros=z, out_dtype=F32), dp.dp_gemm_fwd(X, dp.int4_dequantize(q, s, zeros=z), out_dtype=F32)
    mag = X.double().abs() @ expand(q, s, z, 64).abs().T
    assert bool(((got - wide).double().abs() <= (2.0 ** -8 + K * 2.0 ** -22) * mag).all())


def test_refusals():
    q, s, z = problem(0, 16, 256, 64, True, BF16, 1, False)
    qe, se, ze = problem(2, 16, 256, 64, True, BF16, 1, False)
    X, o = rows(3, 256, 1, False), torch.tensor([0, 1, 3], dtype=torch.int32, device=DEV)
    for call, kind, text in [
        (lambda: dp.dp_gemm_fwd_int4(X, q, s.half()), TypeError, "scales"),
        (lambda: dp.dp_gemm_fwd_int4(X, q.char(), s), TypeError, "uint8"),
        (lambda: dp.dp_gemm_fwd_int4(X, q, s[:, :3]), ValueError, "contiguous|groups"),
        (lambda: dp.dp_gemm_fwd_int4(X, q, s[:, :1].contiguous()), ValueError, "groups"),
        (lambda: dp.dp_gemm_fwd_int4(X, q[:8], s), ValueError, "same rows"),
        (lambda: dp.dp_gemm_fwd_int4(X, q, s, zeros=z[:, :2]), ValueError, "same rows"),
        (lambda: dp.dp_gemm_fwd_int4(X, q.t().contiguous().t(), s), ValueError, "contiguous"),
        (lambda: dp.dp_gemm_fwd_int4(X, q[:1].expand(16, 128), s), ValueError, "contiguous"),
        (lambda: dp.dp_gemm_fwd_int4(X.float(), q, s), TypeError, "bfloat16"),
        (lambda: dp.dp_gemm_fwd_int4(X[:, :128], q, s), ValueError, "weights' K"),
        (lambda: dp.dp_gemm_fwd_int4(X[:1].expand(3, 256), q, s), ValueError, "stride 0"),
        (lambda: dp.dp_gemm_fwd_int4(X, qe, se), ValueError, "same rows"),
        (lambda: dp.dp_gemm_fwd_int4(X, q.cpu(), s), ValueError, "CUDA tensor"),
        (lambda: dp.dp_gemm_fwd_int4(X, q[:12], s[:12]), dp.DPError, "status 3"),
        (lambda: dp.dp_gemm_fwd_int4_grouped(X, qe, se, o[:2]), ValueError, "E . 1 values"),
        (lambda: dp.dp_gemm_fwd_int4_grouped(X, qe, se, o.short()), TypeError, "int32 or int64"),
        (lambda: dp.int4_quantize(X, 48), ValueError, "group"),
        (lambda: dp.int4_quantize(X.half(), 64), TypeError, "bfloat16 or float32"),
        (lambda: dp.int4_quantize(X, 64, scale_dtype=torch.float16), TypeError, "scale_dtype"),
        (lambda: dp.int4_quantize(X.view(3, 2, 128).transpose(0, 1), 64), ValueError, "contiguous"),
        (lambda: dp.int4_dequantize(q, s, out_dtype=torch.float16), TypeError, "out_dtype"),
    ]:
        with pytest.raises(kind, match=text):
            call()
