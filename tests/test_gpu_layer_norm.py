"""Layer norm against its definition in 64 bits.

u = 2^-24 (FP32 round to nearest).  A thread adds up to 16 values, then up to 10 + 1 pairwise steps: a sum over a
row is within 28 u of the sum of magnitudes.  With A = mean|x| / sigma the mean is off by 28 u A sigma, so
h = (x - mu) rs by u (28 A + |h| (28 A + 28)) (the variance has the same sums; division, root and
products a few u each).  Outputs in BF16 add half a step, 2^-8 |y|.
Backward, from the FP32 mean and rs: h and g h carry 3 to 5 u, the two means 28 u and theirs, the last operations
4 u:  |dx| within 48 u rs (|g| + mean|g| + |h| mean|g h|).
dw, db: a block adds its rows one after the other (at most T / blocks each), then the rows that it has at a time
(at most 64), then the at most 304 blocks in runs of up to 80: within (T / 152 + 64 + 80 + 8) u of the sum of magnitudes.
"""
import pytest
import torch

import fp32_dense_projection_gb300 as dp
from gpu_common import DEV

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-5


def rows(T, C, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, C, device=DEV, generator=g) * scale + shift
    return x.to(dtype)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def close(got, want, tol):
    off = (got.double() - want).abs()
    assert got.isfinite().all()
    assert bool((off <= tol).all()), float((off / tol.clamp_min(1e-300)).max())


def reference(x, w, b, eps=EPS):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    sigma2 = (x - mean).square().mean(1, keepdim=True)
    rs = 1 / (sigma2 + eps).sqrt()
    h = (x - mean) * rs
    w = torch.ones(x.shape[1], device=DEV, dtype=torch.float64) if w is None else w.double()
    b = torch.zeros(x.shape[1], device=DEV, dtype=torch.float64) if b is None else b.double()
    return mean, rs, h, h * w + b, w, b


def check_fwd(x, w, b, out, eps=EPS):
    y, mean, rstd = dp.layer_norm_fwd(x, w, b, eps=eps, out_dtype=out)
    m, rs, h, ref, wd, bd = reference(x, w, b, eps)
    A = x.double().abs().mean(1, keepdim=True) * rs
    assert y.dtype is out and y.shape == x.shape and mean.shape == rstd.shape == (x.shape[0],)
    close(mean[:, None], m, 28 * U * x.double().abs().mean(1, keepdim=True))
    close(rstd[:, None], rs, rs * U * (28 * A + 28))
    tol = wd.abs() * U * (28 * A + h.abs() * (28 * A + 30)) + 2 * U * (ref.abs() + bd.abs())
    close(y, ref, tol + (half_step(out) * (ref.abs() + tol) if out is BF16 else 0))
    return y, mean, rstd


def check_bwd(dy, x, w, mean, rstd, out):
    dx, dw, db = dp.layer_norm_bwd(dy, x, mean, rstd, w, dx_dtype=out)
    T, C = x.shape
    rs = rstd.double()[:, None]
    h = (x.double() - mean.double()[:, None]) * rs
    d = dy.double()
    g = d if w is None else d * w.double()
    ref = rs * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    tol = 48 * U * rs * (g.abs() + g.abs().mean(1, keepdim=True) + h.abs() * (g * h).abs().mean(1, keepdim=True))
    assert dx.dtype is out
    close(dx, ref, tol + (half_step(out) * (ref.abs() + tol) if out is BF16 else 0))
    if w is None:
        assert dw is None and db is None
        return
    depth = T / 152 + 160
    close(dw, (d * h).sum(0), (depth + 5) * U * (d * h).abs().sum(0))
    close(db, d.sum(0), depth * U * d.abs().sum(0))


SIZES = [(1, 8), (1, 4096), (2, 64), (3, 72), (7, 1000), (33, 136), (129, 256), (64, 1024), (31, 1032), (1000, 2048), (17, 2056),
         (300, 4096), (40, 4104), (25, 8192), (12, 8200), (9, 16384), (5, 12288), (4031, 1024), (1215, 4096)]


@pytest.mark.parametrize("T,C", SIZES)
@pytest.mark.parametrize("xt,wt,out", [(BF16, BF16, BF16), (F32, F32, F32), (BF16, F32, F32), (F32, BF16, BF16)])
def test_forward_and_backward(T, C, xt, wt, out):
    x = rows(T, C, xt, T + C, shift=0.5)
    w, b = rows(1, C, wt, 1)[0] + 1, rows(1, C, wt, 2)[0]
    _, mean, rstd = check_fwd(x, w, b, out)
    for gt in (BF16, F32):
        check_bwd(rows(T, C, gt, 3 * T + C), x, w, mean, rstd, out)
    assert dp.device_error() == 0


# Rows enough that blocks go round their shared memory several times, in each form: threads of a row a power of two or whole
# warps, one row or several a block.
@pytest.mark.parametrize("T,C", [(20000, 72), (9000, 200), (5000, 776), (3001, 1544), (2003, 2560), (1300, 4160), (1200, 5120), (1000, 6152), (901, 8192),
                                 (700, 8200), (703, 10240), (500, 16384)])
@pytest.mark.parametrize("xt,gt", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
def test_many_rows(T, C, xt, gt):
    x = rows(T, C, xt, T + C, shift=0.5)
    w, b = rows(1, C, F32, 1)[0] + 1, rows(1, C, BF16, 2)[0].float()
    _, mean, rstd = check_fwd(x, w, b, BF16)
    check_bwd(rows(T, C, gt, 3 * T + C), x, w, mean, rstd, F32)
    assert dp.device_error() == 0


@pytest.mark.parametrize("T,C", [(5, 64), (200, 1000), (50, 4096), (3, 16384)])
def test_without_weight_or_bias(T, C):
    x, dy = rows(T, C, BF16, 1, shift=1.0), rows(T, C, BF16, 2)
    w = rows(1, C, F32, 3)[0]
    check_fwd(x, None, w, F32)
    check_fwd(x, w, None, BF16)
    _, mean, rstd = check_fwd(x, None, None, F32)
    check_bwd(dy, x, None, mean, rstd, BF16)
    check_bwd(dy, x, None, mean, rstd, F32)


@pytest.mark.parametrize("scale,shift", [(1.0, 1000.0), (1e-4, 0.0), (1e4, 0.0), (1e-3, 100.0)])
def test_rows_far_from_zero(scale, shift):
    """The variance is that of the distances: a large mean costs no more than the values' own rounding."""
    x = rows(100, 1024, F32, 5, scale, shift)
    w, b = rows(1, 1024, F32, 1)[0], rows(1, 1024, F32, 2)[0]
    _, mean, rstd = check_fwd(x, w, b, F32)
    check_bwd(rows(100, 1024, F32, 6), x, w, mean, rstd, F32)


def test_constant_and_zero_rows():
    x = torch.zeros(3, 256, device=DEV)
    x[1] = 7.0
    w, b = rows(1, 256, F32, 1)[0], rows(1, 256, F32, 2)[0]
    y, mean, rstd = dp.layer_norm_fwd(x, w, b, eps=0.25, out_dtype=F32)
    assert torch.equal(y, b.expand(3, -1)) and mean.tolist() == [0.0, 7.0, 0.0] and rstd.tolist() == [2.0] * 3
    y, _, rstd = dp.layer_norm_fwd(x, w, b, eps=0.0, out_dtype=F32)  # 0 / 0
    assert y.isnan().all() and rstd.isinf().all()


@pytest.mark.parametrize("C", [64, 1000, 4096, 16384])
def test_bad_rows_stay_by_themselves(C):
    """An infinity or a NaN reaches its own row's outputs (and dw, db) only."""
    x, dy, w = rows(70, C, BF16, 1), rows(70, C, BF16, 2), rows(1, C, BF16, 3)[0]
    clean = dp.layer_norm_fwd(x, w, w)
    grads = dp.layer_norm_bwd(dy, x, clean[1], clean[2], w)
    bad = x.clone()
    bad[5, 3], bad[64, C - 1] = float("inf"), float("nan")
    got = dp.layer_norm_fwd(bad, w, w)
    keep = torch.ones(70, dtype=torch.bool, device=DEV)
    keep[[5, 64]] = False
    for a, c in zip(got, clean):
        assert torch.equal(a[keep], c[keep])
    assert got[0][5].isnan().any() and got[0][64].isnan().all()
    dx, dw, _ = dp.layer_norm_bwd(dy, bad, got[1], got[2], w)
    assert torch.equal(dx[keep], grads[0][keep]) and dx[64].isnan().all() and dw.isnan().any()


@pytest.mark.parametrize("C", [64, 1024, 4104])
def test_padded_rows(C):
    """Rows further apart than their length: the same bits, and nothing between them is written."""
    T = 77
    x, dy = rows(T, C + 16, BF16, 1)[:, :C], rows(T, C + 32, F32, 2)[:, :C]
    w, b = rows(1, C, F32, 3)[0], rows(1, C, F32, 4)[0]
    ybuf, dbuf = torch.full((T, C + 24), 7.0, device=DEV, dtype=BF16), torch.full((T, C + 8), 7.0, device=DEV)
    y, mean, rstd = dp.layer_norm_fwd(x, w, b, out=ybuf[:, :C])
    dx, dw, db = dp.layer_norm_bwd(dy, x, mean, rstd, w, dX=dbuf[:, :C])
    want = dp.layer_norm_fwd(x.contiguous(), w, b)
    grads = dp.layer_norm_bwd(dy.contiguous(), x.contiguous(), mean, rstd, w, dx_dtype=F32)
    for a, c in zip((y, mean, rstd, dx, dw, db), (*want, *grads)):
        assert torch.equal(a, c)
    assert bool((ybuf[:, C:] == 7).all()) and bool((dbuf[:, C:] == 7).all())


def test_no_tokens():
    x, w = torch.empty(0, 64, device=DEV, dtype=BF16), torch.ones(64, device=DEV)
    y, mean, rstd = dp.layer_norm_fwd(x, w, w)
    assert y.shape == (0, 64) and mean.shape == rstd.shape == (0,)
    dx, dw, db = dp.layer_norm_bwd(x, x, mean, rstd, w)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_repeats_bit_for_bit():
    x, dy, w = rows(5000, 1024, BF16, 1), rows(5000, 1024, BF16, 2), rows(1, 1024, F32, 3)[0]
    _, mean, rstd = dp.layer_norm_fwd(x, w, w)
    first = dp.layer_norm_bwd(dy, x, mean, rstd, w)
    for _ in range(5):
        for a, b in zip(first, dp.layer_norm_bwd(dy, x, mean, rstd, w)):
            assert torch.equal(a, b)


def test_gradient_against_differences():
    """d/de of sum(dy * norm(x + e v)) by central differences of the definition in 64 bits.  The differences' own error is
    e^2 times the third derivative (1e-10 for e = 1e-5 on rows of deviation 1), the kernel's as above."""
    T, C, e = 6, 200, 1e-5
    x, dy, w, b = rows(T, C, F32, 1), rows(T, C, F32, 2), rows(1, C, F32, 3)[0], rows(1, C, F32, 4)[0]
    _, mean, rstd = dp.layer_norm_fwd(x, w, b, out_dtype=F32)
    dx, dw, db = dp.layer_norm_bwd(dy, x, mean, rstd, w, dx_dtype=F32)

    def f(x, w, b):
        return float((dy.double() * reference(x, w, b)[3]).sum())
    for seed in range(4):
        v, vw, vb = rows(T, C, F32, 10 + seed).double(), rows(1, C, F32, 20 + seed)[0].double(), rows(1, C, F32, 30 + seed)[0].double()
        for got, vec, lo, hi in ((dx, v, (x - e * v, w, b), (x.double() + e * v, w, b)), (dw, vw, (x, w.double() - e * vw, b), (x, w.double() + e * vw, b)),
                                 (db, vb, (x, w, b.double() - e * vb), (x, w, b.double() + e * vb))):
            want = (f(*hi) - f(lo[0].double(), lo[1], lo[2])) / (2 * e)
            scale = float((got.double() * vec).abs().sum())
            assert abs(float((got.double() * vec).sum()) - want) <= 1e-5 * scale


def test_streams_and_graphs():
    """On a stream of its own, and captured: replays follow new inputs, two graphs do not disturb each other."""
    shapes = [(64, 1024), (900, 4096)]
    w = {C: rows(1, C, F32, C)[0] for _, C in shapes}
    x = {s: rows(*s, BF16, 1) for s in shapes}
    dy = {s: rows(*s, BF16, 2) for s in shapes}

    def step(s):
        y, mean, rstd = dp.layer_norm_fwd(x[s], w[s[1]], w[s[1]])
        return (y, mean, rstd, *dp.layer_norm_bwd(dy[s], x[s], mean, rstd, w[s[1]]))
    side = torch.cuda.Stream()
    want = {s: [t.clone() for t in step(s)] for s in shapes}
    side.wait_stream(torch.cuda.current_stream())
    y, mean, rstd = dp.layer_norm_fwd(x[shapes[0]], w[1024], w[1024], stream=side)
    got = dp.layer_norm_bwd(dy[shapes[0]], x[shapes[0]], mean, rstd, w[1024], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip((y, mean, rstd, *got), want[shapes[0]]):
        assert torch.equal(a, b)
    graphs, outs = {}, {}
    for s in shapes:
        graphs[s] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[s]):
            outs[s] = step(s)
    for s in shapes:
        x[s].copy_(rows(*s, BF16, 7))
    want = {s: [t.clone() for t in step(s)] for s in shapes}
    torch.cuda.synchronize()
    streams = {s: torch.cuda.Stream() for s in shapes}
    for _ in range(3):
        for s in shapes:
            with torch.cuda.stream(streams[s]):
                graphs[s].replay()
    torch.cuda.synchronize()
    for s in shapes:
        for a, b in zip(outs[s], want[s]):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """2^31 elements and more: the last rows are where they belong."""
    T, C = (1 << 31) // 4096 + 100, 4096
    x = torch.empty(T, C, device=DEV, dtype=BF16)
    tail = rows(200, C, BF16, 1)
    x[:-200] = 1
    x[-200:] = tail
    w = rows(1, C, F32, 2)[0]
    y, mean, rstd = dp.layer_norm_fwd(x, w, w)
    want = dp.layer_norm_fwd(tail, w, w)
    assert torch.equal(y[-200:], want[0]) and torch.equal(mean[-200:], want[1]) and torch.equal(rstd[-200:], want[2])
    dx, _, _ = dp.layer_norm_bwd(x, x, mean, rstd, w)
    assert torch.equal(dx[-200:], dp.layer_norm_bwd(tail, tail, *want[1:], w)[0])


def test_refusals():
    x, w = torch.zeros(4, 64, device=DEV, dtype=BF16), torch.ones(64, device=DEV)
    y, mean, rstd = dp.layer_norm_fwd(x, w)
    for call, kind, text in [
        (lambda: dp.layer_norm_fwd(x, w.cpu()), ValueError, "CUDA tensor"),
        (lambda: dp.layer_norm_fwd(x, w[:32]), ValueError, "vector of 64"),
        (lambda: dp.layer_norm_fwd(x, w, w.bfloat16()), TypeError, "same type"),
        (lambda: dp.layer_norm_fwd(x.half(), w), TypeError, "bfloat16 or float32"),
        (lambda: dp.layer_norm_fwd(x[:1].expand(4, 64), w), ValueError, "stride 0"),
        (lambda: dp.layer_norm_fwd(x, w, out=y[:, :32]), ValueError, "out must have shape"),
        (lambda: dp.layer_norm_fwd(x, w, out_dtype=torch.float16), TypeError, "out_dtype"),
        (lambda: dp.layer_norm_fwd(x, w, eps=-1.0), dp.DPError, "status 1"),
        (lambda: dp.layer_norm_fwd(x[:, :60], w[:60]), dp.DPError, "status 3"),
        (lambda: dp.layer_norm_fwd(x[:, 4:60], w[4:60]), dp.DPError, "status 2"),
        (lambda: dp.layer_norm_bwd(x, x[:2], mean, rstd, w), ValueError, "same shape"),
        (lambda: dp.layer_norm_bwd(x, x, mean[:2], rstd, w), ValueError, "vector of 4"),
        (lambda: dp.layer_norm_bwd(x, x, mean, rstd.double(), w), TypeError, "float32"),
        (lambda: dp.layer_norm_bwd(x, x, mean, rstd, w, workspace=torch.empty(16, dtype=torch.uint8, device=DEV)), dp.DPError, "status 4"),
    ]:
        with pytest.raises(kind, match=text):
            call()


@pytest.mark.parametrize("T,C,xt,gt", [(5, 8192, F32, F32), (5, 8200, F32, F32), (3, 16384, F32, BF16), (4, 4096, BF16, BF16), (7, 4104, BF16, BF16)])
@pytest.mark.parametrize("sigma,dy", [(1e-20, 1.0), (1e-22, 1.0), (1e17, 1e-6)])
def test_gradient_of_tiny_and_large_deviations(T, C, xt, gt, sigma, dy):
    """rs of 1e20, 1e22 and 1e-17, whose squares leave FP32's range or its normal numbers: only rs itself may meet a row's values."""
    x, g, w = rows(T, C, xt, 1, sigma), rows(T, C, gt, 2, dy), rows(1, C, F32, 3)[0] + 1
    mean, rs = reference(x, None, None, 0.0)[:2]
    check_bwd(g, x, w, mean[:, 0].float(), rs[:, 0].float(), F32)


@pytest.mark.parametrize("T,C,xt,gt", [(1, 64, BF16, BF16), (200, 1000, BF16, F32), (50, 4096, F32, F32), (900, 4104, BF16, BF16), (3, 16384, F32, BF16)])
def test_parameter_gradients_without_a_weight(T, C, xt, gt):
    """A bias alone has its gradient, and a weight of ones that is not there too; with a weight they can be left out."""
    x, dy = rows(T, C, xt, 1, shift=0.5), rows(T, C, gt, 2)
    w, b = rows(1, C, F32, 3)[0], rows(1, C, F32, 4)[0]
    _, mean, rstd = dp.layer_norm_fwd(x, None, b)
    dx, dw, db = dp.layer_norm_bwd(dy, x, mean, rstd, param_grads=True)
    ones = dp.layer_norm_bwd(dy, x, mean, rstd, torch.ones(C, device=DEV))
    for got, same in zip((dx, dw, db), ones):
        assert torch.equal(got, same)
    d, h, depth = dy.double(), (x.double() - mean.double()[:, None]) * rstd.double()[:, None], T / 152 + 160
    close(dw, (d * h).sum(0), (depth + 5) * U * (d * h).abs().sum(0))
    close(db, d.sum(0), depth * U * d.abs().sum(0))
    given = dp.layer_norm_bwd(dy, x, mean, rstd, param_grads=True, workspace=torch.empty(64 << 20, dtype=torch.uint8, device=DEV))
    assert torch.equal(given[1], dw) and torch.equal(given[2], db)
    got = dp.layer_norm_bwd(dy, x, mean, rstd, w, param_grads=False)
    assert got[1] is None and got[2] is None and torch.equal(got[0], dp.layer_norm_bwd(dy, x, mean, rstd, w)[0])
    empty = dp.layer_norm_bwd(dy[:0], x[:0], mean[:0], rstd[:0], param_grads=True)
    assert empty[0].shape == (0, C) and not empty[1].any() and not empty[2].any()


@pytest.mark.parametrize("T,C,block,tpr", [(16384, 4096, 256, 256), (20001, 2304, 160, 160), (30000, 1024, 256, 64), (60000, 72, 256, 8)])
def test_parameter_gradients_at_the_blocks_own_bound(T, C, block, tpr):
    """BF16 rows of two pieces of eight columns a thread: `block` threads, tpr for a row, 512 threads an SM.  Each group of tpr adds
    n = T / groups rows one after the other (a fused step each), a block its groups, the second launch the blocks in 32 runs of
    `per` and the runs in 5 steps; h itself has 2 roundings, and one is left for the products of these: n + groups a block + per + 8."""
    x, dy = rows(T, C, BF16, 1, shift=0.5), rows(T, C, BF16, 2)
    w = rows(1, C, F32, 3)[0]
    _, mean, rstd = dp.layer_norm_fwd(x, w, w)
    _, dw, db = dp.layer_norm_bwd(dy, x, mean, rstd, w)
    at_a_time = block // tpr
    blocks = min(-(-T // at_a_time), torch.cuda.get_device_properties(0).multi_processor_count * (512 // block))
    steps = -(-T // (blocks * at_a_time)) + at_a_time + -(-blocks // 32) + 8
    d, h = dy.double(), (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    close(dw, (d * h).sum(0), steps * U * (d * h).abs().sum(0))
    close(db, d.sum(0), steps * U * d.abs().sum(0))
