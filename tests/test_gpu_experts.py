"""The way of tokens to their experts and back: the router's choice, the sort, gather and combine and
their gradients, against plain 64-bit forms.

u = 2^-24.  Gates: l - m is rounded once (u |l - m|), expf is within 2 ulp, a sum over E <= 1024 takes 32 + 5
steps, the quotient one more: relative error within 2 u (R + 24), R the row's range of open logits.
Sums over k choices: k + 1 steps; dot products over C: a thread adds C / (8 threads) pieces of 8 one after the other
and then 8 pairwise steps: within (C / 16 + 16) u of the sum of magnitudes, for any division among
at least 16 threads, or C (one thread).
"""
import pytest
import torch

import fp32_dense_projection_gb300 as dp
from gpu_common import DEV

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(shape, seed, dtype=F32):
    return torch.randn(shape, device=DEV, generator=gen(seed)).to(dtype)


def close(got, want, tol):
    assert got.isfinite().all()
    off = (got.double() - want).abs()
    assert bool((off <= tol).all()), float((off / tol.clamp_min(1e-300)).max())


# ------------------------------------------------------------------------ route

def plain_route(logits, k, renormalize):
    l = logits.double()
    top, choice = l.sort(dim=1, descending=True, stable=True)
    top, choice = top[:, :k], choice[:, :k]
    live = top > -INF
    # (quotients, not exp(l - log sum): beside a logit of -3e38 the logarithm of the sum is lost in 64 bits too)
    most = torch.where(live[:, :1], top[:, :1], 0.0)
    total = (top - most if renormalize else l - most).exp().sum(1, keepdim=True)
    gates = torch.where(live, (top - most).exp() / total, 0.0)
    return gates, torch.where(live, choice, -1).int()


def plain_route_bwd(dg, logits, gates, choice, renormalize):
    T, E = logits.shape
    dg = torch.where(choice >= 0, dg.double(), 0.0)
    at = torch.where(choice >= 0, choice.long(), E)
    full = torch.zeros(T, E + 1, dtype=torch.float64, device=DEV).scatter_add_(1, at, dg)[:, :E]
    if renormalize:
        p = torch.zeros(T, E + 1, dtype=torch.float64, device=DEV).scatter_add_(1, at, gates.double())[:, :E]
    else:
        l = logits.double()
        most = l.amax(1, keepdim=True)
        e = torch.where(l > -INF, (l - most).exp(), 0.0)
        p = torch.where(e > 0, e / e.sum(1, keepdim=True), 0.0)
    s = (p * full).sum(1, keepdim=True)
    return p * (full - s), p * (full.abs() + (p * full.abs()).sum(1, keepdim=True))


def spread(logits):
    open_ = torch.where(logits > -INF, logits, 0.0).double()
    return (open_.amax(1) - open_.amin(1)).clamp_min(0)[:, None]


def check_route(logits, k, renormalize, seed=1):
    gates, choice = dp.route_topk(logits, k, renormalize=renormalize)
    want, at = plain_route(logits, k, renormalize)
    assert gates.dtype is F32 and choice.dtype is torch.int32
    assert torch.equal(choice, at)
    rel = 2 * U * (spread(logits) + 24)
    close(gates, want, rel * want + 1e-37)
    dg = normal(gates.shape, seed)
    got = dp.route_topk_bwd(dg, logits, gates, choice, renormalize=renormalize)
    ref, mag = plain_route_bwd(dg, logits, want, at, renormalize)
    close(got, ref, (3 * rel + 2 * U * (k + 10)) * mag + 1e-37)
    return gates, choice, got


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (3, 2, 2), (8, 64, 8), (5, 31, 3), (100, 33, 32), (7, 65, 5), (200, 128, 1),
                                   (1000, 256, 8), (4031, 256, 4), (9, 257, 7), (33, 512, 16), (50, 513, 8), (20, 1000, 10), (3, 1024, 32)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route(T, E, k, renormalize):
    check_route(normal((T, E), T + E) * 2, k, renormalize)


@pytest.mark.parametrize("renormalize", [True, False])
def test_route_equal_logits(renormalize):
    """The lowest index first among equals; -0 equals 0."""
    few = torch.randint(-2, 3, (500, 256), device=DEV, generator=gen(1)).float()
    check_route(few, 8, renormalize)
    zeros = torch.zeros(4, 100, device=DEV)
    zeros[1, ::2] = -0.0
    _, choice, _ = check_route(zeros, 6, renormalize)
    assert choice.tolist() == [list(range(6))] * 4


@pytest.mark.parametrize("values", [1, 2, 5, 40])
@pytest.mark.parametrize("E,k", [(40, 3), (64, 16), (128, 8), (250, 2), (256, 16), (256, 17), (500, 12), (1000, 16), (1000, 32)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_few_values(values, E, k, renormalize):
    """Logits of few values, a third of them closed: more candidates above the bound than lanes, or just as many."""
    l = torch.randint(0, values, (300, E), device=DEV, generator=gen(E + k)).float() / 4
    l[:, ::3] = -INF
    l[7, 5:] = -INF
    check_route(l, k, renormalize)


@pytest.mark.parametrize("renormalize", [True, False])
def test_route_closed_experts(renormalize):
    """Rows with some, all but one, and all experts closed; the smallest finite logits are open."""
    l = normal((300, 96), 3)
    l[:, ::3] = -INF
    l[10:20] = -INF
    l[20:30, 1:] = -INF
    l[20:30, 0] = 4.0
    l[30:40, 5:] = -INF
    l[40] = torch.finfo(F32).min
    gates, choice, d = check_route(l, 8, renormalize)
    assert not gates[10:20].any() and bool((choice[10:20] == -1).all()) and not d[10:20].any()
    assert bool((choice[20:30, 1:] == -1).all()) and bool((gates[20:30, 0] == 1).all())
    assert torch.equal(choice[40], torch.arange(8, device=DEV, dtype=torch.int32))


@pytest.mark.parametrize("T,E,k", [(3, 1, 1), (300, 64, 8), (300, 64, 20), (100, 250, 16), (50, 1000, 8), (50, 1024, 32)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gates_far_below_the_largest(T, E, k, renormalize):
    """Logits up to 80 apart whose distances are exact in FP32 (multiples of 1/64), so that the exponential's own error is what is
    left: 2 ulp, 4 u of a term at any distance.  The sum of at most E / 32 terms a lane and 5 steps over the warp: 4 + E / 32 + 5
    u, the quotient 1: a gate is off by (14 + E / 32) u of itself, and one u for the products of these.
    Gradient over all, of an expert that is not chosen: p s with s = sum dg gate of gates this far off, k <= 32 products and
    5 steps; of a chosen one gate (dg - s), two steps more.  Below FP32's normal numbers each of two products is off by half
    their spacing."""
    l = torch.randint(-80 * 64, 1, (T, E), device=DEV, generator=gen(E + k)).float() / 64
    l[:, 0] = 0.0  # (the largest, so that the others are as far below as they say)
    gates, choice = dp.route_topk(l, k, renormalize=renormalize)
    want, at = plain_route(l, k, renormalize)
    rel = (15 + E / 32) * U
    assert torch.equal(choice, at)
    close(gates, want, rel * want)
    dg = normal((T, k), 1)
    ref, mag = plain_route_bwd(dg, l, want, at, renormalize)
    close(dp.route_topk_bwd(dg, l, gates, choice, renormalize=renormalize), ref, (2 * rel + 9 * U) * mag + 2.0 ** -149)


@pytest.mark.parametrize("renormalize", [True, False])
def test_route_nan_and_infinity(renormalize):
    """A NaN is the largest, its row's gates are NaN; +infinity likewise; other rows do not notice."""
    l = normal((20, 64), 4)
    clean = dp.route_topk(l, 4, renormalize=renormalize)
    bad = l.clone()
    bad[3, 17], bad[7, 40], bad[7, 50] = float("nan"), INF, -INF
    bad[9, 60], bad[9, 2] = -float("nan"), INF
    gates, choice = dp.route_topk(bad, 4, renormalize=renormalize)
    keep = torch.ones(20, dtype=torch.bool, device=DEV)
    keep[[3, 7, 9]] = False
    assert torch.equal(gates[keep], clean[0][keep]) and torch.equal(choice[keep], clean[1][keep])
    assert choice[3, 0] == 17 and choice[7, 0] == 40 and choice[9].tolist()[:2] == [60, 2]
    assert bool(gates[3].isnan().all()) and bool(gates[9].isnan().all()) and bool(gates[7, 0].isnan())
    d = dp.route_topk_bwd(normal((20, 4), 5), bad, gates, choice, renormalize=renormalize)
    assert d[keep].isfinite().all() and bool(d[3].isnan().any()) and bool(d[7].isnan().any())


def test_route_gradient_takes_any_choice():
    """An index twice adds up; indexes outside [0, E) and their gradients, whatever they are, take no part."""
    l, dg = normal((40, 50), 1), normal((40, 4), 2)
    gates, choice = dp.route_topk(l, 4)
    choice[:, 1] = choice[:, 0]
    want, mag = plain_route_bwd(dg, l, gates, choice, True)
    g, d = gates.double(), dg.double()
    own = g * (d - (g * d).sum(1, keepdim=True))
    want = torch.zeros_like(want).scatter_add_(1, choice.long(), own)
    close(dp.route_topk_bwd(dg, l, gates, choice), want, 30 * U * (g * (d.abs() + (g * d).abs().sum(1, keepdim=True))).sum(1, keepdim=True))
    choice[:, 1], choice[:, 2] = -1, 50
    dg[:, 1], dg[:, 2] = float("nan"), INF
    assert dp.route_topk_bwd(dg, l, gates, choice).isfinite().all()
    assert dp.route_topk_bwd(dg, l, gates, choice, renormalize=False).isfinite().all()


@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_against_differences(renormalize):
    """Central differences of the 64-bit gates with the choice held fixed (e = 1e-5: their own error is below 1e-9)."""
    l, dg = normal((12, 40), 1), normal((12, 6), 2)
    gates, choice = dp.route_topk(l, 6, renormalize=renormalize)
    d = dp.route_topk_bwd(dg, l, gates, choice, renormalize=renormalize).double()

    def f(l):
        top = l.gather(1, choice.long())
        return float((dg.double() * (top - torch.logsumexp(top if renormalize else l, 1, keepdim=True)).exp()).sum())
    for seed in range(4):
        v = normal((12, 40), 10 + seed).double()
        want = (f(l.double() + 1e-5 * v) - f(l.double() - 1e-5 * v)) / 2e-5
        assert abs(float((d * v).sum()) - want) <= 1e-5 * float((d * v).abs().sum())


def test_route_strides():
    """Rows further apart than E, at any 4-byte offset; the columns behind are left alone."""
    wide = normal((50, 90), 1)
    l = wide[:, 7:70]
    gates, choice = dp.route_topk(l, 5, renormalize=False)
    want = dp.route_topk(l.contiguous(), 5, renormalize=False)
    assert torch.equal(gates, want[0]) and torch.equal(choice, want[1])
    dg = normal((50, 5), 2)
    buf = torch.full((50, 80), 7.0, device=DEV)
    d = dp.route_topk_bwd(dg, l, gates, choice, renormalize=False, out=buf[:, 3:66])
    assert torch.equal(d, dp.route_topk_bwd(dg, l.contiguous(), gates, choice, renormalize=False))
    assert bool((buf[:, :3] == 7).all()) and bool((buf[:, 66:] == 7).all())


# ------------------------------------------------------------------------- sort

def plain_sort(choice, E):
    flat = choice.flatten().long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = key.argsort(stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel(), device=DEV)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.bincount(key, minlength=E + 1)[:E].cumsum(0)
    return offsets, torch.where(key < E, row, ~row).int().view(choice.shape), order.int()


def check_sort(choice, E):
    got = dp.expert_sort(choice, E)
    for a, b in zip(got, plain_sort(choice, E)):
        assert a.dtype is torch.int32 and torch.equal(a, b)
    return got


@pytest.mark.parametrize("T,k", [(0, 3), (1, 1), (1, 8), (8, 8), (31, 1), (33, 1), (100, 7), (341, 3), (1024, 4), (2048, 8), (4031, 6),
                                 (16384, 8), (50021, 5), (300000, 4)])
@pytest.mark.parametrize("E", [1, 2, 8, 64, 256, 385, 1000, 1024])
def test_sort(T, k, E):
    choice = torch.randint(0, E, (T, k), device=DEV, generator=gen(T + E), dtype=torch.int32)
    check_sort(choice, E)
    if T in (0, 33, 2048, 50021):
        some = torch.where(torch.rand(T, k, device=DEV, generator=gen(2)) < 0.3, -1, choice)
        check_sort(some, E)
        check_sort(some.long(), E)


@pytest.mark.parametrize("pairs", [1, 77, 5000, 400000])
def test_sort_one_sided(pairs):
    """All pairs with one expert, none with any, descending and alternating experts, entries far outside."""
    at = torch.arange(pairs, device=DEV)
    for E in (1, 3, 256, 1024):
        for choice in (torch.full((pairs,), E - 1, device=DEV), torch.zeros(pairs, device=DEV, dtype=torch.int64), torch.full((pairs,), -1, device=DEV),
                       (pairs - 1 - at) * E // pairs, at % E, torch.where(at % 2 == 0, 0, E - 1)):
            check_sort(choice.int(), E)
            check_sort(choice.long(), E)
        far = torch.where(at % 3 == 0, torch.tensor(1 << 40, device=DEV), torch.where(at % 3 == 1, torch.tensor(-(1 << 33), device=DEV), at % E))
        check_sort(far, E)
        check_sort(torch.where(at % 2 == 0, E, at % E).int(), E)


@pytest.mark.parametrize("cluster", ["0", "1"])
@pytest.mark.parametrize("pairs", [1, 500, 4096, 70001, 262144, 500000])
def test_sort_forms(pairs, cluster, monkeypatch):
    """One launch of a cluster, and two launches."""
    monkeypatch.setenv("DP_FORCE_SORT_CLUSTER", cluster)
    for E in (1, 64, 257, 1024):
        choice = torch.randint(-1, E, (pairs,), device=DEV, generator=gen(E), dtype=torch.int32)
        check_sort(choice, E)
        check_sort(torch.sort(choice, descending=True).values.long(), E)


def test_sort_feeds_the_grouped_products():
    """The offsets are the grouped products', whose padding the pairs without an expert are."""
    E, T, k, C = 16, 500, 2, 64
    choice = torch.randint(-1, E, (T, k), device=DEV, generator=gen(1), dtype=torch.int32)
    x = torch.randint(-3, 4, (T, C), device=DEV, generator=gen(2)).bfloat16()
    W = torch.randint(-3, 4, (E, 32, C), device=DEV, generator=gen(3)).bfloat16()
    gates = torch.randint(1, 4, (T, k), device=DEV, generator=gen(4)).float()
    offsets, row_of, order = dp.expert_sort(choice, E)
    y = dp.dp_gemm_fwd_grouped(dp.expert_gather(x, row_of), W, offsets, out_dtype=F32)
    out = dp.expert_combine(y, row_of, gates, out_dtype=F32)
    live = (choice >= 0).double()
    want = torch.einsum("tkn,tk->tn", torch.einsum("tc,tknc->tkn", x.double(), W.double()[choice.long().clamp_min(0)]), gates.double() * live)
    assert torch.equal(out, want.float()) and dp.device_error() == 0


# --------------------------------------------------------------- gather, combine

def pairs_of(T, k, E, seed, dropped=0.1):
    choice = torch.randint(0, E, (T, k), device=DEV, generator=gen(seed), dtype=torch.int32)
    choice = torch.where(torch.rand(T, k, device=DEV, generator=gen(seed + 1)) < dropped, -1, choice)
    return dp.expert_sort(choice, E)[1]


SHAPES = [(1, 1, 8), (1, 8, 4096), (5, 3, 64), (8, 8, 1000), (33, 2, 136), (100, 12, 2048), (257, 4, 2056), (1000, 1, 256), (64, 6, 8192),
          (3, 2, 20480), (40, 40, 72)]


@pytest.mark.parametrize("T,k,C", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gather(T, k, C, dtype):
    row_of = pairs_of(T, k, 16, T)
    x = normal((T, C), 3, dtype)
    got = dp.expert_gather(x, row_of)
    at = row_of.flatten().long()
    want = torch.empty(T * k, C, device=DEV, dtype=dtype)
    want[torch.where(at < 0, ~at, at)] = torch.where((at >= 0)[:, None], x.repeat_interleave(k, 0), 0)
    assert got.dtype is dtype and torch.equal(got, want)


def plain_combine(y, row_of, gates, add, mag=False):
    f = (lambda t: t.double().abs()) if mag else (lambda t: t.double())
    T, k = row_of.shape
    at = row_of.long()
    g = torch.ones(T, k, device=DEV, dtype=torch.float64) if gates is None else f(gates)
    out = (f(y)[at.clamp_min(0).flatten()].view(T, k, -1) * torch.where(at >= 0, g, 0.0)[:, :, None]).sum(1)
    return out if add is None else out + f(add)


@pytest.mark.parametrize("T,k,C", SHAPES)
@pytest.mark.parametrize("yt,out", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
def test_combine(T, k, C, yt, out):
    row_of = pairs_of(T, k, 16, T)
    y, gates, add = normal((T * k, C), 1, yt), normal((T, k), 2), normal((T, C), 3, out)
    for g in (gates, None):
        for a in (add, None):
            got = dp.expert_combine(y, row_of, g, add=a, out_dtype=out)
            want = plain_combine(y, row_of, g, a)
            tol = (k + 1) * U * plain_combine(y, row_of, g, a, True)
            assert got.dtype is out
            close(got, want, tol + (2.0 ** -8 * (want.abs() + tol) if out is BF16 else 0))


def check_combine_bwd(d, y, row_of, gates, out):
    d_y, d_gates = dp.expert_combine_bwd(d, y, row_of, gates, dy_dtype=out)
    T, k = row_of.shape
    C = y.shape[1]
    at = row_of.flatten().long()
    live, place = (at >= 0)[:, None], torch.where(at < 0, ~at, at)
    dd = d.double().repeat_interleave(k, 0)
    want = torch.empty(T * k, C, device=DEV, dtype=torch.float64)
    want[place] = torch.where(live, dd * gates.double().flatten()[:, None], 0.0)
    assert d_y.dtype is out
    close(d_y, want, 2 * U * want.abs() + (2.0 ** -8 * want.abs() if out is BF16 else 0))
    prod = torch.where(live, dd * y.double()[place], 0.0)
    close(d_gates, prod.sum(1).view(T, k), (C / 16 + 24) * U * prod.abs().sum(1).view(T, k))


@pytest.mark.parametrize("T,k,C", SHAPES)
@pytest.mark.parametrize("dt,yt,out", [(BF16, BF16, BF16), (F32, F32, F32), (F32, BF16, BF16), (BF16, F32, F32), (F32, F32, BF16),
                                       (BF16, BF16, F32), (F32, BF16, F32), (BF16, F32, BF16)])
def test_combine_gradient(T, k, C, dt, yt, out):
    check_combine_bwd(normal((T, C), 1, dt), normal((T * k, C), 2, yt), pairs_of(T, k, 16, T), normal((T, k), 3), out)


def test_gradients_are_the_adjoints():
    """combine without gates is the transpose of gather, and combine's gradient that of combine: inner products agree exactly
    on small integers."""
    T, k, C = 60, 3, 128
    row_of = pairs_of(T, k, 8, 5)

    def ints(shape, seed):
        return torch.randint(-4, 5, shape, device=DEV, generator=gen(seed)).float()
    x, r, y, gates, d = ints((T, C), 1), ints((T * k, C), 2), ints((T * k, C), 3), ints((T, k), 4), ints((T, C), 5)
    assert float((dp.expert_gather(x, row_of) * r).sum()) == float((x * dp.expert_combine(r, row_of, out_dtype=F32)).sum())
    out = dp.expert_combine(y, row_of, gates, out_dtype=F32)
    d_y, d_gates = dp.expert_combine_bwd(d, y, row_of, gates, dy_dtype=F32)
    total = float((out * d).sum())
    assert float((d_y * y).sum()) == total and float((d_gates * gates).sum()) == total


def test_bad_values_stay_by_themselves():
    """Infinities and NaN in one token's rows, and in rows and gates without an expert, reach nothing else."""
    T, k, C = 30, 4, 264
    row_of = pairs_of(T, k, 6, 3, 0.3)
    y, gates, d = normal((T * k, C), 1, BF16), normal((T, k), 2), normal((T, C), 3, BF16)
    out, grads = dp.expert_combine(y, row_of, gates), dp.expert_combine_bwd(d, y, row_of, gates)
    gone = row_of < 0
    y2, g2 = y.clone(), gates.clone()
    y2[(~row_of[gone]).long()] = float("nan")
    g2[gone] = INF
    assert torch.equal(dp.expert_combine(y2, row_of, g2), out)
    for a, b in zip(dp.expert_combine_bwd(d, y2, row_of, g2), grads):
        assert torch.equal(a, b)
    t, j = [int(v[0]) for v in torch.where(row_of >= 0)]
    y2 = y.clone()
    y2[int(row_of[t, j]), 5] = INF
    got = dp.expert_combine(y2, row_of, gates)
    same = torch.arange(T, device=DEV) != t
    assert torch.equal(got[same], out[same]) and not got[t, 5].isfinite() and torch.equal(got[t, :5], out[t, :5])
    got = dp.expert_combine_bwd(d, y2, row_of, gates)
    assert torch.equal(got[0], grads[0]) and torch.equal(got[1][same], grads[1][same]) and not got[1][t, j].isfinite()


def test_rows_outside_the_buffer_are_reported():
    """Entries that name no row are left out and reported; their neighbours are not harmed."""
    T, k, C = 20, 2, 64
    row_of = pairs_of(T, k, 4, 1, 0.0)
    y, gates, d = normal((T * k, C), 1), normal((T, k), 2), normal((T, C), 3)
    want = dp.expert_combine(y, row_of, gates, out_dtype=F32)
    dp.device_error()
    bad = row_of.clone()
    bad[3, 0], bad[7, 1], bad[9, 0] = T * k, 2 ** 31 - 1, -(2 ** 31)
    calls = (lambda: dp.expert_combine(y, bad, gates, out_dtype=F32), lambda: dp.expert_gather(d, bad), lambda: dp.expert_combine_bwd(d, y, bad, gates))
    for call in calls:
        got = call()
        assert dp.device_error() == 1 and dp.device_error() == 0
    got = calls[0]()
    same = torch.ones(T, dtype=torch.bool, device=DEV)
    same[[3, 7, 9]] = False
    assert torch.equal(got[same], want[same])
    assert float(calls[2]()[1][3, 0]) == 0.0
    dp.device_error()


def test_padded_rows():
    """Rows further apart than their length: the same bits, and nothing between them is written."""
    T, k, C = 50, 3, 136
    row_of = pairs_of(T, k, 8, 1)
    x, y = normal((T, C + 8), 1, BF16)[:, :C], normal((T * k, C + 16), 2, BF16)[:, :C]
    gates, add = normal((T, k), 3), normal((T, C + 24), 4, BF16)[:, :C]
    buf = [torch.full((n, C + 8), 7.0, device=DEV, dtype=BF16) for n in (T * k, T, T * k)]
    rows = dp.expert_gather(x, row_of, out=buf[0][:, :C])
    out = dp.expert_combine(y, row_of, gates, add=add, out=buf[1][:, :C])
    d_y, d_gates = dp.expert_combine_bwd(x, y, row_of, gates, d_y=buf[2][:, :C])
    xc, yc = x.contiguous(), y.contiguous()
    want = dp.expert_combine_bwd(xc, yc, row_of, gates)
    assert torch.equal(rows, dp.expert_gather(xc, row_of)) and torch.equal(out, dp.expert_combine(yc, row_of, gates, add=add.contiguous()))
    assert torch.equal(d_y, want[0]) and torch.equal(d_gates, want[1])
    assert all(bool((b[:, C:] == 7).all()) for b in buf)


def test_no_tokens():
    choice = torch.empty(0, 4, device=DEV, dtype=torch.int32)
    offsets, row_of, order = dp.expert_sort(choice, 8)
    assert not offsets.any() and offsets.shape == (9,) and row_of.shape == (0, 4) and order.shape == (0,)
    x, g = torch.empty(0, 64, device=DEV, dtype=BF16), torch.empty(0, 4, device=DEV)
    assert dp.expert_gather(x, row_of).shape == (0, 64) and dp.expert_combine(x, row_of, g).shape == (0, 64)
    assert [t.shape for t in dp.expert_combine_bwd(x, x, row_of, g)] == [(0, 64), (0, 4)]
    gates, c = dp.route_topk(torch.empty(0, 16, device=DEV), 2)
    assert gates.shape == c.shape == (0, 2)
    assert dp.route_topk_bwd(gates, torch.empty(0, 16, device=DEV), gates, c).shape == (0, 16)


def test_rows_past_32_bits():
    """2^31 elements and more in the sorted buffer: the last tokens' rows are where they belong."""
    k, C = 8, 4096
    T = (1 << 31) // (C * k) + 50
    choice = torch.randint(0, 64, (T, k), device=DEV, generator=gen(1), dtype=torch.int32)
    choice[-50:] = 63
    _, row_of, _ = dp.expert_sort(choice, 64)
    x = torch.empty(T, C, device=DEV, dtype=BF16)
    x[:-50], x[-50:] = 0.5, normal((50, C), 2, BF16)
    rows = dp.expert_gather(x, row_of)
    assert torch.equal(rows[row_of[-50:].long().flatten()], x[-50:].repeat_interleave(k, 0))
    gates = torch.full((T, k), 0.125, device=DEV)
    assert torch.equal(dp.expert_combine(rows, row_of, gates), x)
    d_y, d_gates = dp.expert_combine_bwd(x, rows, row_of, gates)
    assert torch.equal(d_y[row_of[-50:].long().flatten()], (x[-50:].float() * 0.125).bfloat16().repeat_interleave(k, 0))
    want = x[-50:].double().square().sum(1)
    close(d_gates[-50:], want[:, None].expand(50, k), (C / 16 + 24) * U * want[:, None])


# ------------------------------------------------------------- streams, graphs

def layer(x, logits, W, d_out, k, E):
    gates, choice = dp.route_topk(logits, k)
    offsets, row_of, order = dp.expert_sort(choice, E)
    rows = dp.expert_gather(x, row_of)
    y = dp.dp_gemm_fwd_grouped(rows, W, offsets)
    out = dp.expert_combine(y, row_of, gates)
    d_y, d_gates = dp.expert_combine_bwd(d_out, y, row_of, gates)
    d_rows = dp.dp_gemm_dgrad_grouped(d_y, W, offsets)
    d_x = dp.expert_combine(d_rows, row_of)
    d_logits = dp.route_topk_bwd(d_gates, logits, gates, choice)
    return gates, choice, offsets, row_of, order, rows, out, d_y, d_gates, d_x, d_logits


@pytest.mark.parametrize("T", [16, 3000, 20000])
def test_a_layer_on_streams_and_in_graphs(T):
    """The operators together: eager, on another stream, and two graphs that are replayed beside each other on new
    inputs give the same bits."""
    E, k, C = 32, 4, 256
    W = normal((E, C, C), 1, BF16)

    def inputs(seed):
        return normal((T, C), seed, BF16), normal((T, E), seed + 1), W, normal((T, C), seed + 2, BF16), k, E
    first, second = inputs(10), inputs(20)
    want = [layer(*first), layer(*second)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gates, choice = dp.route_topk(first[1], k, stream=side)
    offsets, row_of, order = dp.expert_sort(choice, E, stream=side)
    rows = dp.expert_gather(first[0], row_of, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip((gates, choice, offsets, row_of, order, rows), want[0]):
        assert torch.equal(a, b)
    held = [[t.clone() for t in i[:4]] for i in (first, first)]
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for g, h in zip(graphs, held):
        with torch.cuda.graph(g):
            outs.append(layer(*h, k, E))
    for h, i in zip(held, (second, first)):
        for a, b in zip(h, i[:4]):
            a.copy_(b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got, ref in zip(outs, (want[1], want[0])):
        for a, b in zip(got, ref):
            assert torch.equal(a, b)
    assert dp.device_error() == 0


def test_refusals():
    x, y = torch.zeros(4, 64, device=DEV, dtype=BF16), torch.zeros(8, 64, device=DEV, dtype=BF16)
    row_of = torch.arange(8, device=DEV, dtype=torch.int32).view(4, 2)
    l, gates = torch.zeros(4, 16, device=DEV), torch.zeros(4, 2, device=DEV)
    for call, kind, text in [
        (lambda: dp.route_topk(l, 0), ValueError, "k must lie"),
        (lambda: dp.route_topk(l, 17), ValueError, "k must lie"),
        (lambda: dp.route_topk(l.bfloat16(), 2), TypeError, "float32"),
        (lambda: dp.route_topk(l.t(), 2), ValueError, "unit column stride"),
        (lambda: dp.route_topk(l[:1].expand(4, 16), 2), ValueError, "stride 0"),
        (lambda: dp.route_topk(torch.zeros(2, 1025, device=DEV), 2), dp.DPError, "status 3"),
        (lambda: dp.route_topk(torch.zeros(2, 64, device=DEV), 33), dp.DPError, "status 3"),
        (lambda: dp.route_topk_bwd(gates, l, gates, row_of.long()), TypeError, "int32"),
        (lambda: dp.route_topk_bwd(gates[:, :1], l, gates, row_of), ValueError, "contiguous with shape"),
        (lambda: dp.route_topk_bwd(gates, l, gates, row_of, out=l.bfloat16()), TypeError, "float32"),
        (lambda: dp.expert_sort(row_of.short(), 4), TypeError, "int32 or int64"),
        (lambda: dp.expert_sort(row_of.t(), 4), ValueError, "contiguous"),
        (lambda: dp.expert_sort(row_of, 0), dp.DPError, "status 1"),
        (lambda: dp.expert_sort(row_of, 1025), dp.DPError, "status 3"),
        (lambda: dp.expert_sort(torch.zeros(1 << 20, device=DEV, dtype=torch.int32), 4, workspace=torch.empty(4, device=DEV)), dp.DPError, "status 4"),
        (lambda: dp.expert_gather(x, row_of.flatten()), ValueError, "T, k"),
        (lambda: dp.expert_gather(x[:2], row_of), ValueError, "same tokens"),
        (lambda: dp.expert_gather(x.half(), row_of), TypeError, "bfloat16 or float32"),
        (lambda: dp.expert_gather(x[:, :60], row_of), dp.DPError, "status 3"),
        (lambda: dp.expert_gather(x, row_of, out=y.float()), TypeError, "x's type"),
        (lambda: dp.expert_gather(x, row_of, out=y[:1].expand(8, 64)), ValueError, "stride 0"),
        (lambda: dp.expert_combine(x, row_of), ValueError, "shape"),
        (lambda: dp.expert_combine(y, row_of, gates.bfloat16()), TypeError, "float32"),
        (lambda: dp.expert_combine(y, row_of, gates, add=x.float()), TypeError, "out's type"),
        (lambda: dp.expert_combine(y, row_of, gates, add=x[:1].expand(4, 64)), ValueError, "stride 0"),
        (lambda: dp.expert_combine(y, row_of, gates.cpu()), ValueError, "CUDA tensor"),
        (lambda: dp.expert_combine_bwd(x, y, row_of, gates[:, :1]), ValueError, "contiguous with shape"),
        (lambda: dp.expert_combine_bwd(x[:2], y, row_of, gates), ValueError, "shape"),
    ]:
        with pytest.raises(kind, match=text):
            call()
