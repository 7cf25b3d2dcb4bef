"""Products grouped by expert against the definition in 64 bits.

Integer operands: every sum is exact in FP32, so outputs must be equal bit for bit.
Real operands: each tensor-core step (16 products and the running sum) loses at most a few
units of 2^-23 of the sum of magnitudes S = sum |a||b|; a piece of 2048 contraction elements
has 128 steps, and the pieces are added in FP32.  So
    |got - ref| <= 4 (min(K, 2048) / 16 + K / 2048 + 2) 2^-23 S     (FP32 out)
and a BF16 output adds its rounding, 2^-8 |ref| (half a unit is 2^-9).
"""
import numpy as np
import pytest
import torch

import fp32_dense_projection_gb300 as dp
from gpu_common import DEV

pytestmark = pytest.mark.gpu

OPS = ("fwd", "dgrad", "wgrad")


def edges_of(counts, front=0):
    return np.concatenate([[front], front + np.cumsum(counts)]).astype(np.int64)


def tensors(edges, T, N, K, seed, kn=False, real=False):
    E = len(edges) - 1
    g = torch.Generator(device=DEV).manual_seed(seed)

    def make(*shape):
        if real:
            return torch.randn(shape, device=DEV, generator=g).bfloat16()
        return torch.randint(-3, 4, shape, device=DEV, generator=g).bfloat16()
    return {"X": make(T, K), "dY": make(T, N), "W": make(E, K, N) if kn else make(E, N, K),
            "offsets": torch.tensor(edges, dtype=torch.int32, device=DEV)}


def reference(op, c, edges, kn, mag=False):
    """In 64 bits; mag: the sums of magnitudes."""
    f = (lambda t: t.double().abs()) if mag else (lambda t: t.double())
    E = len(edges) - 1
    rows = c["X"] if op == "fwd" else c["dY"]
    W = c["W"].transpose(1, 2) if kn else c["W"]
    if op == "wgrad":
        out = torch.zeros_like(W, dtype=torch.float64)
    else:
        out = torch.zeros(rows.shape[0], W.shape[1] if op == "fwd" else W.shape[2], dtype=torch.float64, device=DEV)
    for e in range(E):
        s = slice(int(edges[e]), int(edges[e + 1]))
        if op == "wgrad":
            out[e] = f(c["dY"][s]).T @ f(c["X"][s])
        else:
            w = f(W[e])
            out[s] = f(rows[s]) @ (w.T if op == "fwd" else w)
    return out.transpose(1, 2) if op == "wgrad" and kn else out


def call(op, c, kn=False, **kw):
    lay = "kn" if kn else "nk"
    if op == "fwd":
        return dp.dp_gemm_fwd_grouped(c["X"], c["W"], c["offsets"], weight_layout=lay, **kw)
    if op == "dgrad":
        return dp.dp_gemm_dgrad_grouped(c["dY"], c["W"], c["offsets"], weight_layout=lay, **kw)
    return dp.dp_gemm_wgrad_grouped(c["dY"], c["X"], c["offsets"], weight_layout=lay, **kw)


GROUPS = {
    "one_row": (0, [1], 0),
    "one_row_of_many": (0, [0, 0, 1, 0], 0),
    "ragged": (0, [5, 0, 129, 64, 1, 300, 0, 127], 0),
    "padded": (7, [33, 128, 0, 65], 200),
    "all_empty": (10, [0, 0, 0], 3),
    "whole_tiles": (0, [128, 256, 128], 0),
    "tails": (0, [15, 16, 17, 31, 47, 48, 49, 63, 65, 66], 0),
    "many_experts": (3, [(7 * i) % 5 for i in range(385)], 1),
    "most_experts": (0, [i % 3 for i in range(1024)], 0),
}


@pytest.mark.parametrize("groups", sorted(GROUPS))
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("kn", [False, True])
def test_integers_are_exact(op, groups, kn):
    front, counts, back = GROUPS[groups]
    edges = edges_of(counts, front)
    T = int(edges[-1]) + back
    for N, K in ((72, 136), (8, 8), (264, 64)) if len(counts) < 100 else ((40, 72),):
        c = tensors(edges, T, N, K, seed=len(counts) + N, kn=kn)
        for f32 in (False, True):
            got = call(op, c, kn, out_dtype=torch.float32 if f32 else torch.bfloat16)
            ref = reference(op, c, edges, kn)
            assert torch.equal(got, ref.float() if f32 else ref.to(torch.bfloat16)), (N, K, f32)
    assert dp.device_error() == 0


@pytest.mark.parametrize("counts,front,back", [([300, 0, 517, 256, 1, 900, 128, 700], 3, 250), ([4100], 0, 0), ([255, 257, 2000], 5, 1)])
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("kn", [False, True])
def test_integers_are_exact_on_many_tiles(op, kn, counts, front, back):
    """Sizes whose tiles fill the device: two SMs share a tile of 256 rows."""
    edges = edges_of(counts, front)
    T = int(edges[-1]) + back
    for N, K in ((2600, 2056), (2056, 2568)):
        c = tensors(edges, T, N, K, seed=T, kn=kn)
        ref = reference(op, c, edges, kn)
        assert torch.equal(call(op, c, kn, out_dtype=torch.float32), ref.float())
        assert torch.equal(call(op, c, kn), ref.to(torch.bfloat16))
    assert dp.device_error() == 0


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("T,E,N,K", [(1, 8, 256, 512), (64, 64, 1024, 512), (700, 4, 520, 4104), (2500, 3, 264, 2056),
                                     (5000, 1, 128, 136), (4031, 32, 1024, 512)])
def test_real_values(op, T, E, N, K):
    g = np.random.default_rng(T + E)
    counts = np.bincount(g.choice(E, T, p=g.dirichlet(np.ones(E))), minlength=E)
    edges = edges_of(counts)
    c = tensors(edges, T, N, K, seed=T, real=True)
    depth = {"fwd": K, "dgrad": N, "wgrad": int(counts.max())}[op]
    ref, mag = reference(op, c, edges, False), reference(op, c, edges, False, mag=True)
    tol = 4 * (min(depth, 2048) / 16 + depth / 2048 + 2) * 2.0 ** -23 * mag
    got = call(op, c, out_dtype=torch.float32)
    assert bool(((got.double() - ref).abs() <= tol).all())
    got = call(op, c)
    assert bool(((got.double() - ref).abs() <= tol + 2.0 ** -8 * ref.abs()).all())


@pytest.mark.parametrize("op", OPS)
def test_strided_views_and_int64_offsets(op):
    """Column slices of wider buffers, a slice of the experts, an output inside a buffer."""
    edges = edges_of([30, 0, 141, 70], 2)
    T, N, K, E = int(edges[-1]) + 5, 72, 136, 4
    c = tensors(edges, T, N, K, seed=3)
    wide = {"X": torch.full((T, K + 24), float("nan"), device=DEV).bfloat16(),
            "dY": torch.full((T, N + 8), float("nan"), device=DEV).bfloat16(),
            "W": torch.full((2 * E, N + 3, K + 16), float("nan"), device=DEV).bfloat16()}
    wide["X"][:, 8:8 + K] = c["X"]
    wide["dY"][:, 8:] = c["dY"]
    wide["W"][::2, :N, 16:] = c["W"]
    v = {"X": wide["X"][:, 8:8 + K], "dY": wide["dY"][:, 8:], "W": wide["W"][::2, :N, 16:], "offsets": c["offsets"].long()}
    ref = reference(op, c, edges, False)
    big = torch.full((*ref.shape[:-1], ref.shape[-1] + 16), 7.0, device=DEV)
    out = big[..., 8:8 + ref.shape[-1]]
    got = call(op, v, out=out)
    assert got is out and torch.equal(got, ref.float())
    assert bool((big[..., :8] == 7).all()) and bool((big[..., 8 + ref.shape[-1]:] == 7).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3.4e38])
@pytest.mark.parametrize("op", OPS)
def test_values_outside_a_group_reach_nothing(op, bad):
    """Padding rows, and another expert's rows next door, hold NaN, infinities or the lowest value."""
    edges = edges_of([37, 21, 0, 90], 11)
    T, N, K = int(edges[-1]) + 60, 136, 72
    c = tensors(edges, T, N, K, seed=9)
    clean = reference(op, c, edges, False)
    dirty = {k: v.clone() for k, v in c.items()}
    for k in ("X", "dY"):
        dirty[k][:11] = bad
        dirty[k][edges[-1]:] = bad
        dirty[k][edges[1]:edges[2]] = bad  # expert 1's rows
    got = call(op, dirty, out_dtype=torch.float32)
    if op == "wgrad":
        keep = [0, 2, 3]
        assert torch.equal(got[keep], clean[keep].float())
    else:
        keep = torch.ones(T, dtype=torch.bool, device=DEV)
        keep[edges[1]:edges[2]] = False
        assert torch.equal(got[keep], clean[keep].float())


@pytest.mark.parametrize("op", OPS)
def test_wrong_offsets_are_clamped_and_reported(op):
    """Offsets that decrease or leave [0, T] act as their running maximum within [0, T]."""
    T, N, K = 200, 72, 64
    dp.device_error()
    for raw in ([0, 90, 40, 260, 150], [-5, 20, 20, 120, 2 ** 31 - 1], [300, 0, 0, 0, 0]):
        fixed = np.maximum.accumulate(np.clip(raw, 0, T))
        c = tensors(np.array(raw), T, N, K, seed=4)
        ref = reference(op, c, fixed, False)
        assert torch.equal(call(op, c, out_dtype=torch.float32), ref.float()), raw
        assert dp.device_error() == 1
        assert dp.device_error() == 0
    c["offsets"] = torch.tensor([0, 2 ** 40, -2 ** 40, 50, 2 ** 62], device=DEV)
    ref = reference(op, c, np.array([0, T, T, T, T]), False)
    assert torch.equal(call(op, c, out_dtype=torch.float32), ref.float())
    assert dp.device_error() == 1


@pytest.mark.parametrize("op", OPS)
def test_no_rows(op):
    c = tensors(np.zeros(4, np.int64), 0, 72, 64, seed=1)
    out = call(op, c, out_dtype=torch.float32)
    assert out.numel() == 0 or bool((out == 0).all())
    c = tensors(np.array([0]), 50, 72, 64, seed=1)  # no experts at all: every row is padding
    if op != "wgrad":
        assert bool((call(op, c) == 0).all())
    else:
        assert call(op, c).shape == (0, 72, 64)


@pytest.mark.parametrize("op", OPS)
def test_graph_replay_follows_the_offsets(op):
    """One captured call serves any distribution: the host never reads the offsets.  Repeated
    calls give the same bits."""
    T, N, K, E = 600, 136, 264, 6
    c = tensors(edges_of([100] * E), T, N, K, seed=2, real=True)
    call(op, c, out_dtype=torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out = call(op, c, out_dtype=torch.float32)
    for counts in ([600, 0, 0, 0, 0, 0], [1, 2, 3, 4, 5, 400], [0, 0, 0, 0, 0, 0]):
        c["offsets"].copy_(torch.tensor(edges_of(counts), dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        first = out.clone()
        assert torch.equal(call(op, c, out_dtype=torch.float32), first)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)


def test_gradients_against_differences():
    """L = sum(Y G) is linear in X and in W: with integers its differences are exact."""
    edges = edges_of([40, 0, 77, 3])
    c = tensors(edges, 120, 72, 64, seed=5)
    c["dY"] = torch.randint(-2, 3, (120, 72), device=DEV).bfloat16()

    def loss(x, w):
        return float((dp.dp_gemm_fwd_grouped(x, w, c["offsets"], out_dtype=torch.float32).double() * c["dY"].double()).sum())
    dX, dW = call("dgrad", c, out_dtype=torch.float32).double(), call("wgrad", c, out_dtype=torch.float32).double()
    for seed in range(4):
        g = torch.Generator(device=DEV).manual_seed(seed)
        ux = torch.randint(-1, 2, c["X"].shape, device=DEV, generator=g).bfloat16()
        uw = torch.randint(-1, 2, c["W"].shape, device=DEV, generator=g).bfloat16()
        assert (loss(c["X"] + ux, c["W"]) - loss(c["X"] - ux, c["W"])) / 2 == float((dX * ux.double()).sum())
        assert (loss(c["X"], c["W"] + uw) - loss(c["X"], c["W"] - uw)) / 2 == float((dW * uw.double()).sum())


def test_call_on_another_stream():
    edges = edges_of([100, 300, 50])
    c = tensors(edges, 450, 264, 520, seed=6)
    ref = reference("fwd", c, edges, False).float()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [call("fwd", c, out_dtype=torch.float32, stream=side) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, ref) for x in got)


def test_output_beyond_32_bit_offsets():
    """More than 2^31 output elements: the last rows lie where they belong."""
    T, N, K = 140_000, 16_384, 64
    edges = edges_of([T // 2, T - T // 2 - 3])
    c = tensors(edges, T, 8, K, seed=7)
    c["W"] = torch.randint(-3, 4, (2, N, K), device=DEV).bfloat16()
    out = call("fwd", c)
    for s in (slice(0, 130), slice(T // 2 - 70, T // 2), slice(T - 140, T - 3)):
        e = 0 if s.start < T // 2 else 1
        assert torch.equal(out[s], (c["X"][s].double() @ c["W"][e].double().T).to(torch.bfloat16))
    assert bool((out[T - 3:] == 0).all())


@pytest.mark.parametrize("depth", [64, 512, 2048, 16384])
def test_error_does_not_grow_with_the_contraction(depth):
    """FP32 outputs: the tensor core's sums over 16384 elements are 1.9e-5 off, so over 512 elements
    6e-7; up to 32 such sums added in FP32 give 2e-7 more."""
    g = torch.Generator(device=DEV).manual_seed(depth)
    X = torch.randn(96, depth, device=DEV, generator=g).bfloat16()
    W = torch.randn(3, 128, depth, device=DEV, generator=g).bfloat16()
    offsets = torch.tensor([0, 40, 40, 96], device=DEV, dtype=torch.int32)
    D = torch.randn(depth, 96, device=DEV, generator=g).bfloat16()
    Z = torch.randn(depth, 128, device=DEV, generator=g).bfloat16()

    def error(got, want):
        return float((got.double() - want).norm() / want.norm())
    want = torch.cat([X[:40].double() @ W[0].double().T, X[40:].double() @ W[2].double().T])
    assert error(dp.dp_gemm_fwd_grouped(X, W, offsets, out_dtype=torch.float32), want) < 8e-7
    one = torch.tensor([0, depth], device=DEV, dtype=torch.int32)
    assert error(dp.dp_gemm_wgrad_grouped(D, Z, one, out_dtype=torch.float32)[0], D.double().T @ Z.double()) < 8e-7
