"""The operators of a layer of experts as they are used together: a decoding step on 4-bit weights and a training step
behind a layer norm, against 64-bit forms with the same choice of experts (and, for gradients, the same signs in front
of relu: its derivative jumps there, so that a sign that a rounding turns moves a gradient by all of itself).

Each BF16 value between the operators is off by half a step, 2^-8 of itself; errors of independent roundings add up in
the sums like their squares, so in norm an output is off by about 2^-8 times the root of the number of
roundings on its way (each at most 2^-8, on average 2^-8 / sqrt(3) of the value): with up to 5 roundings, 5 2^-8 bounds it."""
import pytest
import torch

import fp32_dense_projection_gb300 as dp
from gpu_common import DEV

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
TOL = 5 * 2.0 ** -8


def normal(shape, seed, scale=1.0, dtype=BF16):
    return (torch.randn(shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed)) * scale).to(dtype)


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


class Layer:
    def __init__(self, C=256, inner=384, E=16, k=4):
        self.C, self.E, self.k = C, E, k
        self.gamma, self.beta = normal((C,), 1, 0.2, F32) + 1, normal((C,), 2, 0.1, F32)
        self.router = normal((E, C), 3, C ** -0.5, F32)
        self.w1, self.w2 = normal((E, inner, C), 4, C ** -0.5), normal((E, C, inner), 5, inner ** -0.5)
        self.q1, self.q2 = dp.int4_quantize(self.w1, 64, zeros=True), dp.int4_quantize(self.w2, 128)

    def serve(self, x, closed=None):
        h, _, _ = dp.layer_norm_fwd(x, self.gamma, self.beta)
        logits = dp.router_fwd(h.float(), self.router)
        if closed is not None:
            logits = logits.masked_fill(closed, float("-inf"))
        gates, choice = dp.route_topk(logits, self.k)
        offsets, row_of, _ = dp.expert_sort(choice, self.E)
        a = dp.dp_gemm_fwd_int4_grouped(dp.expert_gather(h, row_of), *self.q1[:2], offsets, zeros=self.q1[2]).relu()
        y = dp.dp_gemm_fwd_int4_grouped(a, *self.q2[:2], offsets, zeros=self.q2[2])
        return dp.expert_combine(y, row_of, gates, add=x), choice

    def plain(self, x, choice, w1, w2, gamma, beta, router, signs=None):
        """In 64 bits, the choice (and the signs [T, k, inner]) given: (T, C)."""
        d = x - x.mean(1, keepdim=True)
        h = d / (d.square().mean(1, keepdim=True) + 1e-5).sqrt() * gamma + beta
        live = choice >= 0
        at = choice.long().clamp_min(0)
        logits = (h @ router.T).gather(1, at).masked_fill(~live, float("-inf"))
        gates = torch.where(live.any(1, keepdim=True), logits.softmax(1), 0.0).nan_to_num(0.0)
        out = x
        for j in range(choice.shape[1]):
            a = torch.einsum("tc,tnc->tn", h, w1[at[:, j]])
            a = a.relu() if signs is None else a * signs[:, j]
            out = out + gates[:, j:j + 1] * torch.einsum("tn,tcn->tc", a, w2[at[:, j]])
        return out


@pytest.fixture(scope="module")
def layer():
    return Layer()


@pytest.mark.parametrize("T", [1, 5, 40])
def test_serving_with_4_bit_weights(layer, T):
    x = normal((T, layer.C), T)
    closed = torch.zeros(T, layer.E, dtype=torch.bool, device=DEV)
    closed[:, 3] = True   # an expert that is down
    if T > 1:
        closed[T - 1] = True  # a padding token
    out, choice = layer.serve(x, closed)
    w1, w2 = (dp.int4_dequantize(*q[:2], zeros=q[2], out_dtype=F32).double() for q in (layer.q1, layer.q2))
    want = layer.plain(x.double(), choice, w1, w2, layer.gamma.double(), layer.beta.double(), layer.router.double())
    assert bool((choice != 3).all()) and off(out, want) <= TOL
    if T > 1:
        assert bool((choice[-1] == -1).all()) and torch.equal(out[-1], x[-1])
    assert dp.device_error() == 0


def test_serving_in_a_graph_follows_its_input(layer):
    """Captured once, replayed on other tokens: nothing of the routing is fixed by the capture."""
    x = normal((8, layer.C), 1)
    layer.serve(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, choice = layer.serve(x)
    for seed in (2, 3):
        x.copy_(normal((8, layer.C), seed))
        g.replay()
        want, at = layer.serve(x)
        assert torch.equal(choice, at) and torch.equal(out, want)


@pytest.mark.parametrize("T", [3, 700])
def test_training_behind_a_layer_norm(layer, T):
    """Gradients of input, norm, router and experts against autograd in 64 bits."""
    x, d_out = normal((T, layer.C), T), normal((T, layer.C), T + 1, 0.1)
    h, mean, rstd = dp.layer_norm_fwd(x, layer.gamma, layer.beta)
    h32 = h.float()
    logits = dp.router_fwd(h32, layer.router)
    gates, choice = dp.route_topk(logits, layer.k)
    offsets, row_of, _ = dp.expert_sort(choice, layer.E)
    rows = dp.expert_gather(h, row_of)
    pre = dp.dp_gemm_fwd_grouped(rows, layer.w1, offsets)
    a = pre.relu()
    y = dp.dp_gemm_fwd_grouped(a, layer.w2, offsets)
    out = dp.expert_combine(y, row_of, gates, add=x)

    d_y, d_gates = dp.expert_combine_bwd(d_out, y, row_of, gates)
    d_w2 = dp.dp_gemm_wgrad_grouped(d_y, a, offsets, out_dtype=F32)
    d_pre = dp.dp_gemm_dgrad_grouped(d_y, layer.w2, offsets) * (pre > 0)
    d_w1 = dp.dp_gemm_wgrad_grouped(d_pre, rows, offsets, out_dtype=F32)
    d_logits = dp.route_topk_bwd(d_gates, logits, gates, choice)
    d_router = dp.router_wgrad(d_logits, h32)
    d_h = dp.expert_combine(dp.dp_gemm_dgrad_grouped(d_pre, layer.w1, offsets), row_of, add=dp.router_dgrad(d_logits, layer.router), out_dtype=F32)
    d_x, d_gamma, d_beta = dp.layer_norm_bwd(d_h, x, mean, rstd, layer.gamma, dx_dtype=F32)
    d_x = d_x + d_out

    leaves = [t.double().requires_grad_() for t in (x, layer.w1, layer.w2, layer.gamma, layer.beta, layer.router)]
    want = layer.plain(leaves[0], choice, *leaves[1:], signs=(pre > 0)[row_of.long()].double())
    grads = torch.autograd.grad(want, leaves, d_out.double())
    assert off(out, want.detach()) <= TOL
    for got, ref in zip((d_x, d_w1, d_w2, d_gamma, d_beta, d_router), grads):
        assert off(got, ref) <= TOL
    assert dp.device_error() == 0


@pytest.mark.parametrize("T", [8, 700])
def test_calls_one_after_another_share_buffers(T):
    """Launches that begin while the ones before them end: many steps through the same buffers give what steps
    with a pause after each call give, bit for bit."""
    E, k, C, steps = 64, 4, 1024, 40
    g = torch.Generator(device=DEV).manual_seed(T)
    logits = torch.randn(steps, T, E, device=DEV, generator=g)
    x = torch.randn(steps, T, C, device=DEV, generator=g).bfloat16()
    rows = torch.empty(T * k, C, device=DEV, dtype=torch.bfloat16)
    d_rows = torch.empty_like(rows)

    def run(pause):
        outs = torch.empty(steps, T, C, device=DEV, dtype=torch.bfloat16)
        d_logits = torch.empty(steps, T, E, device=DEV)
        for i in range(steps):
            for call in (lambda: state.update(zip(("gates", "choice"), dp.route_topk(logits[i], k))),
                         lambda: state.update(row_of=dp.expert_sort(state["choice"], E)[1]),
                         lambda: dp.expert_gather(x[i], state["row_of"], out=rows),
                         lambda: dp.expert_combine(rows, state["row_of"], state["gates"], out=outs[i]),
                         lambda: state.update(d_gates=dp.expert_combine_bwd(outs[i], rows, state["row_of"], state["gates"], d_y=d_rows)[1]),
                         lambda: dp.route_topk_bwd(state["d_gates"], logits[i], state["gates"], state["choice"], out=d_logits[i])):
                call()
                if pause:
                    torch.cuda.synchronize()
        return outs, d_logits

    state = {}
    want = run(True)
    for _ in range(3):
        got = run(False)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert dp.device_error() == 0


def test_capture_on_two_streams():
    """A graph that forks behind the sort, with torch's kernels and fills between the calls, follows its inputs."""
    T, E, k, C = 300, 32, 2, 512
    logits, x = normal((T, E), 1, 1.0, F32), normal((T, C), 2)
    side = torch.cuda.Stream()

    def work(fork):
        gates, choice = dp.route_topk(logits, k)
        _, row_of, _ = dp.expert_sort(choice, E)
        halved = x * 0.5
        main = torch.cuda.current_stream()
        other = side if fork else main
        other.wait_stream(main)
        with torch.cuda.stream(other):
            rows = dp.expert_gather(halved, row_of)
            first = dp.expert_combine(rows, row_of, gates, out_dtype=F32)
        mine = dp.expert_gather(x, row_of, out=torch.zeros(T * k, C, device=DEV, dtype=BF16))
        second = dp.expert_combine(mine, row_of, None, add=torch.zeros(T, C, device=DEV), out_dtype=F32)
        main.wait_stream(other)
        d = dp.route_topk_bwd(dp.expert_combine_bwd(first, mine, row_of, gates)[1], logits, gates, choice)
        return first + second, d

    work(True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work(True)
    for i in range(5):
        logits.copy_(normal((T, E), 10 + i, 1.0, F32))
        x.copy_(normal((T, C), 20 + i))
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        want = work(False)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert dp.device_error() == 0
