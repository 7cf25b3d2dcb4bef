"""AdamW over many tensors against the update in 64 bits.

32-bit moments: m and v take three roundings beside their constants' (5e-7 of the terms'
magnitudes covers them), p about eight more on |p| and on the update (1e-6).
8-bit moments: the decoded state is within half an E4M3 code of the 64-bit value of the same
old state: 2^-4 of it, or half (for v's root, which never becomes zero: one) smallest code;
the FP32 arithmetic before it adds 1e-6 of the block's largest value, 448 scales.
"""
import math

import numpy as np
import pytest
import torch

import fp32_dense_projection_gb300 as dp
from gpu_common import DEV

pytestmark = pytest.mark.gpu

H = dict(lr=2e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)


def make(sizes, seed, p_type, g_type):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(scale, dtype):
        return [(torch.randn(s, device=DEV, generator=g) * scale).to(dtype) for s in sizes]
    return normal(0.05, p_type), normal(1e-3, g_type), normal(3e-4, torch.float32), [x.square() for x in normal(1e-3, torch.float32)]


def update64(p, g, m, v, t, scale=1.0, lr=None):
    b1, b2 = H["betas"]
    lr = H["lr"] if lr is None else lr
    g = g.double() * scale
    m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    step = lr / (1 - b1 ** t) * m / (v.sqrt() / math.sqrt(1 - b2 ** t) + H["eps"])
    return p.double() * (1 - lr * H["weight_decay"]) - step, m, v, step


def decode(q, s):
    return (q.double().view(-1) * s.double().repeat_interleave(128)[:q.numel()]).view(q.shape)


def encode(x):
    flat = torch.nn.functional.pad(x.reshape(-1), (0, -x.numel() % 128)).view(-1, 128)
    a = flat.abs().amax(1).clamp_min(1e-30)
    return (flat * (448.0 / a)[:, None]).to(torch.float8_e4m3fn).view(-1)[:x.numel()].view(x.shape), a / 448.0


SIZES = {
    "one": [(1,)],
    "odd": [(7,), (1, 129), (64, 33), (2049,), (3,)],
    "aligned": [(128,), (4096,), (96, 128)],
    "empty_among": [(0,), (300,), (0, 4), (2048 * 3 + 5,)],
    "many": [(1 + 37 * i % 700,) for i in range(300)],
}


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", sorted(SIZES))
@pytest.mark.parametrize("p_type,g_type", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.bfloat16),
                                           (torch.float32, torch.float32), (torch.bfloat16, torch.float32)])
def test_two_steps(sizes, bits, p_type, g_type):
    p, g, m, v = make(SIZES[sizes], 1, p_type, g_type)
    copies = [torch.full_like(x, 9, dtype=torch.bfloat16) for x in p]
    state = dict(exp_avg=m, exp_avg_sq=v)
    if bits == 8:
        qm, qv = [encode(x) for x in m], [encode(x.sqrt()) for x in v]
        state = dict(exp_avg=[x[0] for x in qm], exp_avg_scale=[x[1] for x in qm],
                     exp_avg_sq=[x[0] for x in qv], exp_avg_sq_scale=[x[1] for x in qv])
    opt = dp.AdamW(p, state_bits=bits, copies=copies, step=3, **state, **H)
    for t in (4, 5):
        old = [x.clone() for x in p]
        if bits == 8:
            om = [decode(a, b) for a, b in zip(opt.exp_avg, opt.exp_avg_scale)]
            ov = [decode(a, b).square() for a, b in zip(opt.exp_avg_sq, opt.exp_avg_sq_scale)]
        else:
            om, ov = [x.double() for x in opt.exp_avg], [x.double() for x in opt.exp_avg_sq]
        opt.step(g, grad_scale=0.5)
        assert opt.step_count == t
        for i in range(len(p)):
            rp, rm, rv, step = update64(old[i], g[i], om[i], ov[i], t, 0.5)
            tol = 1e-6 * (rp.abs() + step.abs()) + (2.0 ** -8 * rp.abs() if p_type == torch.bfloat16 else 0)
            assert bool(((p[i].double() - rp).abs() <= tol).all())
            assert torch.equal(copies[i], p[i].to(torch.bfloat16))
            if bits == 32:
                assert bool(((opt.exp_avg[i].double() - rm).abs() <= 5e-7 * (om[i].abs() + g[i].double().abs())).all())
                assert bool(((opt.exp_avg_sq[i].double() - rv).abs() <= 5e-7 * rv).all())
            elif p[i].numel():
                for got, s, ref, least in ((opt.exp_avg[i], opt.exp_avg_scale[i], rm, 2.0 ** -10),
                                           (opt.exp_avg_sq[i], opt.exp_avg_sq_scale[i], rv.sqrt(), 2.0 ** -9)):
                    room = least * s.double().repeat_interleave(128)[:ref.numel()].view(ref.shape)
                    assert bool(((decode(got, s) - ref).abs() <= (2.0 ** -4 * ref.abs()).maximum(room) + 448e-6 * room / least).all())
                assert bool((opt.exp_avg_sq[i].float()[rv > 0] > 0).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_unaligned_views(bits):
    """Tensors at odd elements of a buffer: same values as aligned ones, neighbours untouched."""
    n = 5000
    p, g, _, _ = make([(n,)], 2, torch.float32, torch.bfloat16)
    a = dp.AdamW([p[0].clone()], state_bits=bits, **H)
    buf_p, buf_g = torch.full((n + 9,), 3.0, device=DEV), torch.full((n + 9,), 3.0, device=DEV).bfloat16()
    buf_c = torch.full((n + 9,), 3.0, device=DEV).bfloat16()
    buf_p[3:3 + n], buf_g[5:5 + n] = p[0], g[0]
    copy = buf_c[1:1 + n]
    b = dp.AdamW([buf_p[3:3 + n]], state_bits=bits, copies=[copy], **H)
    for _ in range(3):
        a.step(g)
        b.step([buf_g[5:5 + n]])
    assert torch.equal(a.params[0], b.params[0]) and torch.equal(copy, b.params[0].to(torch.bfloat16))
    assert torch.equal(a.exp_avg[0].float(), b.exp_avg[0].float()) and torch.equal(a.exp_avg_sq[0].float(), b.exp_avg_sq[0].float())
    assert bool((buf_p[:3] == 3).all()) and bool((buf_p[3 + n:] == 3).all())
    assert bool((buf_c[:1] == 3).all()) and bool((buf_c[1 + n:] == 3).all())


def test_skipped_gradients_rates_and_device_scale():
    p, g, _, _ = make([(500,), (60,), (4000,)], 3, torch.float32, torch.float32)
    start = [x.clone() for x in p]
    opt = dp.AdamW(p, **H)
    scale = torch.tensor([0.25], device=DEV)
    opt.step([g[0], None, g[2]], lr=5e-3, grad_scale=scale)
    zero = torch.zeros((), dtype=torch.float64, device=DEV)
    for i in (0, 2):
        rp, _, _, step = update64(start[i], g[i], zero, zero, 1, 0.25, lr=5e-3)
        assert bool(((p[i].double() - rp).abs() <= 1e-6 * (rp.abs() + step.abs())).all())
    assert torch.equal(p[1], start[1]) and bool((opt.exp_avg[1] == 0).all())
    opt.step([None, None, None])
    assert opt.step_count == 2


@pytest.mark.parametrize("bits", [32, 8])
def test_non_finite_gradients_show(bits):
    """A NaN or infinity marks its element, and in 8 bits its 128 elements' state; no other block."""
    p, g, _, _ = make([(1024,)], 4, torch.float32, torch.float32)
    g[0][130], g[0][700] = float("nan"), float("inf")
    opt = dp.AdamW(p, state_bits=bits, **H)
    opt.step(g)
    ok = torch.ones(1024, dtype=torch.bool, device=DEV)
    ok[130] = ok[700] = False
    assert bool(torch.isfinite(p[0][ok]).all()) and not bool(torch.isfinite(p[0][~ok]).any())
    if bits == 8:
        fine = [0, 2, 3, 4, 6, 7]
        assert bool(torch.isfinite(opt.exp_avg_scale[0][fine]).all()) and not bool(torch.isfinite(opt.exp_avg_scale[0][[1, 5]]).any())


def test_8_bit_moments_follow_32_bit_ones():
    """A noisy quadratic: both reach the same neighbourhood of the minimum."""
    target = torch.linspace(-1, 1, 4096, device=DEV)
    last = {}
    for bits in (32, 8):
        x = [torch.zeros(4096, device=DEV)]
        opt = dp.AdamW(x, lr=2e-2, betas=(0.9, 0.95), weight_decay=0.0, state_bits=bits)
        g = torch.Generator(device=DEV).manual_seed(0)
        for i in range(400):
            opt.step([(x[0] - target) + 0.05 * torch.randn(4096, device=DEV, generator=g)], lr=2e-2 * (1 - i / 400))
        last[bits] = float((x[0] - target).square().mean())
    assert last[32] < 1e-3 and last[8] < 1e-3


def test_streams_and_graph():
    p, g, _, _ = make([(3000,), (77,)], 5, torch.float32, torch.bfloat16)
    ref = [x.clone() for x in p]
    a, b = dp.AdamW(p, **H), dp.AdamW(ref, **H)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a.step(g, stream=side)
    b.step(g)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(p, ref))


def test_more_than_2_31_elements():
    n = 2 ** 31 + 300
    p = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    g[-200:] = 1.0
    opt = dp.AdamW([p], state_bits=8, lr=0.5, weight_decay=0.0)
    opt.step([g])
    assert bool((p[-200:] == -0.5).all()) and bool((p[-300:-200] == 0).all()) and bool((p[:1000] == 0).all())


@pytest.mark.parametrize("scale", [1.0, 0.3])
def test_8_bit_state_is_the_fp32_formulas_bit_for_bit(scale):
    """Every operation on the moments is rounded once: FP32 arithmetic elsewhere gives the same codes and scales."""
    n = 1 << 20
    p, g, m, v = make([(n,)], 6, torch.float32, torch.bfloat16)
    (qm, sm), (qv, sv) = encode(m[0]), encode(v[0].sqrt())
    f = np.float32
    state = [x.float().cpu().numpy() for x in (qm, sm, qv, sv)]
    opt = dp.AdamW(p, state_bits=8, exp_avg=[qm], exp_avg_scale=[sm], exp_avg_sq=[qv], exp_avg_sq_scale=[sv], **H)
    grad = g[0].float().cpu().numpy() * f(scale)
    (b1, b2), c1, c2 = H["betas"], f(1 - H["betas"][0]), f(1 - H["betas"][1])
    for _ in range(2):
        dm, dv = state[0].reshape(-1, 128) * state[1][:, None], state[2].reshape(-1, 128) * state[3][:, None]
        x = grad.reshape(-1, 128)
        nm = dm * f(b1) + x * c1
        root = np.sqrt((dv * dv) * f(b2) + (x * x) * c2)
        state = []
        for y, low in ((nm, None), (root, f(2.0 ** -9))):
            a = np.maximum(np.abs(y).max(1), f(1e-30))
            z = y * ((f(1) / a) * f(448))[:, None]
            z = z if low is None else np.where(y > 0, np.maximum(z, low), z)
            state += [torch.from_numpy(z).to(torch.float8_e4m3fn).float().numpy().reshape(-1), a * (f(1) / f(448))]
        opt.step(g, grad_scale=scale)
        for got, want in zip((opt.exp_avg, opt.exp_avg_scale, opt.exp_avg_sq, opt.exp_avg_sq_scale), state):
            assert np.array_equal(got[0].float().cpu().numpy().reshape(-1), want)


def test_tensors_that_move_between_steps():
    """Parameters, copies and moments may get new memory; of another shape it is refused."""
    (p,), (g,), _, _ = make([(64, 64)], 8, torch.float32, torch.bfloat16)
    ref = p.clone()
    copy = torch.empty_like(p, dtype=torch.bfloat16)
    a, b = dp.AdamW([p], copies=[copy], **H), dp.AdamW([ref], **H)
    a.step([g])
    b.step([g])
    moved = (p, copy, a.exp_avg[0], a.exp_avg_sq[0])
    kept, old = [x.clone() for x in moved], [x.data for x in moved]
    for x in moved:
        x.data = x.clone()
    a.step([g])
    b.step([g])
    assert torch.equal(p, ref) and torch.equal(copy, ref.bfloat16()) and torch.equal(a.exp_avg[0], b.exp_avg[0])
    assert all(torch.equal(x, y) for x, y in zip(old, kept))
    good = p.data
    for bad in (good[:32].clone(), good.clone().t()):
        p.data = bad
        with pytest.raises(ValueError, match="params"):
            a.step([g])
    p.data = good
    a.step([g])
    b.step([g])
    assert torch.equal(p, ref)
