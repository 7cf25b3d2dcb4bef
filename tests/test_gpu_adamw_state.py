"""AdamW's tensors between steps: what a replaced .data may be."""
import numpy as np
import pytest
import torch

import fp32_dense_projection_gb300 as dp
from gpu_common import DEV

pytestmark = pytest.mark.gpu


def make(n=64, **kw):
    p = torch.randn(n, n, device=DEV)
    opt = dp.AdamW([p], copies=[torch.empty_like(p, dtype=torch.bfloat16)], **kw)
    return p, opt, [torch.randn(n, n, device=DEV)]


def bits(x):
    return x.contiguous().view(torch.uint8)


def refused(opt, g, match):
    before = [x.clone() for x in opt.params + opt.exp_avg]
    with pytest.raises((ValueError, TypeError), match=match):
        opt.step(g)
    assert all(torch.equal(bits(x), bits(y)) for x, y in zip(before, opt.params + opt.exp_avg))


def test_another_view_at_the_same_address_is_refused():
    p, opt, g = make()
    opt.step(g)
    good = p.data
    for bad in (good.t(), good[:32], good.view(-1)[:64 * 32].view(32, 64), good[:, :32]):
        assert bad.data_ptr() == good.data_ptr()
        p.data = bad
        refused(opt, g, "params")
    p.data = good
    for x in (opt.copies[0], opt.exp_avg[0], opt.exp_avg_sq[0]):
        good = x.data
        x.data = good.t()
        refused(opt, g, "contiguous")
        x.data = good
    opt.step(g)


def test_another_type_at_the_same_address_is_entered_or_refused():
    """BF16 in the first half of the FP32 parameter's memory: the second half stays as it was."""
    p, opt, g = make()
    opt.step(g)
    whole = p.data
    half = whole.view(torch.bfloat16).view(-1)[:64 * 64].view(64, 64)
    assert half.data_ptr() == whole.data_ptr()
    rest = whole.view(-1)[64 * 32:].clone()
    p.data = half
    opt.step(g)
    assert torch.equal(whole.view(-1)[64 * 32:], rest) and p.dtype == torch.bfloat16
    assert torch.equal(bits(opt.copies[0]), bits(p))  # (bits: FP32 halves read as BF16 hold NaN)
    m = opt.exp_avg[0].data
    opt.exp_avg[0].data = m.view(torch.int32)
    refused(opt, g, "exp_avg")
    opt.exp_avg[0].data = m


def test_a_refused_step_enters_nothing():
    """The parameter moves and the moment becomes unfit: refused.  With the moment fit and the parameter back in its old
    place, the step writes there and not to the place seen by the refused one."""
    p, opt, g = make()
    ref, twin, _ = make()
    ref.copy_(p)
    opt.step(g)
    twin.step(g)
    old, moved, m = p.data, p.data.clone(), opt.exp_avg_sq[0].data
    p.data, opt.exp_avg_sq[0].data = moved, m[:32].clone()
    seen = moved.clone()
    with pytest.raises(ValueError, match="exp_avg_sq"):
        opt.step(g)
    p.data, opt.exp_avg_sq[0].data = old, m
    opt.step(g)
    twin.step(g)
    assert torch.equal(moved, seen) and torch.equal(p, ref) and opt.step_count == 2


def test_capture_is_refused():
    """A replay would repeat one step's bias corrections; the refusal leaves the count, and the stream usable."""
    p, opt, g = make()
    opt.step(g)
    before = p.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        g[0].mul_(1.0)
        with pytest.raises(RuntimeError, match="captured"):
            opt.step(g)
        with pytest.raises(RuntimeError, match="captured"):
            opt.step(g, stream=side)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(p, before) and opt.step_count == 1
    opt.step(g)
    assert opt.step_count == 2 and not torch.equal(p, before)


@pytest.mark.parametrize("state_bits", [32, 8])
def test_a_parameter_that_missed_steps_has_its_own_corrections(state_bits):
    """Without a gradient a parameter makes no step: alone in an optimizer of its own, called only when it has a
    gradient, it gets the same bits.  The same after a resume from ``steps``."""
    kw = dict(lr=1e-2, betas=(0.9, 0.999), state_bits=state_bits)
    gen = torch.Generator(device=DEV).manual_seed(6)
    start = [torch.randn(s, device=DEV, generator=gen) for s in (300, 2048, 77)]
    has = [(1, 0, 1), (1, 1, 0), (0, 0, 0), (1, 1, 1), (0, 1, 1), (1, 1, 1)]
    opt = dp.AdamW([x.clone() for x in start], **kw)
    own = [dp.AdamW([x.clone()], **kw) for x in start]
    for n, row in enumerate(has):
        grads = [torch.randn(x.shape, device=DEV, generator=gen) for x in start]
        opt.step([g if h else None for g, h in zip(grads, row)])
        for o, g, h in zip(own, grads, row):
            if h:
                o.step([g])
        if n == 3:
            opt = dp.AdamW(opt.params, step=opt.steps, exp_avg=opt.exp_avg, exp_avg_sq=opt.exp_avg_sq, exp_avg_scale=opt.exp_avg_scale,
                           exp_avg_sq_scale=opt.exp_avg_sq_scale, **kw)
    assert opt.steps == (4, 4, 4) and tuple(o.step_count for o in own) == (4, 4, 4)
    for i, o in enumerate(own):
        assert torch.equal(opt.params[i], o.params[0]) and torch.equal(bits(opt.exp_avg_sq[i]), bits(o.exp_avg_sq[0]))
    with pytest.raises(ValueError, match="per parameter"):
        dp.AdamW(opt.params, step=(1, 2), **kw)
    with pytest.raises(ValueError, match="negative"):
        dp.AdamW(opt.params, step=(1, -2, 0), **kw)


def test_autograd_notices_the_update():
    """A backward pass through a parameter or a copy saved before the step is refused, as for other in-place
    updates; one through a tensor that the step left alone is not.  Inference tensors have no version and are updated too."""
    p, opt, g = make()
    q = torch.randn(8, device=DEV)
    both = dp.AdamW([p, q])
    for saved, step, changed in ((p, lambda: opt.step(g), True), (opt.copies[0], lambda: opt.step(g), True),
                                 (p, lambda: both.step([g[0], None]), True), (q, lambda: both.step([g[0], None]), False)):
        x = torch.ones_like(saved, requires_grad=True)
        y = (x * saved).sum()
        step()
        if changed:
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                y.backward()
        else:
            y.backward()
    with torch.inference_mode():
        w = torch.ones(16, device=DEV)
    before = w.clone()
    dp.AdamW([w]).step([torch.ones(16, device=DEV)])
    assert bool((w < before).all())


@pytest.mark.parametrize("beta2", [0.95, 0.999])
def test_tiny_second_moments_beside_a_large_one(beta2):
    """One large gradient in each block among ones 1e-7 to 1e-12 of it and zeros: what is above zero is held as the
    smallest code at least, zeros as zero, bit for bit the FP32 formula's (nearest and stochastic codes agree there: the
    smallest code is a value of the grid)."""
    n, f, betas = 128 * 64, np.float32, (0.9, beta2)
    rng = np.random.default_rng(7)
    grad = (10.0 ** rng.uniform(-12, -7, n) * rng.choice([-1, 1], n)).astype(f)
    grad[rng.random(n) < 0.2] = 0
    grad[::128] = 1
    opt = dp.AdamW([torch.zeros(n, device=DEV)], betas=betas, state_bits=8)
    codes, scales = np.zeros(n, f), np.zeros(n // 128, f)
    for t in range(2):
        opt.step([torch.from_numpy(grad).to(DEV)])
        x, old = grad.reshape(-1, 128), codes.reshape(-1, 128) * scales[:, None]
        root = np.sqrt((old * old) * f(betas[1]) + (x * x) * f(1 - betas[1]))
        a = np.maximum(root.max(1), f(1e-30))
        y = root * ((f(1) / a) * f(448))[:, None]
        held = np.where(y > 0, np.maximum(y, f(2.0 ** -9)), y)
        # (at first they would round to zero; then they are the smallest code, decayed)
        assert ((0 < y) & (y < 2.0 ** (-9 if t else -10))).sum() > n // 2
        codes, scales = torch.from_numpy(held).to(torch.float8_e4m3fn).float().numpy().reshape(-1), a * (f(1) / f(448))
        got = opt.exp_avg_sq[0].view(torch.uint8).cpu().numpy()
        assert np.array_equal(opt.exp_avg_sq[0].float().cpu().numpy(), codes)
        assert np.array_equal(opt.exp_avg_sq_scale[0].cpu().numpy(), scales)
        assert (got[grad == 0] == 0).all() and (got[np.abs(grad) < 1e-6][grad[np.abs(grad) < 1e-6] != 0] == 1).all()
        assert bool(torch.isfinite(opt.params[0]).all())


def test_shared_memory_is_refused():
    """The same or overlapping memory twice would be updated by blocks that run beside each other."""
    w = torch.randn(4096, device=DEV)
    h = torch.zeros(4096, dtype=torch.bfloat16, device=DEV)
    m, v = torch.zeros_like(w), torch.zeros_like(w)
    for kw in (dict(params=[w, w]), dict(params=[w, w.view(64, 64)]), dict(params=[w[:3000], w[2999:]]), dict(params=[h[:64]], copies=[h[32:96]]),
               dict(params=[w], exp_avg=[m], exp_avg_sq=[m]), dict(params=[h, w], copies=[None, h]), dict(params=[w[:96], w[96:]], copies=[h[:96], h[90:4090]])):
        with pytest.raises(ValueError, match="share memory"):
            dp.AdamW(**kw)
    a, b = h.clone(), h.clone()  # a BF16 parameter may be its own copy
    for opt in (dp.AdamW([a], copies=[a]), dp.AdamW([b])):
        opt.step([w])
    assert torch.equal(a, b) and bool((a != 0).any())
    opt = dp.AdamW([w[:96], w[96:], w[:0]], copies=[h[:96], h[96:], None])  # neighbours in one buffer
    opt.step([torch.ones(96, device=DEV), torch.ones(4000, device=DEV), torch.ones(0, device=DEV)])
    opt.params[0].data = w[1:97]
    with pytest.raises(ValueError, match="share memory"):
        opt.step([torch.ones(96, device=DEV), torch.ones(4000, device=DEV), torch.ones(0, device=DEV)])


@pytest.mark.parametrize("state_bits", [32, 8])
def test_moments_that_were_looked_at_are_watched(state_bits):
    """Moments made by the optimizer are its own until someone reads the attribute; what is then put in their place is
    followed or refused.  The attributes cannot be set: the steps would not go by what was set."""
    p, opt, g = make(state_bits=state_bits)
    ref, twin, _ = make(state_bits=state_bits)
    ref.copy_(p)
    for _ in range(2):
        opt.step(g)
        twin.step(g)
    names = ["exp_avg", "exp_avg_sq"] + ["exp_avg_scale", "exp_avg_sq_scale"] * (state_bits == 8)
    for name in names:
        with pytest.raises(AttributeError):
            setattr(opt, name, getattr(opt, name))
        x = getattr(opt, name)[0]
        assert getattr(opt, name)[0] is x
        good = x.data
        x.data = good[:1]
        refused(opt, g, name)
        x.data, kept = good.clone(), good.clone()
        g = [torch.randn_like(p)]
        opt.step(g)
        twin.step(g)
        assert torch.equal(bits(good), bits(kept))
        assert not torch.equal(bits(x), bits(good)) and torch.equal(bits(x), bits(getattr(twin, name)[0])) and torch.equal(p, ref)
    assert (opt.exp_avg_scale is None) == (state_bits == 32)
