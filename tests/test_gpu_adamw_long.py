"""8-bit moments with a long memory: their codes are rounded stochastically, and follow the 32-bit moments.

Rounding a value between neighbouring codes a distance D apart, up with the probability p of its place between them, adds
nothing on average and at most p (1 - p) D^2 of variance.  A step at rate 1 - beta2 = 2 d moves sqrt(v) (and the
block's scale) by about d of itself each, so p D <= 2 d r and the variance is at most 2 d D r^2 a step; v's recurrence forgets
it at the rate 2 d: at most D r^2 in all, D <= 1/8 r.  sqrt(v) thus keeps a standard deviation of at most 36% (its mean
square at most 1/8 above v's, its mean within 6%).
"""
import numpy as np
import pytest
import torch

import fp32_dense_projection_gb300 as dp
from gpu_common import DEV
from test_gpu_adamw import decode

pytestmark = pytest.mark.gpu

N = 1 << 16
E4 = torch.float8_e4m3fn


def ratio(a, b, half):
    """Mean and deviation of the 8-bit optimizer's sqrt(v) over the 32-bit one's, on every other element."""
    r = decode(a.exp_avg_sq[0], a.exp_avg_sq_scale[0])[half::2] / b.exp_avg_sq[0].double().sqrt()[half::2]
    return float(r.mean()), float(r.std())


@pytest.mark.parametrize("beta2", [0.96, 0.98, 0.99, 0.999])
def test_second_moment_follows_falls_and_rises(beta2):
    """Stationary gradients, then a tenfold fall of the even elements' gradients, then a fivefold rise of the odd ones', six
    time constants each."""
    a = dp.AdamW([torch.zeros(N, device=DEV)], betas=(0.9, beta2), state_bits=8)
    b = dp.AdamW([torch.zeros(N, device=DEV)], betas=(0.9, beta2), state_bits=32)
    g = torch.Generator(device=DEV).manual_seed(1)
    size = torch.ones(N, device=DEV)
    for phase in range(3):
        if phase == 1:
            size[::2] = 0.1
        if phase == 2:
            size[1::2] = 5.0
        for _ in range(round(6 / (1 - beta2))):
            grad = [torch.randn(N, device=DEV, generator=g) * size]
            a.step(grad)
            b.step(grad)
        for half in (0, 1):
            mean, std = ratio(a, b, half)
            assert abs(mean - 1) <= 0.06 and std <= 0.36, (phase, half, mean, std)


def test_first_moment_follows():
    """beta1 = 0.999: the mean of m over 32-bit m's sign stays the 32-bit m's; its codes do not freeze.  D r^2 of variance as for
    sqrt(v), with a step of 2 d: averaged over 65536 elements of |m| about 0.3 the slope is within 2%."""
    a = dp.AdamW([torch.zeros(N, device=DEV)], betas=(0.999, 0.95), state_bits=8)
    b = dp.AdamW([torch.zeros(N, device=DEV)], betas=(0.999, 0.95), state_bits=32)
    g = torch.Generator(device=DEV).manual_seed(2)
    mean = 0.3 * torch.sin(torch.arange(N, device=DEV).float())
    for _ in range(6000):
        grad = [mean + torch.randn(N, device=DEV, generator=g)]
        a.step(grad)
        b.step(grad)
    m8, m32 = decode(a.exp_avg[0], a.exp_avg_scale[0]), b.exp_avg[0].double()
    assert abs(float((m8 * m32).sum() / (m32 * m32).sum()) - 1) <= 0.02


def neighbours(y):
    """E4M3's values at and above |y| (on a code: that code twice), y in [0, 448]."""
    exponent = np.floor(np.log2(np.maximum(y, 2.0 ** -6)))
    d = np.exp2(exponent - 3)
    return np.floor(y / d) * d, np.ceil(y / d) * d, d


@pytest.mark.parametrize("which", ["v", "m"])
def test_codes_are_neighbours_and_unbiased(which):
    """Each code is one of the two next to the FP32 formula's value, and the errors' mean is zero: n errors of at most
    half a step's deviation each have a mean within 5 / (2 sqrt(n)) steps."""
    n, betas = 1 << 20, (0.9, 0.999) if which == "v" else (0.99, 0.9)
    g = torch.Generator(device=DEV).manual_seed(3)
    grad = torch.randn(n, device=DEV, generator=g)
    p = torch.zeros(n, device=DEV)
    opt = dp.AdamW([p], betas=betas, state_bits=8)
    opt.step([grad])
    f = np.float32
    x = grad.cpu().numpy().reshape(-1, 128)
    y = np.sqrt((x * x) * f(1 - betas[1])) if which == "v" else x * f(1 - betas[0])
    a = np.maximum(np.abs(y).max(1), f(1e-30))
    want = (y * ((f(1) / a) * f(448))[:, None]).astype(np.float64).reshape(-1)
    got = (opt.exp_avg_sq if which == "v" else opt.exp_avg)[0].float().cpu().numpy().astype(np.float64)
    assert (np.sign(got) * np.sign(want) >= 0).all()
    got, want = np.abs(got), np.minimum(np.abs(want), 448.0)
    lo, hi, d = neighbours(want)
    assert ((got == lo) | (got == hi) | ((want > 0) & (want < 2.0 ** -9) & (got == 2.0 ** -9))).all()
    inner = want >= 2.0 ** -9
    assert abs(((got - want) / d)[inner].mean()) <= 5 / (2 * inner.sum() ** 0.5)
    assert ((got == lo) & (lo < hi)).sum() > n // 4 and ((got == hi) & (lo < hi)).sum() > n // 4


def test_runs_repeat_and_resume_bit_for_bit():
    """Two runs, one of them stopped and taken up again from its state, in tables of different lengths and at odd addresses."""
    sizes = [5000, 129, 2048, 1]
    g = torch.Generator(device=DEV).manual_seed(4)
    start = [torch.randn(s, device=DEV, generator=g) for s in sizes]
    grads = [[torch.randn(s, device=DEV, generator=g) for s in sizes] for _ in range(6)]
    kw = dict(betas=(0.99, 0.999), state_bits=8)
    a = dp.AdamW([x.clone() for x in start], **kw)
    for x in grads:
        a.step(x)
    odd = [torch.zeros(s + 3, device=DEV) for s in sizes]
    for o, x in zip(odd, start):
        o[3:] = x
    b = dp.AdamW([o[3:] for o in odd], **kw)
    for x in grads[:3]:
        b.step(x)
    more = [torch.zeros(1, device=DEV) for _ in range(30)]
    c = dp.AdamW([*more, *b.params], step=3, exp_avg=[*(x.to(E4) for x in more), *b.exp_avg], exp_avg_scale=[*(x.clone() for x in more), *b.exp_avg_scale],
                 exp_avg_sq=[*(x.to(E4) for x in more), *b.exp_avg_sq], exp_avg_sq_scale=[*(x.clone() for x in more), *b.exp_avg_sq_scale], **kw)
    for x in grads[3:]:
        c.step([*(None for _ in more), *x])
    for u, v in ((a.params, c.params[30:]), (a.exp_avg, c.exp_avg[30:]), (a.exp_avg_sq, c.exp_avg_sq[30:]), (a.exp_avg_scale, c.exp_avg_scale[30:])):
        assert all(torch.equal(x.float(), y.float()) for x, y in zip(u, v))
