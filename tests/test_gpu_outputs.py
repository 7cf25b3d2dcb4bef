"""Outputs that the bindings of the expert layer's operators make: what watches torch's own allocations sees them."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import fp32_dense_projection_gb300 as dp
from fp32_dense_projection_gb300 import _call
from gpu_common import DEV

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


class Seen(TorchDispatchMode):
    """The addresses of all tensors that torch makes under it."""

    def __init__(self):
        super().__init__()
        self.at = set()

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if isinstance(out, torch.Tensor):
            self.at.add(out.data_ptr())
        return out


def operators():
    """Each operator's outputs on small inputs."""
    x, w, l = torch.randn(6, 64, device=DEV, dtype=BF16), torch.ones(64, device=DEV), torch.randn(6, 8, device=DEV)
    W = torch.randn(8, 16, 64, device=DEV, dtype=BF16)
    dp.device_error()

    def run():
        y, mean, rstd = dp.layer_norm_fwd(x, w, w)
        grads = dp.layer_norm_bwd(x, x, mean, rstd, w)
        gates, choice = dp.route_topk(l, 2)
        d_l = dp.route_topk_bwd(gates, l, gates, choice)
        offsets, row_of, order = dp.expert_sort(choice, 8)
        rows = dp.expert_gather(x, row_of)
        q, s, z = dp.int4_quantize(W, 32, zeros=True)
        wide = dp.int4_dequantize(q, s, zeros=z)
        y4 = dp.dp_gemm_fwd_int4_grouped(rows, q, s, offsets, zeros=z)
        y1 = dp.dp_gemm_fwd_int4(x, q[0], s[0], zeros=z[0])
        out = dp.expert_combine(y4, row_of, gates)
        return (y, mean, rstd, *grads, gates, choice, d_l, offsets, row_of, order, rows, q, s, z, wide, y4, y1, out,
                *dp.expert_combine_bwd(out, y4, row_of, gates))
    return run


def test_dispatch_modes_see_the_outputs():
    run = operators()
    want = run()
    with Seen() as seen:
        got = run()
    for a, b in zip(got, want):
        assert a.data_ptr() in seen.at and torch.equal(a, b) and a.stride() == b.stride()


@pytest.fixture
def deterministic():
    before = torch.are_deterministic_algorithms_enabled(), torch.is_deterministic_algorithms_warn_only_enabled()
    torch.use_deterministic_algorithms(True)
    yield
    torch.use_deterministic_algorithms(before[0], warn_only=before[1])


def test_deterministic_algorithms_fill_what_is_not_written(deterministic):
    """A pair whose entry names no row leaves its place as it was made: NaN then, and not what the memory held."""
    x = torch.randn(4, 64, device=DEV)
    row_of = torch.arange(8, device=DEV, dtype=torch.int32).view(4, 2)
    row_of[1, 1] = 8  # (row 3 gets no pair)
    dp.device_error()
    for _ in range(3):
        rows = dp.expert_gather(x, row_of)
        d_y, _ = dp.expert_combine_bwd(x, rows.nan_to_num(), row_of, torch.ones(4, 2, device=DEV), dy_dtype=F32)
        assert rows[3].isnan().all() and d_y[3].isnan().all()
        keep = [0, 1, 2, 4, 5, 6, 7]
        assert torch.equal(rows[keep], x.repeat_interleave(2, 0)[keep]) and torch.equal(d_y[keep], rows[keep])
    assert dp.device_error() == 1


def test_without_the_shorter_way(monkeypatch):
    """Where torch has no such function, or another one under its name, tensors come from its public call."""
    def meta():
        return [(t.shape, t.dtype, t.stride(), t.device) for t in operators()()]
    want = meta()
    assert _call._direct is not _call._public or not hasattr(_call, "_found")
    for other in (None, lambda *a: torch.empty(3), lambda shape: None):
        assert _call._choose(other) is _call._public
    monkeypatch.setattr(_call, "_direct", _call._public)
    assert meta() == want
