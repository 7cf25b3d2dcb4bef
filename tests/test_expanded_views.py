"""Views that repeat their memory (stride 0, as expand makes them) are refused before any launch: the C ABI takes a
stride of 0 as packed, which would lead past the storage."""
import pytest
import torch

import fp32_dense_projection_gb300 as dp
from fp32_dense_projection_gb300 import _call, grouped


def bf16(*shape, device="cpu"):
    return torch.zeros(shape, dtype=torch.bfloat16, device=device)


def test_marshalling_refuses_stride_0():
    with pytest.raises(ValueError, match="stride 0"):
        _call.ld(bf16(1, 64).expand(128, 64), "f", "x")
    with pytest.raises(ValueError, match="stride 0"):
        grouped._experts(bf16(64, 32).expand(8, 64, 32), "f", "w", (8, 64, 32))
    with pytest.raises(ValueError, match="stride 0"):
        grouped._experts(bf16(8, 1, 32).expand(8, 64, 32), "f", "w", (8, 64, 32))
    # one row or expert has no stride to speak of
    assert _call.ld(bf16(1, 64).expand(1, 64), "f", "x") == 64 and _call.ld(bf16(0, 64), "f", "x") == 64
    assert _call.ld(bf16(5, 96)[:, :64], "f", "x") == 96
    assert grouped._experts(bf16(64, 32).expand(1, 64, 32), "f", "w", (1, 64, 32)) == (32, 64 * 32)
    assert grouped._experts(bf16(64, 8, 32).transpose(0, 1), "f", "w", (8, 64, 32)) == (8 * 32, 32)


def test_dense_marshalling_refuses_stride_0():
    with pytest.raises(ValueError, match="stride 0"):
        dp._ld(bf16(1, 64).expand(128, 64))
    for t in (bf16(64, 32).expand(8, 64, 32), bf16(8, 1, 32).expand(8, 64, 32)):
        with pytest.raises(ValueError, match="stride 0"):
            dp._bview(t, "f")
    assert dp._ld(bf16(1, 64).expand(1, 64)) == 64 and dp._ld(bf16(5, 96)[:, :64]) == 96
    assert dp._bview(bf16(64, 8, 32).transpose(0, 1), "f") == (8 * 32, 32) and dp._bview(bf16(1, 4, 32), "f") == (32, 128)


@pytest.mark.gpu
def test_dense_entry_points_refuse_stride_0():
    x, row = bf16(128, 64, device="cuda"), bf16(1, 64, device="cuda").expand(128, 64)
    b, one = bf16(4, 64, 64, device="cuda"), bf16(64, 64, device="cuda").expand(4, 64, 64)
    f, frow = x.float(), row.float()[:1].expand(128, 64)
    calls = [lambda: dp.dp_gemm_fwd(row, x), lambda: dp.dp_gemm_fwd(x, row), lambda: dp.dp_gemm_dgrad(row, x[:64]),
             lambda: dp.dp_gemm_fwd(x, x[:64], out=row), lambda: dp.dp_gemm_wgrad(x, row), lambda: dp.dp_gemm_bwd(row, x, x[:64]),
             lambda: dp.dp_gemm_wgrad_noalloc(row, x, x[:64]), lambda: dp.router_fwd(frow, f), lambda: dp.router_wgrad(f, frow),
             lambda: dp.dp_gemm_fwd_batched(b, one), lambda: dp.dp_gemm_dgrad_batched(one, b),
             lambda: dp.dp_gemm_wgrad_batched(b, b, out=one)]
    for call in calls:
        with pytest.raises(ValueError, match="stride 0"):
            call()


@pytest.mark.gpu
def test_entry_points_refuse_stride_0():
    x, row = bf16(128, 64, device="cuda"), bf16(1, 64, device="cuda").expand(128, 64)
    w, one = bf16(4, 64, 64, device="cuda"), bf16(64, 64, device="cuda").expand(4, 64, 64)
    o = torch.tensor([0, 30, 60, 90, 128], dtype=torch.int32, device="cuda")
    q, s = dp.fp8_quantize(x)
    qc, sc = dp.fp8_quantize(x, "col")
    wq, ws = dp.fp8_quantize(w[0], "block")
    eq = wq[:1].expand(128, 64)
    calls = [lambda: dp.dp_gemm_fwd_grouped(row, w, o), lambda: dp.dp_gemm_fwd_grouped(x, one, o),
             lambda: dp.dp_gemm_fwd_grouped(x, w, o, out=row), lambda: dp.dp_gemm_dgrad_grouped(row, w, o),
             lambda: dp.dp_gemm_dgrad_grouped(x, one, o), lambda: dp.dp_gemm_wgrad_grouped(row, x, o),
             lambda: dp.dp_gemm_wgrad_grouped(x, row, o), lambda: dp.dp_gemm_wgrad_grouped(x, x, o, out=one),
             lambda: dp.fp8_quantize(row), lambda: dp.fp8_quantize(row.float()[:1].expand(128, 64), "both"),
             lambda: dp.dp_gemm_fwd_fp8(eq, s, wq, ws), lambda: dp.dp_gemm_fwd_fp8(q, s, eq[:64], ws),
             lambda: dp.dp_gemm_fwd_fp8(q, s, wq, ws, out=row), lambda: dp.dp_gemm_dgrad_fp8(eq, s, wq, ws),
             lambda: dp.dp_gemm_wgrad_fp8(eq, sc, qc, sc)]
    for f in calls:
        with pytest.raises(ValueError, match="stride 0"):
            f()
    assert torch.equal(dp.dp_gemm_fwd_grouped(row.contiguous(), one.contiguous(), o), x)
