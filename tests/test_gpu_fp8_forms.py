"""The 8-bit products in launch forms that the sizes of test_gpu_fp8.py do not reach, on integers:
every sum is exact in FP32, so outputs must be equal bit for bit."""
import pytest
import torch

import fp32_dense_projection_gb300 as dp
from test_gpu_fp8 import call, operands, product

pytestmark = pytest.mark.gpu


def exact(op, T, N, K, repeats=1):
    (a, da), (b, db) = operands(op, T, N, K, T + N + K, ints=True)
    ref = product(op, da, db)
    for _ in range(repeats):
        assert torch.equal(call(op, a, b, out_dtype=torch.float32), ref.float())
    assert torch.equal(call(op, a, b), ref.to(torch.bfloat16))
    assert dp.device_error() == 0


def force(monkeypatch, **form):
    for k, v in form.items():
        monkeypatch.setenv(f"DP_FORCE_{k}", str(v))


# 256-column tiles over clusters: a rank passes its partial tile through the operand ring, which the last
# block's second MMA may still read.  The blocks are 64 to 67 (32 to 40) over three ranks, so that a rank's last block lies
# in each of the ring's four stages.
@pytest.mark.parametrize("op,T,N,K", [("fwd", 16, 12288, 8192), ("fwd", 100, 12288, 8320), ("fwd", 1, 12288, 8576),
                                      ("fwd", 128, 12288, 8704), ("dgrad", 16, 8192, 12288), ("dgrad", 77, 8448, 12288),
                                      ("dgrad", 3, 8576, 12288), ("wgrad", 4096, 1024, 1536), ("wgrad", 4200, 1024, 1536),
                                      ("wgrad", 4500, 1024, 1536), ("wgrad", 5000, 2048, 768), ("wgrad", 4700, 1024, 1536)])
def test_wide_tiles_split_over_clusters(monkeypatch, op, T, N, K):
    force(monkeypatch, BN=256, PAIR=0, SPLITS=3)
    exact(op, T, N, K, repeats=20)


@pytest.mark.parametrize("op,T,N,K", [("fwd", 16, 8192, 20608), ("fwd", 128, 8192, 28672), ("dgrad", 50, 20736, 8192),
                                      ("wgrad", 8192, 512, 2560), ("wgrad", 16500, 1024, 1024)])
def test_wide_tiles_split_as_planned(op, T, N, K):
    """Sizes at which the planner takes that form by itself on 152 SMs."""
    exact(op, T, N, K, repeats=20)


FORMS = {"128": dict(BN=128, PAIR=0, SPLITS=1), "256": dict(BN=256, PAIR=0, SPLITS=1), "pair": dict(BN=256, PAIR=1, SPLITS=1)}


def sizes(op, gm, gn, gk):
    """(T, N, K) of a product of gm x gn outputs over gk contraction elements."""
    return {"fwd": (gm, gn, gk), "dgrad": (gm, gk, gn), "wgrad": (gk, gm, gn)}[op]


@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("op", ["fwd", "dgrad", "wgrad"])
def test_every_tile(monkeypatch, op, form):
    """One to nine blocks (the rings wrap), a partial last one, ragged tiles; then several tiles for each SM."""
    force(monkeypatch, **FORMS[form])
    for blocks in range(1, 10):
        exact(op, *sizes(op, 208, 528, 128 * blocks - (16 if blocks % 2 else 0)))
    exact(op, *sizes(op, 16, 144, 400))
    exact(op, *sizes(op, 2608, 4112, 656))


@pytest.mark.parametrize("split", range(2, 9))
@pytest.mark.parametrize("bn", [128, 256])
@pytest.mark.parametrize("op", ["fwd", "dgrad", "wgrad"])
def test_every_split(monkeypatch, op, bn, split):
    """Shares of one to six blocks (each residue of the ring's four stages), even and uneven ones."""
    force(monkeypatch, BN=bn, PAIR=0, SPLITS=split)
    for share in range(1, 7):
        exact(op, *sizes(op, 208, 528, 128 * share * split - 48), repeats=3)
        exact(op, *sizes(op, 80, 272, 128 * (share * split + 1)))
    exact(op, *sizes(op, 1, 256, 128 * 3 * split) if op != "wgrad" else sizes(op, 16, 256, 128 * 3 * split))


@pytest.mark.parametrize("form", [dict(BN=128, PAIR=1), dict(BN=64), dict(SPLITS=9), dict(PAIR=1, SPLITS=2), dict(BN=128, SPLITS=4)])
def test_forms_that_do_not_exist_are_refused(monkeypatch, form):
    (a, _), (b, _) = operands("fwd", 64, 256, 384, 1, ints=True)  # (three blocks: no split in four)
    force(monkeypatch, **form)
    with pytest.raises(dp.DPError) as e:
        call("fwd", a, b)
    assert e.value.status == 3


@pytest.mark.parametrize("ea,eb", [(-60, -60), (60, -60), (-60, 60), (60, 50)])
@pytest.mark.parametrize("op", ["fwd", "dgrad", "wgrad"])
def test_scales_at_the_ends_of_their_range(op, ea, eb):
    """Powers of two: exact in FP32 as long as no scale, product of scales or sum leaves its range."""
    for T, N, K in ((130, 144, 272), (2400, 2064, 2064)):
        (a, _), (b, _) = operands(op, T, N, K, 9, ints=True)
        a, b = (a[0], torch.full_like(a[1], 2.0 ** ea)), (b[0], torch.full_like(b[1], 2.0 ** eb))
        ref = product(op, a[0].double(), b[0].double()) * 2.0 ** (ea + eb)
        assert torch.equal(call(op, a, b, out_dtype=torch.float32), ref.float())
