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


# 256-column tiles over clusters of three SMs: a rank passes its partial tile through the operand
# ring, which the last block's second MMA may still read.  The blocks are 64 to 67 (33 to 40), so that a
# rank's last block lies in each of the ring's four stages.
@pytest.mark.parametrize("op,T,N,K", [("fwd", 16, 12288, 8192), ("fwd", 100, 12288, 8320), ("fwd", 1, 12288, 8576),
                                      ("fwd", 128, 12288, 8704), ("dgrad", 16, 8192, 12288), ("dgrad", 77, 8448, 12288),
                                      ("dgrad", 3, 8576, 12288), ("wgrad", 4096, 1024, 1536), ("wgrad", 4200, 1024, 1536),
                                      ("wgrad", 4500, 1024, 1536), ("wgrad", 5000, 2048, 768), ("wgrad", 4700, 1024, 1536)])
def test_wide_tiles_split_over_clusters(op, T, N, K):
    exact(op, T, N, K, repeats=20)
