"""Products grouped by expert on real operands, against the bound of their own summation: pieces of 512 contraction
elements, each 32 tensor-core steps (16 products and the running sum) that lose at most four units of 2^-23 of the sum of
magnitudes S, added in FP32 with one rounding each.  So |got - ref| <= (4 min(K, 512) / 16 + K / 512 + 2) 2^-23 S for FP32
outputs, and 2^-8 |ref| more for BF16 ones."""
import numpy as np
import pytest
import torch

import fp32_dense_projection_gb300 as dp
from gpu_common import DEV
from test_gpu_grouped import call, edges_of, reference, tensors

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("op", ["fwd", "dgrad", "wgrad"])
@pytest.mark.parametrize("T,E,N,K", [(64, 64, 1024, 512), (700, 4, 520, 4104), (3000, 3, 2056, 264), (9000, 1, 136, 128),
                                     (4031, 32, 1024, 512), (40, 2, 8200, 8200)])
def test_real_values_within_the_summations_bound(op, T, E, N, K):
    g = np.random.default_rng(T + E)
    counts = np.bincount(g.choice(E, T, p=g.dirichlet(np.ones(E))), minlength=E)
    edges = edges_of(counts)
    c = tensors(edges, T, N, K, seed=T, real=True)
    depth = {"fwd": K, "dgrad": N, "wgrad": int(counts.max())}[op]
    ref, mag = reference(op, c, edges, False), reference(op, c, edges, False, mag=True)
    tol = (4 * min(depth, 512) / 16 + depth / 512 + 2) * 2.0 ** -23 * mag
    assert bool(((call(op, c, out_dtype=torch.float32).double() - ref).abs() <= tol).all())
    assert bool(((call(op, c).double() - ref).abs() <= tol + 2.0 ** -8 * ref.abs()).all())


def test_padding_rows_of_more_than_2_31_bytes_are_zero():
    """An output row whose bytes pass 32 bits: the padding row is zeroed to its end, the expert's row is right at both ends."""
    N, K = 2 ** 29 + 64, 8
    W = torch.zeros(1, N, K, dtype=torch.bfloat16, device=DEV)
    W[0, :64] = 2
    W[0, -64:] = 3
    X = torch.ones(2, K, dtype=torch.bfloat16, device=DEV)
    out = torch.full((2, N), 5.0, device=DEV)
    dp.dp_gemm_fwd_grouped(X, W, torch.tensor([0, 1], dtype=torch.int32, device=DEV), out=out)
    assert bool((out[1] == 0).all())
    assert bool((out[0, :64] == 16).all()) and bool((out[0, -64:] == 24).all()) and bool((out[0, 64:-64] == 0).all())
