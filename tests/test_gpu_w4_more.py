"""More of the 4-bit products on the GPU, with the checks and tolerances of test_gpu_w4.py."""

import numpy as np
import pytest

from test_gpu_w4 import ACT, DEV, DT, Weights, announce

import torch

import tiled_movement_amd as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("dt,group", [("bf16", 128), ("bf16", 32), ("fp16", 64)])
@pytest.mark.parametrize("n,k", [(70, 1312), (4200, 544)])
def test_few_rows_have_the_bits_of_a_full_block(n, k, dt, group, zero):
    """Areas of 4 and 8 rows of X: the bits that a call of 16 rows gives, whose sums go in the same order."""
    announce("w4 few rows", n, k, dt, group, zero)
    rng = np.random.default_rng(n + k)
    w = [Weights(rng, n, k, group, dt, zero) for _ in range(2)]
    x = torch.from_numpy(rng.standard_normal((16, k))).to(DT[dt][0]).to(DEV)

    def run(m, two):
        c = torch.full((m, n), 7.0, dtype=x.dtype, device=DEV)
        if two:
            T.swz_gated_w4(x[:m], *w[0].on[:2], *w[1].on[:2], c, m, n, k, group=group, x_type=DT[dt][1], act=ACT["silu"],
                           zero_g=w[0].on[2], zero_u=w[1].on[2])
        else:
            T.swz_gemm_w4(x[:m], *w[0].on[:2], c, m, n, k, group=group, x_type=DT[dt][1], zero=w[0].on[2])
        torch.cuda.synchronize()
        return c

    for two in (False, True):
        want = run(16, two)
        for m in range(1, 10):
            assert torch.equal(run(m, two), want[:m]), (m, two)
