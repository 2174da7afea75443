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


def test_products_of_codes_behind_2_to_32_bytes():
    """Codes of 4.9 GB: rows from all over, those around 2^32 bytes among them, have the bits that a call on a copy of them
    gives (a row of W has its sums in the same order whatever stands beside it); one and 20 rows of X, and the gated block."""
    announce("w4 products 2^32")
    n, k, group = 600001, 16416, 128
    g = torch.Generator(device=DEV)
    g.manual_seed(15)
    groups = -(-k // group)
    q = torch.randint(0, 1 << 62, (n * k // 16,), generator=g, device=DEV).view(torch.uint8).view(n, k // 2)
    s = torch.empty(n, groups, device=DEV).uniform_(0.5, 2, generator=g).div_(128).bfloat16()
    z = torch.randint(0, 16, (n, groups), generator=g, device=DEV, dtype=torch.uint8)
    border = (1 << 32) // (k // 2)
    rows = torch.cat([torch.arange(border - 300, border + 300, device=DEV), torch.arange(0, n, 149, device=DEV),
                      torch.arange(n - 40, n, device=DEV)])
    few = [t[rows].contiguous() for t in (q, s, z)]
    assert int(rows.numel()) > 4096  # the same rule for the rows of a workgroup
    x = torch.randn(20, k, generator=g, device=DEV).bfloat16()
    for m in (1, 20):
        for zero, zero_few in ((None, None), (z, few[2])):
            c, want = torch.full((m, n), float("nan"), dtype=x.dtype, device=DEV), torch.empty(m, rows.numel(), dtype=x.dtype, device=DEV)
            T.swz_gemm_w4(x[:m], q, s, c, m, n, k, group=group, zero=zero)
            T.swz_gemm_w4(x[:m], *few[:2], want, m, rows.numel(), k, group=group, zero=zero_few)
            torch.cuda.synchronize()
            assert torch.equal(c[:, rows], want) and bool(c.isfinite().all())
            assert want.double().std(dim=1).min() > 0.1  # nothing that zeros or one row in all places would give
    c, want = torch.full((2, n), float("nan"), dtype=x.dtype, device=DEV), torch.empty(2, rows.numel(), dtype=x.dtype, device=DEV)
    T.swz_gated_w4(x[:2], q, s, q, s, c, 2, n, k, group=group)
    T.swz_gated_w4(x[:2], *few[:2], *few[:2], want, 2, rows.numel(), k, group=group)
    torch.cuda.synchronize()
    assert torch.equal(c[:, rows], want) and bool(c.isfinite().all()) and want.double().std(dim=1).min() > 0.1
