"""Sizes whose threads do not fit one launch along one axis."""

import pytest
import torch

import tiled_movement_amd as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def announce(*what):
    print("case:", *what, flush=True)


def test_gemm_rows_behind_2_to_22_tiles():
    """2^29 + 517 rows of one result each, in tiles of 128 rows (fp32 result and scales): small whole numbers under
    powers of two, equal to the 64-bit product at both ends and around the 2^29 rows of a launch."""
    announce("gemm 2^29 rows")
    m, n, k = (1 << 29) + 517, 1, 16
    a = torch.randint(0, 4, (m, 16), dtype=torch.uint8, device=DEV)
    a.mul_(8).add_(0x30)  # 0.5, 1, 2, 4
    sa = torch.ones(m, 1, device=DEV)
    sa[::3] = 0.25
    b = torch.randint(0, 2, (1, 16), dtype=torch.uint8, device=DEV) * 0x38
    b[0, 3] = 0x38
    sb = torch.full((1, 1), 2.0, device=DEV)
    c = torch.full((m, 1), float("nan"), device=DEV)
    T.swz_gemm_f8(a, sa, b, sb, c, m, n, k, b_block=T.BLOCK_1X128, scale_type=T.SCALE_F32, c_type=T.C_F32)
    torch.cuda.synchronize()
    assert not bool(torch.isnan(c).any())
    part = 1 << 18
    for r in (slice(0, part), slice((1 << 29) - part, (1 << 29) + 517)):
        ref = (a[r].view(torch.float8_e4m3fn).double() * b.view(torch.float8_e4m3fn).double()).sum(dim=1, keepdim=True)
        assert torch.equal(c[r].double(), ref * sa[r].double() * 2.0)
