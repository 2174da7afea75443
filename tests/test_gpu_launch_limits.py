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


@pytest.mark.parametrize("v,k", [(1 << 20, 8200), (8200, 8200), (3, 8)])
def test_no_rows_clear_a_gradient_of_any_size(v, k):
    """dw of 17 GB: more 4-byte words than a launch has threads."""
    announce("n = 0", v, k)
    dw = torch.full((v * k + 8,), float("nan"), dtype=torch.bfloat16, device=DEV)
    status = T.lib.swz_linear_ce_grad(None, None, T.X_BF16, None, None, None, None, None, dw.data_ptr(), 0, v, k, None, 0,
                                      torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert status == T.SWZ_OK
    assert not bool(dw[:-8].view(torch.int64).any()) and bool(torch.isnan(dw[-8:]).all())


@pytest.mark.parametrize("n,k", [(8200, 8200), (3, 4104), (70, 1028 * 8), (1000, 8), (129, 520)])
def test_input_gradient_of_any_shape(n, k):
    """Every element of dh is some thread's, whatever k leaves of its workgroups' 256 pieces.  H = 0 makes both words'
    logits zero and their probabilities one half, so dh is the upstream 2 times (w0 + w1) / 2 - w0."""
    announce("dh", n, k)
    h = torch.zeros(n, k, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(2, k, dtype=torch.bfloat16, device=DEV)
    w[0] = 1.0
    w[1] = 1.0 + torch.arange(k, device=DEV) % 5
    target = torch.zeros(n, dtype=torch.int64, device=DEV)
    ws = torch.empty(T.swz_linear_loss_workspace(n, 2, k, grad=True), dtype=torch.uint8, device=DEV)
    loss, lse, zt = (torch.empty(n, device=DEV) for _ in range(3))
    dh = torch.full_like(h, float("nan"))
    T.swz_linear_ce(h, w, target, loss, lse, zt, n, 2, k, ws)
    T.swz_linear_ce_grad(h, w, target, lse, zt, torch.full((n,), 2.0, device=DEV), dh, None, n, 2, k, ws)
    torch.cuda.synchronize()
    # p is 1/2 within fp32's rounding of log 2 and fp16's of dz (2^-11), the result's rounding 2^-8: less than 2^-7; the
    # two words' parts where w0 = w1 cancel to their dz's difference
    ref = (w[1] - w[0]).double().expand(n, k)
    assert bool(((dh.double() - ref).abs() <= 2.0 ** -7 * ref + 2.0 ** -10).all())
