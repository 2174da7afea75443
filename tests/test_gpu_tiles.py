"""Every product tile that large calls take, at sizes just past the rules' borders (tile_cases.py).

8-bit products of small whole numbers under scales from 2^-2 to 2^2 are multiples of 2^-4 whose
magnitudes add up to at most 9 * 16 * k < 2^18 (k <= 1000): exact in fp32, in the 8-bit instruction
too (products below 16 in every group), so an fp32 result has to be equal and a bf16 result equal to
the rounded one.  The losses are held to the bounds of test_gpu_loss_rows.py."""

import pytest
import torch

import tiled_movement_amd as T
from test_gpu_loss import Case
from test_gpu_loss_rows import check_rows
from tile_cases import GEMM, GEMM_K, LOSS

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = {"e4m3": (torch.float8_e4m3fn, T.F8_E4M3), "e5m2": (torch.float8_e5m2, T.F8_E5M2)}


def announce(*what):
    print("case:", *what, flush=True)


def operand(r, k, kind, square, scale_type, seed):
    """(bytes [r][ld], scales, float64 values); bytes behind k are NaN bytes."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    ld = -(-k // 16) * 16 + 16
    v = torch.randint(-3, 4, (r, k), generator=g, device=DEV).float()
    data = torch.full((r, ld), 0x7F, dtype=torch.uint8, device=DEV)
    data[:, :k] = v.to(F8[kind][0]).view(torch.uint8)
    e = torch.randint(-2, 3, (-(-r // 128) if square else r, -(-k // 128)), generator=g, device=DEV)
    s = (e + 127).to(torch.uint8) if scale_type == T.SCALE_E8M0 else torch.exp2(e.float())
    f = torch.exp2(e.double()).repeat_interleave(128, 1)[:, :k]
    f = f.repeat_interleave(128, 0)[:r] if square else f
    return data, s, v.double() * f


def product(m, n, k, ak, bk, sqa, sqb, scale_type, seed):
    a, b = operand(m, k, ak, sqa, scale_type, seed), operand(n, k, bk, sqb, scale_type, seed + 1)
    ref = a[2] @ b[2].t()
    for c_type, dt in ((T.C_F32, torch.float32), (T.C_BF16, torch.bfloat16)):
        c = torch.full((m, n), float("nan"), dtype=dt, device=DEV)
        T.swz_gemm_f8(a[0], a[1], b[0], b[1], c, m, n, k, lda=a[0].shape[1], ldb=b[0].shape[1], a_type=F8[ak][1],
                      b_type=F8[bk][1], a_block=int(sqa), b_block=int(sqb), scale_type=scale_type, c_type=c_type)
        assert torch.equal(c, ref.to(dt)), (c_type, int((c != ref.to(dt)).sum()))


SCALES = [(T.SCALE_E8M0, False, True), (T.SCALE_E8M0, False, False), (T.SCALE_E8M0, True, True), (T.SCALE_F32, False, True),
          (T.SCALE_F32, False, False), (T.SCALE_F32, True, False)]


@pytest.mark.parametrize("scale_type,sqa,sqb", SCALES)
@pytest.mark.parametrize("k", GEMM_K)
@pytest.mark.parametrize("tile", GEMM)
def test_gemm_in_every_tile(tile, k, scale_type, sqa, sqb):
    m, n = GEMM[tile]
    announce("gemm tile", tile, m, n, k, scale_type, sqa, sqb)
    product(m, n, k, "e4m3", "e4m3", sqa, sqb, scale_type, k)


@pytest.mark.parametrize("ak,bk", [("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("scale_type,sqa,sqb", [SCALES[0], SCALES[1], SCALES[3], SCALES[4]])
@pytest.mark.parametrize("tile", GEMM)
def test_gemm_types_in_every_tile(tile, scale_type, sqa, sqb, ak, bk):
    m, n = GEMM[tile]
    announce("gemm tile types", tile, ak, bk, scale_type, sqa, sqb)
    product(m, n, 392, ak, bk, sqa, sqb, scale_type, 7)


@pytest.mark.parametrize("n", [2199, 2201])
def test_gemm_large_tile_with_unaligned_rows(n):
    announce("gemm large tile, rows of C off 16 bytes", n)
    product(2100, n, 520, "e4m3", "e4m3", False, True, T.SCALE_E8M0, 9)


@pytest.mark.parametrize("m,n", [(8200, 300), (300, 8200), (5000, 5100)])
def test_gemm_over_wide_and_tall_grids(m, n):
    """Grids tens of tiles along either axis: every tile is some workgroup's."""
    announce("gemm grid", m, n)
    product(m, n, 136, "e4m3", "e4m3", False, True, T.SCALE_E8M0, 11)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("top,tau", [(0, 1.0), (20, 1.7)])
@pytest.mark.parametrize("shape", LOSS)
def test_losses_in_every_tile(shape, top, tau, dt):
    announce("loss tile", shape, top, dt)
    c = Case(*shape, dt, top=top, tau=tau, seed=shape[0])
    d = c.device()
    c.forward(d)
    c.backward(d)
    torch.cuda.synchronize()
    check_rows(c, d)


@pytest.mark.parametrize("ea,eb", [(1, 200), (253, 60), (30, 200), (0, 254), (127, 127), (254, 4)])
@pytest.mark.parametrize("m,n", [(90, 140), (2100, 2200)])
def test_gemm_far_scales_with_a_rounded_result(m, n, ea, eb):
    """E8M0 scales at the ends of their range, through the 8-bit instruction: exact up to the one rounding to bf16."""
    announce("gemm far scales, bf16", m, n, ea, eb)
    k = 256
    a, b = operand(m, k, "e4m3", False, T.SCALE_E8M0, 13), operand(n, k, "e4m3", True, T.SCALE_E8M0, 14)
    va, vb = (t[0][:, :k].view(torch.float8_e4m3fn).double() for t in (a, b))
    a[1].fill_(ea)
    b[1].fill_(eb)
    ref = (va @ vb.t()) * 2.0 ** (ea + eb - 254)
    c = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device=DEV)
    T.swz_gemm_f8(a[0], a[1], b[0], b[1], c, m, n, k, lda=a[0].shape[1], ldb=b[0].shape[1])
    assert torch.equal(c, ref.to(torch.bfloat16))
