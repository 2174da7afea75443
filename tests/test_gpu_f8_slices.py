"""8-bit operands that are columns of wider matrices: the last row ends with its own last element, and what
lies behind it belongs to others, the call's own results among them."""

import numpy as np
import pytest
import torch

from oracle import products as P

import tiled_movement_amd as T
from test_gpu_f8 import check_quant, values

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def announce(*what):
    print("case:", *what, flush=True)


class Arena:
    """Pieces of one allocation, one right behind the other (16-byte steps)."""

    def __init__(self, size):
        self.mem, self.at = torch.full((size,), 0x5A, dtype=torch.uint8, device=DEV), 0

    def take(self, nbytes, dtype=torch.uint8):
        here = self.at
        self.at += -(-nbytes // 16) * 16
        return self.mem[here:here + nbytes].view(dtype)


@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("first", [0, 128, 744])
def test_quantize_columns_of_a_wider_matrix(square, first):
    announce("quant slice", square, first)
    r, c, ld = 130, 256, 1000
    x = torch.from_numpy(values(r, ld, 1)).to(torch.bfloat16)
    a = Arena(1 << 20)
    end = (r - 1) * ld + first + c
    xd = a.take(2 * end, torch.bfloat16)  # the matrix up to the last row's last column of the slice
    xd.copy_(x.flatten()[:end])
    br = 128 if square else 1
    q, s = a.take((r - 1) * 272 + c), a.take(-(-r // br) * 2)
    qt, st = a.take((c - 1) * 144 + r), a.take(-(-c // br) * 2)
    T.swz_quant_f8(xd[first:], q, s, r, c, block=int(square), ld_x=ld, ld_q=272, qt=qt, scale_t=st, ld_qt=144)
    torch.cuda.synchronize()
    xf = x[:, first:first + c].double().numpy()
    rows = np.full((r, 272), 0x5A, np.uint8)
    rows.flat[:q.numel()] = q.cpu().numpy()
    cols = np.full((c, 144), 0x5A, np.uint8)
    cols.flat[:qt.numel()] = qt.cpu().numpy()
    check_quant(rows, s.cpu().numpy().reshape(-1, 2), xf, "e4m3", square)
    check_quant(cols, st.cpu().numpy().reshape(-1, 2), np.ascontiguousarray(xf.T), "e4m3", square)


@pytest.mark.parametrize("m", [3, 70, 300])
@pytest.mark.parametrize("c_type", [T.C_F32, T.C_BF16])
@pytest.mark.parametrize("first,k", [(128, 256), (256, 250)])
def test_product_of_columns_of_wider_operands(m, c_type, first, k):
    """A part of k of two operands, C right behind both: small whole numbers, equal to the (rounded) 64-bit product."""
    announce("gemm slice", m, c_type, first, k)
    n, ld = 140, 512
    g = np.random.default_rng(m)
    va, vb = g.integers(-3, 4, (m, ld)).astype(np.float32), g.integers(-3, 4, (n, ld)).astype(np.float32)
    a = Arena(1 << 21)
    used = -(-k // 16) * 16

    def operand(v, rows):
        data = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).flatten()
        end = (rows - 1) * ld + first + used
        t = a.take(end)
        t.copy_(data[:end])
        return t[first:]

    b_op, a_op = operand(vb, n), operand(va, m)
    dt = torch.float32 if c_type == T.C_F32 else torch.bfloat16
    c = a.take(m * n * dt.itemsize, dt).view(m, n)
    ones = lambda rows: torch.full((rows, -(-k // 128)), 127, dtype=torch.uint8, device=DEV)  # noqa: E731
    T.swz_gemm_f8(a_op, ones(m), b_op, ones(n), c, m, n, k, lda=ld, ldb=ld, b_block=T.BLOCK_1X128, c_type=c_type)
    torch.cuda.synchronize()
    ref = P.product_f8(va[:, first:first + k].astype(np.float64), vb[:, first:first + k].astype(np.float64))
    assert torch.equal(c.cpu(), torch.from_numpy(ref).to(dt))
