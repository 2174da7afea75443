"""More of the gated block on the GPU, beside test_gpu_gated.py: relative errors where an activation is small.

A product of one x and one w is exact in fp32, so g and u are known to the bit and what remains is the activation's own
error and the result's rounding, at most a half step (2^-8 bf16, 2^-11 fp16, relative, in the normal range)."""

import math

import numpy as np
import pytest

from test_gpu_gated import DEV, DT, announce

import torch

import tiled_movement_amd as T

pytestmark = pytest.mark.gpu

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def gelu64(z):
    """(GELU, its derivative) without a difference of near numbers: Phi(z) = erfc(-z / sqrt 2) / 2."""
    cdf = 0.5 * _erfc(-z / math.sqrt(2))
    return z * cdf, cdf + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def tail(dt, low, top):
    """Gates z from -low to -3 in their type's steps, and powers of two that bring GELU(z) to 1/2 .. 2, up to 2^top."""
    t = DT[dt][0]
    z = torch.linspace(-low, -3, 333).to(t)
    by = np.exp2(np.clip(np.round(-np.log2(np.abs(gelu64(z.double().numpy())[0]))), 0, top))
    return z, by


# fp32's part, relative: erfc(x) moves by 2 x^2 times its argument's rounding, z^2 in all, and the exponential by as much;
# the functions and the products beside them take a few roundings more
def own(z):
    return (z * z + 32) * 2.0 ** -23


@pytest.mark.parametrize("n", [1, 40, 300])
@pytest.mark.parametrize("dt,low,top", [("fp16", 6.0, 30), ("bf16", 8.0, 60)])
def test_gelu_keeps_its_digits_far_below_zero(dt, low, top, n):
    """y, dwu and dwg of gates where 1 + erf(z / sqrt 2) would cancel (2.7e-4 at -4, 4% at -5, all of it from -5.5 on)."""
    announce("gelu tail", dt, n)
    t, xt, step, _ = DT[dt]
    z, by = tail(dt, low, top)
    f, k, half = z.numel(), 8, 2.0 ** 15
    x = torch.zeros(n, k, dtype=t)
    x[:, 0], x[:, 1] = 1.0, half
    wg, wu = torch.zeros(f, k, dtype=t), torch.zeros(f, k, dtype=t)
    wg[:, 0] = z
    wu[:, 1] = torch.from_numpy(by / half).to(t)  # powers of two: u = by
    d = [v.to(DEV) for v in (x, wg, wu)]
    y, pre = torch.empty(n, f, dtype=t, device=DEV), torch.empty(2, n, f, device=DEV)
    T.swz_gated(*d, y, n, f, k, x_type=xt, act=T.ACT_GELU, pre=pre)
    torch.cuda.synchronize()
    zd = z.double().numpy()
    assert np.array_equal(pre[0, 0].double().cpu().numpy(), zd) and np.array_equal(pre[1, 0].double().cpu().numpy(), by)
    a, da = gelu64(zd)
    want = a * by
    tol = (step + own(zd)) * np.abs(want)
    assert np.abs(want).min() > 2.0 ** -10 and np.abs(want).max() < 4
    # what the tolerance is to tell apart
    lost = 0.5 * (np.float32(1) + np.vectorize(math.erf)(zd / math.sqrt(2)).astype(np.float32)) * zd * by
    assert np.any(np.abs(lost - want) > tol)
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= tol)

    # gradients of one row: dwu[:, 0] = du, dwg[:, 0] = dg, held as two terms (the second of fp16 to 2^-25) and rounded again
    if n != 1:
        return
    dy = torch.from_numpy(np.minimum(by, half))[None].to(t)
    ws = torch.empty(T.swz_gated_workspace(n, f, k), dtype=torch.uint8, device=DEV)
    for kept in (pre, None):
        dwg, dwu = torch.empty(f, k, dtype=t, device=DEV), torch.empty(f, k, dtype=t, device=DEV)
        wu.zero_()
        wu[:, 0] = 1.0  # u = 1 for dg
        one = torch.stack([pre[0], torch.ones_like(pre[1])]) if kept is not None else None
        T.swz_gated_grad(d[0], d[1], wu.to(DEV), dy.to(DEV), None, dwg, dwu, n, f, k, ws, x_type=xt, act=T.ACT_GELU, pre=one)
        torch.cuda.synchronize()
        dyd = dy[0].double().numpy()
        for got, v in ((dwu, dyd * a), (dwg, dyd * da)):
            some = np.abs(v) > 2.0 ** -8
            assert some.sum() > 50
            err = np.abs(got[:, 0].double().cpu().numpy() - v)[some]
            assert np.all(err <= (step * (1 + step) + 2 * own(zd[some])) * np.abs(v[some]) + 2.0 ** -25)


@pytest.mark.parametrize("m", [1, 7, 30])
@pytest.mark.parametrize("dt,low,top", [("fp16", 6.0, 29), ("bf16", 8.0, 60)])
def test_gelu_of_4_bit_weights_keeps_its_digits(dt, low, top, m):
    """Gates of one code below the zero point, -scale, and up values of one above it."""
    announce("gelu tail w4", dt, m)
    t, xt, step, _ = DT[dt]
    z, by = tail(dt, low, top)
    n, k, half = z.numel(), 32, 2.0 ** 15
    x = torch.zeros(m, k, dtype=t)
    x[:, 0], x[:, 1] = 1.0, half
    qg, qu = (torch.full((n, k // 2), 0x88, dtype=torch.uint8) for _ in range(2))
    qg[:, 0], qu[:, 0] = 0x87, 0x98  # the even column's code in the low half
    sg, su = (-z)[:, None].contiguous(), torch.from_numpy(by / half)[:, None].to(t)
    c = torch.empty(m, n, dtype=t, device=DEV)
    T.swz_gated_w4(x.to(DEV), qg.to(DEV), sg.to(DEV), qu.to(DEV), su.to(DEV), c, m, n, k, group=32, x_type=xt, act=T.ACT_GELU)
    torch.cuda.synchronize()
    zd = z.double().numpy()
    want = gelu64(zd)[0] * by
    assert np.all(np.abs(c.double().cpu().numpy() - want) <= (step + own(zd)) * np.abs(want))


def test_dx_of_weights_behind_2_to_32_bytes():
    """dx of weights of 4.6 GB each, with dy in a few columns only, on both sides of 2^32 bytes: sums short enough that one
    column left out, or taken from another row of a weight, shows."""
    announce("gated dx 2^32")
    n, f, k = 24, 140001, 16392
    u32 = 2.0 ** -23
    g = torch.Generator(device=DEV)
    g.manual_seed(13)
    wg, wu = (torch.empty(f, k, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for w in (wg, wu):
        for i in range(0, f, 20000):
            w[i:i + 20000] = torch.randn(min(20000, f - i), k, generator=g, device=DEV) / 128
    border = (1 << 32) // (2 * k)
    cols = torch.tensor([0, 65537, border - 1, border, border + 1, 131072, f - 1], device=DEV)
    x = torch.randn(n, k, generator=g, device=DEV).bfloat16()
    dy = torch.zeros(n, f, dtype=torch.bfloat16, device=DEV)
    dy[:, cols] = (torch.rand(n, cols.numel(), generator=g, device=DEV) + 0.5).bfloat16()
    y, pre = torch.empty_like(dy), torch.empty(2, n, f, device=DEV)
    ws = torch.empty(T.swz_gated_workspace(n, f, k), dtype=torch.uint8, device=DEV)
    T.swz_gated(x, wg, wu, y, n, f, k, pre=pre)
    dx = [torch.full_like(x, float("nan")) for _ in range(2)]
    T.swz_gated_grad(x, wg, wu, dy, dx[0], None, None, n, f, k, ws, pre=pre)
    T.swz_gated_grad(x, wg, wu, dy, dx[1], None, None, n, f, k, ws)
    torch.cuda.synchronize()
    zg, zu, d = pre[0][:, cols].double(), pre[1][:, cols].double(), dy[:, cols].double()
    s = torch.sigmoid(zg)
    dg, du = d * zu * s * (1 + zg * (1 - s)), d * zg * s
    terms = torch.stack([dg[:, i, None] * wg[c].double() + du[:, i, None] * wu[c].double() for i, c in enumerate(cols)])
    ref = terms.sum(0)
    size = sum(dg[:, i, None].abs() * wg[c].double().abs() + du[:, i, None].abs() * wu[c].double().abs() for i, c in enumerate(cols))
    # dg and du off by a rounding and 64 u (1 + |z|) of the activation, |z| below 8; some 14 terms in fp32; one rounding
    assert float(zg.abs().max()) < 8 and float(zu.abs().max()) < 8
    tol = (2.0 ** -8 + 64 * 9 * u32 + 64 * u32) * size
    tol += 2.0 ** -8 * (ref.abs() + tol)
    assert bool(((dx[0].double() - ref).abs() <= tol).all())
    for wrong in [torch.zeros_like(ref), -ref] + [ref - t for t in terms] + [ref - t + t.roll(1, 1) for t in terms]:
        assert float(((wrong - ref).abs() > tol).double().mean()) > 0.5
    # g and u made again differ in their sums' order: a step of dg and du each where that tips a rounding
    assert bool(((dx[1].double() - dx[0].double()).abs() <= 2.0 ** -7 * size + 2.0 ** -7 * ref.abs()).all())
