"""More of the gated block on the GPU, beside test_gpu_gated.py: relative errors where an activation is small.

A product of one x and one w is exact in fp32, so g and u are known to the bit and what remains is the activation's own
error and the result's rounding, at most a half step (2^-8 bf16, 2^-11 fp16, relative, in the normal range)."""

import math

import numpy as np
import pytest

from oracle import feed_forward as F
from test_gpu_gated import DEV, DT, Case, announce

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


# ------------------------------------------------- fp16 gradients at the ends of the type's range
class Ranged(Case):
    """fp16 inputs whose dg and du are far from 1, x and the weights being `out` and 1 / out of their usual size, so that
    dx (out > 1) or dwg and dwu (out < 1) are ordinary fp16 numbers."""

    def __init__(self, n, k, f, act, dy, out, seed):
        super().__init__(n, k, f, "fp16", act, seed=seed)
        rng = np.random.default_rng(seed + 1)
        half = DT["fp16"][0]
        self.x = (torch.from_numpy(rng.standard_normal((n, k))) * out).to(half)
        self.wg, self.wu = ((torch.from_numpy(rng.standard_normal((f, k))) * (s / out / np.sqrt(k))).to(half) for s in (1.5, 4.0))
        self.dy = (torch.from_numpy(rng.uniform(-1, 1, (n, f))) * dy).to(half)

    def near(self, d, which):
        """Relative to its norm, a result is off by its rounding and by that of dg and du: each at most a half step, 2^-11,
        and 0.4 of it in the mean, of terms of either sign."""
        x, wg, wu, dy = (getattr(self, a).double().numpy() for a in ("x", "wg", "wu", "dy"))
        want = dict(zip(("dx", "dwg", "dwu"), F.gated_grad(x, wg, wu, self.act, dy)))
        for w in which:
            assert np.abs(want[w]).max() < 65504 and np.linalg.norm(want[w]) > 0
            rms = np.sqrt(np.mean(want[w] ** 2))
            assert rms > 2.0 ** -11  # a normal number, so that steps are relative
            got = d[w].double().cpu().numpy()
            assert np.isfinite(got).all() and np.linalg.norm(got - want[w]) <= 2.0 ** -10 * np.linalg.norm(want[w]), w
        return F.gated_grad(x, wg, wu, self.act, dy)[3:]


SIZES = [(1, 8, 5), (3, 72, 130), (40, 264, 200), (300, 264, 333), (200, 1032, 2000)]


@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("act", F.ACTS)
@pytest.mark.parametrize("n,k,f", SIZES)
@pytest.mark.parametrize("which,dy,out", [(("dx",), 60000.0, 2.0 ** 9), (("dwg", "dwu"), 60000.0, 2.0 ** -9)])
def test_gradients_of_products_beyond_fp16(which, dy, out, n, k, f, act, pre):
    """dg of up to 10^6: no fp16 numbers, but the gradients are."""
    announce("gated range", n, k, f, act, pre, which)
    c = Ranged(n, k, f, act, dy, out, seed=n + f)
    d = c.device()
    c.forward(d, pre)
    c.backward(d, pre, which)
    torch.cuda.synchronize()
    dg, du = c.near(d, which)
    assert n * f < 100 or np.abs(dg).max() > 65520


@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("n,k,f", SIZES)
@pytest.mark.parametrize("which,dy,out", [(("dx",), 2.0 ** -14, 2.0 ** -10), (("dwg", "dwu"), 2.0 ** -14, 2.0 ** 10)])
def test_gradients_of_products_below_fp16(which, dy, out, n, k, f, pre):
    """dg and du of 2^-16 and less keep their digits."""
    announce("gated range", n, k, f, pre, which)
    c = Ranged(n, k, f, "silu", dy, out, seed=n + f)
    c.dy = (c.dy.double() * 2.0 ** -5).half()  # of few digits themselves
    d = c.device()
    c.forward(d, pre)
    c.backward(d, pre, which)
    torch.cuda.synchronize()
    c.near(d, which)


@pytest.mark.parametrize("n,k,f", SIZES[1:])
def test_range_of_one_product_leaves_the_other_alone(n, k, f):
    """dg beyond fp16 and du below its normal numbers in one call: u is large and the activation small."""
    announce("gated two ranges", n, k, f)
    rng = np.random.default_rng(n)
    c = Ranged(n, k, f, "silu", 64.0, 1.0, seed=n + k)
    c.x[:, 0] = 1.0
    c.wg = (torch.from_numpy(rng.standard_normal((f, k))) * 2.0 ** -22).half()
    c.wg[:, 0] = 0.0
    c.wu[:, 0] = 12000.0
    c.wu[:, 1:] = 0.0
    for pre in (True, False):
        d = c.device()
        c.forward(d, pre)
        c.backward(d, pre)
        torch.cuda.synchronize()
        x, wg, wu, dy = (getattr(c, a).double().numpy() for a in ("x", "wg", "wu", "dy"))
        _, _, dwu, dg, du = F.gated_grad(x, wg, wu, "silu", dy)
        assert np.abs(dg).max() > 65520 and np.abs(du).max() < 2.0 ** -8
        got = d["dwu"].double().cpu().numpy()
        # a half step of dwu and of du (held at 2^-10 of the largest at least), fp16's smallest step for what is below it
        assert np.linalg.norm(got - dwu) <= 2.0 ** -10 * np.linalg.norm(dwu) + 2.0 ** -25 * np.sqrt(dwu.size)


def test_infinities_stay_in_their_rows_beyond_the_range():
    """Values that are not finite do not count for the range of the others."""
    announce("gated range, infinities")
    c = Ranged(90, 72, 130, "silu", 60000.0, 2.0 ** 9, seed=4)
    c.dy[4] = 0.0
    d = c.device()
    c.forward(d)
    c.backward(d, which=("dx",))
    torch.cuda.synchronize()
    want = d["dx"].clone()
    assert bool(want.isfinite().all())
    d["dy"][4, 3], d["dy"][5, 7] = float("inf"), float("nan")
    for pre in (True, False):
        c.forward(d, pre)
        c.backward(d, pre, which=("dx",))
        torch.cuda.synchronize()
        keep = [i for i in range(90) if i not in (4, 5)]
        assert bool((d["dx"][keep].float() - want[keep].float()).abs().max() <= 2.0 ** -10 * want.float().abs().max())
        assert not bool(d["dx"][4].isfinite().any()) and bool(d["dx"][5].isnan().all())


def test_range_is_each_calls_own():
    """One workspace, calls of large, ordinary and small gradients in turn, and replays of one graph over all of them."""
    announce("gated range in turn")
    n, k, f = 40, 264, 200
    cases = [Ranged(n, k, f, "silu", dy, out, seed=7) for dy, out in ((60000.0, 2.0 ** 9), (1.0, 1.0), (2.0 ** -16, 2.0 ** -9))]
    d = cases[0].device()
    order = [0, 1, 2, 1, 0, 2, 0]
    want = {}
    for pre in (True, False):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cases[0].forward(d, pre)
            cases[0].backward(d, pre, ("dx",))
        for i in order:
            for a in ("x", "wg", "wu", "dy"):
                d[a].copy_(getattr(cases[i], a))
            cases[i].forward(d, pre)
            cases[i].backward(d, pre, ("dx",))
            torch.cuda.synchronize()
            cases[i].near(d, ("dx",))
            assert torch.equal(want.setdefault((i, pre), d["dx"].clone()), d["dx"])
            d["dx"].fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(d["dx"], want[i, pre])


def test_range_where_workgroups_share_slots():
    """More tiles of dg than the call tells apart (2048): gradients of made-again products, large at one place of the last
    tile, against the same sums in 64 bits on the GPU."""
    announce("gated range, many tiles")
    n, k, f = 4100, 16, 16900
    g = torch.Generator(device=DEV)
    g.manual_seed(21)
    rand = lambda *s: torch.rand(*s, generator=g, device=DEV) - 0.5  # noqa: E731
    x, wg, wu = (rand(n, k) * 2.0 ** -7).half(), (rand(f, k) * 2.0 ** 8).half(), (rand(f, k) * 2.0 ** 8).half()
    dy = (rand(n, f) * 0.01).half()
    ws = torch.full((T.swz_gated_workspace(n, f, k),), 0xFF, dtype=torch.uint8, device=DEV)
    zg, zu = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    for last in (0.0, 60000.0):
        dy[n - 1, f - 1] = last
        x[n - 1] = 2.0 ** -6
        wg[f - 1], wu[f - 1] = 2.0 ** 8, 2.0 ** 8
        zg[n - 1], zu[n - 1] = (w.double() @ x[n - 1].double() for w in (wg, wu))
        zg[:, f - 1], zu[:, f - 1] = (x.double() @ w[f - 1].double() for w in (wg, wu))
        dwg, dwu = torch.full_like(wg, float("nan")), torch.full_like(wu, float("nan"))
        T.swz_gated_grad(x, wg, wu, dy, None, dwg, dwu, n, f, k, ws, x_type=T.X_F16)
        torch.cuda.synchronize()
        s = torch.sigmoid(zg)
        for got, d in ((dwg, dy.double() * zu * s * (1 + zg * (1 - s))), (dwu, dy.double() * zg * s)):
            assert (float(d.abs().max()) > 65520) == (last > 0)
            want = d.t().contiguous() @ x.double()
            err = (got.double() - want).norm(dim=1)
            # rounding of d and of the result; what the largest leaves of the others: 2^-25 of fp16 at its scale
            size = (d.abs().t().contiguous() @ x.double().abs()).norm(dim=1)
            assert bool((err <= 2.0 ** -10 * want.norm(dim=1) + 2.0 ** -12 * size).all())
