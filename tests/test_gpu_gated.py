"""The gated feed-forward block and its gradients on the GPU against their 64-bit definitions.

Tolerances, to first order, from the operations (u = 2^-23 bounds one fp32 operation):

* g and u: k products summed in fp32, e = (k + 2) u sum |x||w|;
* an activation moves by at most 1.2 e with its argument (its slope is below 1.13) and its derivative by 0.9 e (its second
  derivative is below 0.8); by themselves they are off by a relative (|z| + 8) u of the exponential or error function
  that they are made of, the derivative's parts by that times |z| + 2;
* y: the product's parts, then one rounding (2^-8 bf16, 2^-11 fp16; below their normal ranges 2^-134 and 2^-25);
* dg, du: the same, one rounding; gradients: theirs carried through, fp32 sums of 2 f (n) products, one rounding.
"""

import numpy as np
import pytest

from oracle import feed_forward as F

import torch

import tiled_movement_amd as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -23
DT = {"bf16": (torch.bfloat16, T.X_BF16, 2.0 ** -8, 2.0 ** -134), "fp16": (torch.float16, T.X_F16, 2.0 ** -11, 2.0 ** -25)}
ACT = {"silu": T.ACT_SILU, "gelu": T.ACT_GELU, "gelu_tanh": T.ACT_GELU_TANH}


def announce(*what):
    print("case:", *what, flush=True)


class Case:
    def __init__(self, n, k, f, dt="bf16", act="silu", seed=0, scale=1.0):
        self.n, self.k, self.f, self.dt, self.act = n, k, f, dt, act
        rng = np.random.default_rng(seed)
        t = DT[dt][0]
        make = lambda *s: torch.from_numpy(rng.standard_normal(s))  # noqa: E731
        self.x = make(n, k).to(t)
        self.wg = (make(f, k) * scale * 1.5 / np.sqrt(k)).to(t)
        self.wu = (make(f, k) * scale / np.sqrt(k)).to(t)
        self.dy = (make(n, f) * torch.from_numpy(10.0 ** rng.uniform(-2, 0, (n, 1)))).to(t)

    def kw(self):
        return {"x_type": DT[self.dt][1], "act": ACT[self.act]}

    def device(self):
        d = {a: getattr(self, a).to(DEV) for a in ("x", "wg", "wu", "dy")}
        nan = lambda *s: torch.full(s, float("nan"), dtype=d["x"].dtype, device=DEV)  # noqa: E731
        d.update(y=nan(self.n, self.f), dx=nan(self.n, self.k), dwg=nan(self.f, self.k), dwu=nan(self.f, self.k))
        d["pre"] = torch.full((2, self.n, self.f), float("nan"), device=DEV)
        d["ws"] = torch.full((T.swz_gated_workspace(self.n, self.f, self.k),), 0xFF, dtype=torch.uint8, device=DEV)
        return d

    def forward(self, d, pre=True):
        T.swz_gated(d["x"], d["wg"], d["wu"], d["y"], self.n, self.f, self.k, pre=d["pre"] if pre else None, **self.kw())

    def backward(self, d, pre=True, which=("dx", "dwg", "dwu")):
        T.swz_gated_grad(d["x"], d["wg"], d["wu"], d["dy"], *(d[w] if w in which else None for w in ("dx", "dwg", "dwu")), self.n,
                         self.f, self.k, d["ws"], pre=d["pre"] if pre else None, **self.kw())

    def check(self, d, grad=True, pre=True):
        x, wg, wu, dy = (getattr(self, a).double().numpy() for a in ("x", "wg", "wu", "dy"))
        step, tiny = DT[self.dt][2], DT[self.dt][3]
        y, g, u = F.gated(x, wg, wu, self.act)
        a, da = F.activation(self.act, g)
        eg, eu = ((self.k + 2) * U * (np.abs(x) @ np.abs(w).T) for w in (wg, wu))
        z = np.abs(g) + eg
        ea = 1.2 * eg + z * (z + 8) * U
        eda = 0.9 * eg + (z + 2) * (z + 8) * U
        got = {w: d[w].double().cpu().numpy() for w in ("y", "dx", "dwg", "dwu", "pre")}
        if pre:
            assert np.all(np.abs(got["pre"][0] - g) <= eg) and np.all(np.abs(got["pre"][1] - u) <= eu)
        ey = np.abs(a) * eu + (np.abs(u) + eu) * ea + 4 * U * np.abs(y)
        ey += step * (np.abs(y) + ey) + tiny
        assert np.all(np.abs(got["y"] - y) <= ey), np.max(np.abs(got["y"] - y) / ey)
        if not grad:
            return
        dx, dwg, dwu, dg, du = F.gated_grad(x, wg, wu, self.act, dy)
        edg = np.abs(dy) * (np.abs(da) * eu + (np.abs(u) + eu) * eda) + 4 * U * np.abs(dg)
        edu = np.abs(dy) * ea + 4 * U * np.abs(du)
        # dg and du are rounded once, or held as two terms: what the first leaves, at most a half step, is rounded again
        held = step * step if self.n * self.f * self.k <= 1 << 23 else step
        edg, edu = (e + held * (np.abs(v) + e) + tiny for e, v in ((edg, dg), (edu, du)))
        sums = lambda e, v, r, terms: e @ r + (terms + 40) * U * ((np.abs(v) + e) @ r)  # noqa: E731
        bound = {"dx": sums(edg, dg, np.abs(wg), 2 * self.f) + sums(edu, du, np.abs(wu), 2 * self.f),
                 "dwg": sums(edg.T, dg.T, np.abs(x), self.n), "dwu": sums(edu.T, du.T, np.abs(x), self.n)}
        for w, r in (("dx", dx), ("dwg", dwg), ("dwu", dwu)):
            b = bound[w] + step * (np.abs(r) + bound[w]) + tiny
            err = np.abs(got[w] - r)
            assert np.all(err <= b), (w, np.max(err / b))


# one row, few rows, the border between the kernels, tiles' borders, odd features, one feature, k of part of a stage
SIZES = [(1, 8, 1), (1, 256, 300), (3, 72, 17), (16, 1032, 130), (17, 1032, 130), (64, 200, 127), (65, 64, 129), (128, 136, 257),
         (129, 520, 128), (257, 72, 255), (300, 256, 333), (2, 4104, 65)]


@pytest.mark.parametrize("act", F.ACTS)
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("n,k,f", SIZES)
def test_block_and_gradients(n, k, f, dt, act):
    announce("gated", n, k, f, dt, act)
    c = Case(n, k, f, dt, act, seed=n + k + f)
    d = c.device()
    c.forward(d)
    c.backward(d)
    torch.cuda.synchronize()
    c.check(d)


@pytest.mark.parametrize("dt,act", [("bf16", "silu"), ("fp16", "gelu"), ("bf16", "gelu_tanh")])
@pytest.mark.parametrize("n,k,f", SIZES)
def test_gradients_without_kept_products(n, k, f, dt, act):
    announce("gated again", n, k, f, dt, act)
    c = Case(n, k, f, dt, act, seed=n + k + f + 1)
    d = c.device()
    c.forward(d, pre=False)
    c.backward(d, pre=False)
    torch.cuda.synchronize()
    c.check(d, pre=False)


@pytest.mark.parametrize("n,k,f", [(1500, 264, 1100), (40, 2056, 2000), (3000, 64, 72), (520, 1288, 4100)])
def test_larger_tiles_and_split_sums(n, k, f):
    announce("gated large", n, k, f)
    for pre in (True, False):
        c = Case(n, k, f, seed=n)
        d = c.device()
        c.forward(d, pre)
        c.backward(d, pre)
        torch.cuda.synchronize()
        c.check(d, pre=pre)


@pytest.mark.parametrize("which", [("dx",), ("dwg",), ("dwu",), ("dwg", "dwu"), ("dx", "dwu")])
def test_some_of_the_gradients(which):
    announce("gated some", which)
    c = Case(70, 136, 200, seed=5)
    d = c.device()
    c.forward(d)
    c.backward(d)
    torch.cuda.synchronize()
    want = {w: d[w].clone() for w in which}
    for w in ("dx", "dwg", "dwu"):
        d[w].fill_(float("nan"))
    c.backward(d, which=which)
    torch.cuda.synchronize()
    for w in ("dx", "dwg", "dwu"):
        assert torch.equal(d[w], want[w]) if w in which else bool(d[w].isnan().all())


def test_no_rows():
    announce("gated no rows")
    c = Case(0, 64, 40)
    d = c.device()
    c.forward(d)
    c.backward(d)
    torch.cuda.synchronize()
    assert bool((d["dwg"] == 0).all()) and bool((d["dwu"] == 0).all())


@pytest.mark.parametrize("offset", [1, 2, 4, 8])
@pytest.mark.parametrize("n,f", [(5, 64), (70, 64), (300, 136)])
def test_results_off_16_bytes(n, f, offset):
    """y, dy and the kept products at any element; what lies around y stays."""
    announce("gated offset", n, f, offset)
    c = Case(n, 72, f, seed=3)
    d = c.device()
    flat = torch.full((n * f + 32,), 7.0, dtype=d["x"].dtype, device=DEV)
    pre = torch.full((2 * n * f + 32,), 7.0, device=DEV)
    dyf = torch.zeros(n * f + 32, dtype=d["x"].dtype, device=DEV)
    d["y"], d["pre"] = flat[offset:offset + n * f].view(n, f), pre[offset:offset + 2 * n * f].view(2, n, f)
    dyf[offset:offset + n * f] = d["dy"].reshape(-1)
    d["dy"] = dyf[offset:offset + n * f].view(n, f)
    c.forward(d)
    c.backward(d)
    torch.cuda.synchronize()
    c.check(d)
    assert bool((flat[:offset] == 7).all()) and bool((flat[offset + n * f:] == 7).all())
    assert bool((pre[:offset] == 7).all()) and bool((pre[offset + 2 * n * f:] == 7).all())


@pytest.mark.parametrize("act", F.ACTS)
@pytest.mark.parametrize("n", [4, 40])
def test_far_arguments(n, act):
    """Products of +-100 and +-30000: activations at their limits, no NaN, gradients finite."""
    announce("gated far", n, act)
    k, f = 64, 96
    c = Case(n, k, f, "bf16", act, seed=9)
    c.x[:, :] = 0.0
    c.x[:, 0] = 100.0
    c.wg[:, 0] = torch.linspace(-300, 300, f).to(torch.bfloat16)
    for pre in (True, False):
        d = c.device()
        c.forward(d, pre)
        c.backward(d, pre)
        torch.cuda.synchronize()
        c.check(d, pre=pre)


def test_rows_of_nan_and_infinity_stay_their_own():
    """A row of x that is not finite leaves the other rows of y and dx alone."""
    announce("gated nan")
    for n in (10, 90):
        c = Case(n, 72, 130, seed=2)
        d = c.device()
        c.forward(d)
        c.backward(d, which=("dx",))
        torch.cuda.synchronize()
        want = {w: d[w].clone() for w in ("y", "dx")}
        d["x"][3] = float("nan")
        d["x"][7, 5] = float("inf")
        for pre in (True, False):
            c.forward(d, pre)
            c.backward(d, pre, which=("dx",))
            torch.cuda.synchronize()
            keep = [i for i in range(n) if i not in (3, 7)]
            for w in ("y", "dx"):
                assert torch.equal(d[w][keep], want[w][keep])
            assert bool(d["y"][3].isnan().all()) and not bool(d["y"][7].isfinite().any())


def test_weights_of_one_matrix_in_turn():
    """Both weights as halves of one [2 f][k] matrix, and their gradients as halves of another."""
    announce("gated halves")
    c = Case(33, 64, 48, seed=8)
    d = c.device()
    both, grads = torch.cat([d["wg"], d["wu"]]), torch.empty(96, 64, dtype=torch.bfloat16, device=DEV)
    d["wg"], d["wu"], d["dwg"], d["dwu"] = both[:48], both[48:], grads[:48], grads[48:]
    c.forward(d)
    c.backward(d)
    torch.cuda.synchronize()
    c.check(d)


def test_same_bits_on_two_streams_and_in_graphs():
    announce("gated streams, graph")
    cases = [Case(300, 136, 520, seed=1), Case(40, 520, 264, "fp16", "gelu", seed=2)]
    ds, want = [], []
    for c in cases:
        d = c.device()
        c.forward(d)
        c.backward(d)
        torch.cuda.synchronize()
        c.check(d)
        ds.append(d)
        want.append({w: d[w].clone() for w in ("y", "dx", "dwg", "dwu")})

    def clear():
        for d in ds:
            for w in ("y", "dx", "dwg", "dwu", "pre"):
                d[w].fill_(float("nan"))
            d["ws"].fill_(0xFF)
        torch.cuda.synchronize()

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(d[w], e[w]) for d, e in zip(ds, want) for w in e)

    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    clear()
    for _ in range(3):
        for c, d, s in zip(cases, ds, streams):
            with torch.cuda.stream(s):
                c.forward(d)
                c.backward(d)
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c, d in zip(cases, ds):
            c.forward(d)
            c.backward(d)
    for _ in range(3):
        clear()
        graph.replay()
        assert same()
        torch.randn(1000, device=DEV).sum().item()


def test_gradients_against_differences():
    """d(sum dy y) along a direction of x and of both weights by central differences in 64 bits: the truncation is below
    e^2 / 6 times the third derivative, estimated from the differences at 2 e; the kernels' rounding 2^-7 of the sum of
    magnitudes."""
    announce("gated differences")
    c = Case(20, 32, 48, seed=12)
    d = c.device()
    c.forward(d)
    c.backward(d)
    torch.cuda.synchronize()
    rng = np.random.default_rng(1)
    base = {w: getattr(c, w).double().numpy() for w in ("x", "wg", "wu")}
    dy = c.dy.double().numpy()
    for w in base:
        way = rng.choice([-1.0, 1.0], size=base[w].shape)

        def slope(e):
            total = [np.sum(dy * F.gated(*[{**base, w: base[w] + s * e * way}[o] for o in ("x", "wg", "wu")], c.act)[0])
                     for s in (1, -1)]
            return (total[0] - total[1]) / (2 * e)

        near, far = slope(2.0 ** -10), slope(2.0 ** -9)
        got = d["d" + w].double().cpu().numpy()
        tol = abs(near - far) + 1e-9 * abs(near) + 2.0 ** -7 * np.sum(np.abs(got))
        assert abs(np.sum(got * way) - near) <= tol, w
        # entry by entry, which a sign or a transposition would show
        for at in [tuple(rng.integers(0, s) for s in base[w].shape) for _ in range(12)]:
            one = np.zeros(base[w].shape)
            one[at] = 2.0 ** -10
            ends = [np.sum(dy * F.gated(*[{**base, w: base[w] + s * one}[o] for o in ("x", "wg", "wu")], c.act)[0]) for s in (1, -1)]
            diff = (ends[0] - ends[1]) / 2.0 ** -9
            assert abs(got[at] - diff) <= 2.0 ** -6 * np.abs(got).max(), (w, at)


def test_weights_behind_2_to_32_bytes():
    """Weights and their gradients of 4.6 GB each: rows at both ends against torch in 64 bits on the GPU."""
    announce("gated 2^32")
    n, f, k = 24, 140001, 16392
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    wg, wu = (torch.empty(f, k, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for w in (wg, wu):
        for i in range(0, f, 20000):
            w[i:i + 20000] = torch.randn(min(20000, f - i), k, generator=g, device=DEV) / 128
    x = torch.randn(n, k, generator=g, device=DEV).bfloat16()
    dy = torch.randn(n, f, generator=g, device=DEV).bfloat16()
    y, dx, dwg, dwu = torch.empty_like(dy), torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    pre = torch.empty(2, n, f, device=DEV)
    ws = torch.empty(T.swz_gated_workspace(n, f, k), dtype=torch.uint8, device=DEV)
    T.swz_gated(x, wg, wu, y, n, f, k, pre=pre)
    T.swz_gated_grad(x, wg, wu, dy, dx, dwg, dwu, n, f, k, ws, pre=pre)
    rows = torch.tensor([0, 1, 7, 65536, 130999, 131071, 131072, f - 2, f - 1], device=DEV)
    zg, zu = x.double() @ wg[rows].double().t(), x.double() @ wu[rows].double().t()
    s = torch.sigmoid(zg)
    a, da = zg * s, s * (1 + zg * (1 - s))
    e = (k + 2) * U * (x.double().abs() @ torch.maximum(wg[rows].double().abs(), wu[rows].double().abs()).t())
    rel = 2.0 ** -8 + 32 * U
    assert bool(((y[:, rows].double() - a * zu).abs() <= rel * (a * zu).abs() + 1.3 * e * (1 + zg.abs() + zu.abs() + e)).all())
    d = dy[:, rows].double()
    dg, du = d * zu * da, d * a
    for got, z in ((dwg, dg), (dwu, du)):
        err = e * d.abs() * (2 + zg.abs() + zu.abs()) + rel * z.abs()
        tol = (err + z.abs() * (n + 40) * U).t() @ x.double().abs()
        ref = z.t() @ x.double()
        assert bool(((got[rows].double() - ref).abs() <= tol * (1 + 2.0 ** -7) + 2.0 ** -8 * ref.abs()).all())
    ref, tol = torch.zeros(n, k, dtype=torch.float64, device=DEV), torch.zeros(n, k, dtype=torch.float64, device=DEV)
    for i in range(0, f, 20000):
        at = slice(i, i + 20000)
        zg, zu, d = pre[0, :, at].double(), pre[1, :, at].double(), dy[:, at].double()
        s = torch.sigmoid(zg)
        dg, du = d * zu * s * (1 + zg * (1 - s)), d * zg * s
        ref += dg @ wg[at].double() + du @ wu[at].double()
        tol += dg.abs() @ wg[at].double().abs() + du.abs() @ wu[at].double().abs()
    # dg and du off by a rounding and by 64 u (1 + |z|) from the kept products; the sum in fp32 parts
    assert bool(((dx.double() - ref).abs() <= (2.0 ** -8 + 2 * f * U) * tol + 2.0 ** -8 * ref.abs()).all())
