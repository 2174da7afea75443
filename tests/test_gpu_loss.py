"""Output-layer losses on the GPU against their 64-bit definitions.

Tolerances, to first order, from the operations (u = 2^-23 bounds one fp32
operation, half of it where it rounds to nearest):

* a logit: k products summed in fp32, (k + 2) u sum |h||w|;
* lse: the largest logit's error, the exponent's argument (three operations
  on numbers up to |z| / tau + |lse|), and a sum of positive terms in at most
  512 steps;
* dz: its softmax part carries lse's and the logit's errors as relative ones,
  then one rounding to fp16 (2^-11 of the value, or 2^-25 of fp16's unit 2^-14
  of the largest upstream below the normal range);
* H and W widened to fp16: 2^-40 of the largest where not exact;
* gradients: fp32 sums of v (or n) products, one rounding to the result's
  type (2^-8 bf16, 2^-11 fp16; below their normal ranges 2^-134 and 2^-25).
"""

import numpy as np
import pytest

from oracle import products as P

import torch

import tiled_movement_amd as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -23
DT = {"bf16": (torch.bfloat16, T.X_BF16, 2.0 ** -8, 2.0 ** -134), "fp16": (torch.float16, T.X_F16, 2.0 ** -11, 2.0 ** -25)}


def announce(*what):
    print("case:", *what, flush=True)


class Case:
    def __init__(self, n, v, k, dt="bf16", top=0, tau=1.0, seed=0, scale=1.5, absent=0.2):
        self.n, self.v, self.k, self.dt, self.top, self.tau = n, v, k, dt, top, tau
        rng = np.random.default_rng(seed)
        t = DT[dt][0]
        self.h = torch.from_numpy(rng.standard_normal((n, k))).to(t)
        self.w = torch.from_numpy(rng.standard_normal((v, k)) * scale / np.sqrt(k)).to(t)
        shape = (n, max(top, 1))
        self.index = rng.integers(0, v, size=shape)
        self.index[rng.random(shape) < absent] = rng.choice([-100, -1, v, v + 5, -2**62])
        self.teacher = None
        if top:
            self.teacher = (rng.standard_normal(shape) * 3).astype(np.float32)
            if top > 2:
                self.teacher[rng.random(shape) < 0.1] = -np.inf
                self.index[0, 1] = self.index[0, 0]  # a word listed twice
        self.upstream = (rng.standard_normal(n) * 10.0 ** rng.uniform(-3, 1, n)).astype(np.float32)

    def device(self):
        d = {"h": self.h.to(DEV), "w": self.w.to(DEV), "index": torch.from_numpy(self.index).to(DEV),
             "upstream": torch.from_numpy(self.upstream).to(DEV)}
        if self.top:
            d["teacher"] = torch.from_numpy(self.teacher).to(DEV)
        n, v, k, top = self.n, self.v, self.k, max(self.top, 1)
        f = lambda *s: torch.full(s, float("nan"), dtype=torch.float32, device=DEV)  # noqa: E731
        d.update(loss=f(n), lse=f(n), zt=f(n, top), dh=torch.full_like(d["h"], float("nan")),
                 dw=torch.full_like(d["w"], float("nan")))
        d["ws"] = torch.full((T.swz_linear_loss_workspace(n, v, k, top, grad=True),), 0xFF, dtype=torch.uint8, device=DEV)
        return d

    def forward(self, d):
        c = DT[self.dt][1]
        if self.top:
            T.swz_linear_distill(d["h"], d["w"], d["index"], d["teacher"], d["loss"], d["lse"], d["zt"], self.n, self.v, self.k,
                                 self.top, self.tau, d["ws"], x_type=c)
        else:
            T.swz_linear_ce(d["h"], d["w"], d["index"], d["loss"], d["lse"], d["zt"], self.n, self.v, self.k, d["ws"], x_type=c)

    def backward(self, d, dh=True, dw=True):
        c = DT[self.dt][1]
        a = (d["dh"] if dh else None, d["dw"] if dw else None)
        if self.top:
            T.swz_linear_distill_grad(d["h"], d["w"], d["index"], d["teacher"], d["lse"], d["zt"], d["upstream"], *a, self.n,
                                      self.v, self.k, self.top, self.tau, d["ws"], x_type=c)
        else:
            T.swz_linear_ce_grad(d["h"], d["w"], d["index"], d["lse"], d["zt"], d["upstream"], *a, self.n, self.v, self.k, d["ws"],
                                 x_type=c)

    def check(self, d):
        h, w = self.h.double().numpy(), self.w.double().numpy()
        ref = P.linear_loss(h, w, self.index, self.teacher, self.tau, self.upstream)
        g = {x: d[x].double().cpu().numpy() for x in ("loss", "lse", "zt", "dh", "dw")}
        ez = (self.k + 2) * U * (np.abs(h) @ np.abs(w).T) / self.tau  # [n][v], of z / tau
        z = (h @ w.T) / self.tau
        size = np.abs(z).max(axis=1) + np.abs(ref["lse"])
        elog = ez.max(axis=1) + 4 * U * size + 520 * U
        assert np.all(np.abs(g["lse"] - ref["lse"]) <= elog)
        here = (self.index >= 0) & (self.index < self.v)
        if self.top:
            here &= self.teacher > -np.inf
        zt = np.where(here, np.take_along_axis(z, np.where(here, self.index, 0), axis=1), 0.0) * self.tau
        assert np.all(np.abs(g["zt"] - zt) <= np.where(here, self.tau * ez.max(axis=1, keepdims=True), 0.0))
        counts = here.any(axis=1)
        teach = 0.0
        if self.top:  # t / tau, its exponential, and the joined sums
            big = np.where(here, np.abs(np.where(here, self.teacher, 0.0)) / self.tau, 0.0).max(axis=1)
            teach = (6 * big + self.top + 16) * U
        eloss = self.tau ** 2 * (elog + ez.max(axis=1) + 4 * U * size + teach * (2 * size + 2 + np.log(max(self.top, 1))))
        assert np.all(np.abs(g["loss"] - ref["loss"]) <= np.where(counts, eloss, 0.0))
        # gradients
        step, tiny = DT[self.dt][2], DT[self.dt][3]
        up = np.abs(self.upstream.astype(np.float64)) * self.tau * counts
        p = np.exp(z - ref["lse"][:, None])
        e = (elog + 4 * U * size)[:, None] + ez + 8 * U
        edz = up[:, None] * (2.0 ** -11 * np.abs(p - ref["target"]) + (1 + 2.0 ** -11) * (e * p + (teach[:, None] if self.top else 0.0) * ref["target"] + 4 * U * np.abs(p - ref["target"])))
        edz += counts[:, None] * up.max(initial=0.0) * 2.0 ** -39
        dz = np.abs(ref["dz"])
        wide = 2.0 ** -40 if self.dt == "bf16" else 0.0
        for name, r, left, el, right in (("dh", ref["dh"], dz, edz, np.abs(w)), ("dw", ref["dw"], dz.T, edz.T, np.abs(h))):
            bound = el @ right + (left + el) @ (np.full_like(right, right.max() * wide) + (right.shape[0] + 24) * U * right)
            bound = bound + step * (np.abs(r) + bound) + tiny
            err = np.abs(g[name] - r)
            assert np.all(err <= bound), (name, np.max(err / np.maximum(bound, 1e-300)))
        assert np.all(g["dh"][~counts] == 0)
        return g


SIZES = [(1, 1, 8), (1, 300, 64), (5, 257, 72), (64, 1000, 128), (65, 513, 200), (128, 255, 136), (129, 1025, 136),
         (300, 2000, 256), (257, 256, 1032), (40, 33000, 64)]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("n,v,k", SIZES)
def test_cross_entropy(n, v, k, dt):
    announce("ce", n, v, k, dt)
    c = Case(n, v, k, dt, seed=n + v + k)
    d = c.device()
    c.forward(d)
    c.backward(d)
    torch.cuda.synchronize()
    c.check(d)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("top,tau", [(1, 1.0), (5, 2.0), (64, 0.7), (256, 3.5)])
@pytest.mark.parametrize("n,v,k", [(1, 1, 8), (3, 300, 64), (70, 513, 200), (150, 1025, 136), (300, 2000, 256), (33, 33001, 64)])
def test_distill(n, v, k, top, tau, dt):
    announce("distill", n, v, k, top, tau, dt)
    c = Case(n, v, k, dt, top=top, tau=tau, seed=n + v + k + top)
    d = c.device()
    c.forward(d)
    c.backward(d)
    torch.cuda.synchronize()
    c.check(d)


@pytest.mark.parametrize("top", [0, 4])
def test_no_row_counts(top):
    announce("no row counts", top)
    c = Case(70, 600, 64, top=top, seed=5)
    c.index[:] = -100
    d = c.device()
    c.forward(d)
    c.backward(d)
    torch.cuda.synchronize()
    assert torch.all(d["loss"] == 0) and torch.all(d["dh"] == 0) and torch.all(d["dw"] == 0) and torch.all(d["zt"] == 0)
    assert torch.all(torch.isfinite(d["lse"]))


@pytest.mark.parametrize("tau", [0.5, 1.0, 4.0])
def test_teacher_entries_masked_by_the_lowest_float(tau):
    """Entries at the lowest float have no weight beside others, and equal weights among themselves."""
    announce("lowest float", tau)
    c = Case(20, 300, 64, top=6, tau=tau, seed=13, absent=0.0)
    c.teacher[:] = np.random.default_rng(0).standard_normal(c.teacher.shape)
    low = np.finfo(np.float32).min
    c.teacher[3, 2:] = low
    c.teacher[4, :] = low
    c.teacher[5, 1:] = -np.inf
    d = c.device()
    c.forward(d)
    c.backward(d)
    torch.cuda.synchronize()
    assert torch.all(torch.isfinite(d["loss"])) and torch.all(torch.isfinite(d["dw"]))
    # the same weights without the overflow that the bounds would meet
    c.teacher[3, 2:] = -200 * tau
    c.teacher[4, :] = 0
    c.check(d)


def test_rows_that_do_not_count_may_hold_anything():
    """NaN in a row whose target is absent stays in its lse."""
    announce("nan in an ignored row")
    c = Case(20, 300, 64, seed=6, absent=0.0)
    c.index[3] = -100
    d = c.device()
    d["h"][3] = float("nan")
    c.forward(d)
    c.backward(d)
    torch.cuda.synchronize()
    assert torch.isnan(d["lse"][3]) and d["loss"][3] == 0 and torch.all(d["dh"][3] == 0)
    rest = torch.tensor([i for i in range(20) if i != 3], device=DEV)
    assert torch.all(torch.isfinite(d["loss"][rest])) and torch.all(torch.isfinite(d["dh"][rest]))
    assert torch.all(torch.isfinite(d["dw"]))


@pytest.mark.parametrize("top", [0, 7])
def test_one_gradient_at_a_time_is_the_same(top):
    announce("one gradient", top)
    c = Case(100, 700, 96, top=top, tau=1.0 if not top else 2.0, seed=7)
    d = c.device()
    c.forward(d)
    c.backward(d)
    torch.cuda.synchronize()
    both = d["dh"].clone(), d["dw"].clone()
    d["dh"].fill_(float("nan"))
    c.backward(d, dw=False)
    torch.cuda.synchronize()
    assert torch.equal(d["dh"], both[0]) and torch.equal(d["dw"], both[1])
    d["dw"].fill_(float("nan"))
    c.backward(d, dh=False)
    torch.cuda.synchronize()
    assert torch.equal(d["dw"], both[1])


def test_no_rows():
    announce("n = 0")
    w = torch.randn(50, 16, device=DEV).bfloat16()
    dw = torch.full_like(w, float("nan"))
    raw = T.lib.swz_linear_ce_grad(None, None, T.X_BF16, None, None, None, None, None, dw.data_ptr(), 0, 50, 16, None, 0,
                                   torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert raw == 0 and torch.all(dw == 0)


@pytest.mark.parametrize("scale", [1e-30, 1.0, 1e3, 1e30])
def test_upstream_of_any_size(scale):
    """The largest upstream is taken out before dz is rounded: scaling all of it by a power of two scales dh by it exactly."""
    announce("upstream", scale)
    c = Case(50, 400, 64, seed=8)
    d = c.device()
    c.forward(d)
    c.backward(d)
    torch.cuda.synchronize()
    base = d["dh"].double().clone()
    s = 2.0 ** round(np.log2(scale))
    d["upstream"] *= s
    c.backward(d)
    torch.cuda.synchronize()
    assert torch.equal(d["dh"].double(), base * s)


@pytest.mark.parametrize("size,upstream", [(1e-4, 1.0), (1e4, 1.0), (2.0 ** 118, 2.0 ** -60), (2.0 ** -110, 2.0 ** 10)])
def test_operands_far_from_one(size, upstream):
    """Also where the largest operand times the gradient's other factors would leave fp32's range on the way."""
    announce("operand size", size, upstream)
    c = Case(60, 500, 64, seed=9)
    c.upstream = (c.upstream * upstream).astype(np.float32)
    c.h = (c.h.double() * size).to(torch.bfloat16)
    c.w = (c.w.double() / size).to(torch.bfloat16)
    d = c.device()
    c.forward(d)
    c.backward(d)
    torch.cuda.synchronize()
    c.check(d)


def test_confident_rows():
    """Logits hundreds apart: no overflow, and gradients of nearly certain rows keep their digits."""
    announce("confident")
    c = Case(80, 300, 64, seed=10, scale=60.0)
    d = c.device()
    c.forward(d)
    c.backward(d)
    torch.cuda.synchronize()
    c.check(d)


@pytest.mark.parametrize("top", [0, 9])
def test_repeats_streams_and_graphs_give_the_same_bits(top):
    announce("graph", top)
    c = Case(130, 9000, 64, top=top, tau=1.0 if not top else 1.5, seed=11)
    d = c.device()
    c.forward(d)
    c.backward(d)
    torch.cuda.synchronize()
    names = ("loss", "lse", "zt", "dh", "dw")
    want = {x: d[x].clone() for x in names}

    def clear():
        for x in names:
            d[x].fill_(float("nan"))
        d["ws"].fill_(0xFF)
        torch.cuda.synchronize()

    clear()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.forward(d)
        c.backward(d)
    side.synchronize()
    assert all(torch.equal(d[x], want[x]) for x in names)
    clear()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.forward(d)
        c.backward(d)
    for _ in range(3):
        clear()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(d[x], want[x]) for x in names)
        torch.randn(1000, device=DEV).sum().item()
        c.check(d)


def test_gradient_against_differences():
    """d(sum upstream loss) along a direction, by central differences of the kernel's own losses.  H and the step are
    multiples of 2^-6 below 2 (exact in bf16); the third derivative's part is below e^2 / 6 max |dz/de|^3, with logits
    moving by at most sum |w| |dir| per unit."""
    announce("differences")
    c = Case(30, 200, 32, seed=12, absent=0.1)
    rng = np.random.default_rng(1)
    c.h = torch.from_numpy(rng.integers(-60, 61, size=(30, 32)) / 64.0).to(torch.bfloat16)
    c.upstream = np.ones(30, np.float32)
    d = c.device()
    c.forward(d)
    c.backward(d)
    torch.cuda.synchronize()
    direction = rng.choice([-1.0, 1.0], size=(30, 32))
    eps = 2.0 ** -6
    slope = (d["dh"].double().cpu().numpy() * direction).sum(axis=1)
    losses = []
    for sgn in (1, -1):
        hh = (c.h.double().numpy() + sgn * eps * direction)
        t = torch.from_numpy(hh).to(torch.bfloat16)
        assert np.array_equal(t.double().numpy(), hh)
        d["h"] = t.to(DEV)
        c.forward(d)
        torch.cuda.synchronize()
        losses.append(d["loss"].double().cpu().numpy())
    diff = (losses[0] - losses[1]) / (2 * eps)
    w = c.w.double().numpy()
    move = np.abs(w @ direction.T).max(axis=0)
    tol = eps ** 2 / 6 * (2 * move) ** 3 + 64 * 30 * U / eps + 2.0 ** -7 * np.abs(d["dh"].double().cpu().numpy()).sum(axis=1)
    assert np.all(np.abs(diff - slope) <= tol)


def test_vocabulary_behind_2_to_32_bytes():
    """W and dW of 4.6 GB: losses, dh and the first and last rows of dW against torch in 64 bits on the GPU, with the
    tolerances of one rounding of dz (2^-11) and of the result (2^-8), and fp32 sums of k and v products."""
    announce("ce 2^32")
    n, v, k = 8, 140001, 16392
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    w = torch.empty(v, k, dtype=torch.bfloat16, device=DEV)
    for i in range(0, v, 20000):
        w[i:i + 20000] = torch.randn(min(20000, v - i), k, generator=g, device=DEV) / 128
    h = torch.randn(n, k, generator=g, device=DEV).bfloat16()
    target = torch.tensor([0, 131071, 131072, v - 1, -1, 7, 140000, 65536], device=DEV)
    up = torch.full((n,), 0.125, device=DEV)
    f = [torch.empty(n, device=DEV) for _ in range(3)]
    ws = torch.empty(T.swz_linear_loss_workspace(n, v, k, grad=True), dtype=torch.uint8, device=DEV)
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    T.swz_linear_ce(h, w, target, *f, n, v, k, ws)
    T.swz_linear_ce_grad(h, w, target, f[1], f[2], up, dh, dw, n, v, k, ws)
    z = torch.cat([h.double() @ w[i:i + 20000].double().t() for i in range(0, v, 20000)], dim=1)
    lse = torch.logsumexp(z, dim=1)
    counts = target >= 0
    at = target.clamp(min=0)
    loss = torch.where(counts, lse - z[torch.arange(n, device=DEV), at], 0.0)
    ez = (k + 2) * U * (h.double().abs().sum(1) * w.abs().max().double()).max().item() + 1100 * U
    assert (f[1].double() - lse).abs().max().item() <= ez and (f[0].double() - loss).abs().max().item() <= 2 * ez
    p = torch.exp(z - lse[:, None])
    p[torch.arange(n, device=DEV), at] -= 1
    dz = torch.where(counts[:, None], 0.125 * p, 0.0)
    rel = 2.0 ** -11 + 2 * ez + 2.0 ** -8
    rows = torch.tensor([0, 1, 7, 65536, 131071, 131072, v - 2, v - 1], device=DEV)
    ref, size = dz[:, rows].t() @ h.double(), dz[:, rows].t().abs() @ h.double().abs()
    assert bool(((dw[rows].double() - ref).abs() <= rel * size + 1e-30).all())
    ref = sum(dz[:, i:i + 20000] @ w[i:i + 20000].double() for i in range(0, v, 20000))
    size = sum(dz[:, i:i + 20000].abs() @ w[i:i + 20000].double().abs() for i in range(0, v, 20000))
    assert bool(((dh.double() - ref).abs() <= rel * size + 1e-30).all())


def test_layer_and_loss_as_a_step():
    """The 8-bit layer, the loss on its output, and back through both: what a training step runs."""
    announce("step")
    rng = np.random.default_rng(30)
    tok, hid, v = 200, 256, 1111
    x = torch.from_numpy(rng.standard_normal((tok, hid))).bfloat16().to(DEV)
    w1 = torch.from_numpy(rng.standard_normal((hid, hid)) / 16).float().to(DEV)
    w2 = torch.from_numpy(rng.standard_normal((v, hid)) / 16).bfloat16().to(DEV)
    target = torch.from_numpy(rng.integers(0, v, tok)).to(DEV)
    u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device=DEV)  # noqa: E731
    xq, xs, xt, xts = u8(tok, hid), u8(tok, 2), u8(hid, 208), u8(hid, 2)
    wq, wsc, wt, wts = u8(hid, hid), u8(2, 2), u8(hid, hid), u8(2, 2)
    T.swz_quant_f8(x, xq, xs, tok, hid, qt=xt, scale_t=xts)
    T.swz_quant_f8(w1, wq, wsc, hid, hid, x_type=T.X_F32, block=T.BLOCK_128X128, qt=wt, scale_t=wts)
    h = torch.empty(tok, hid, dtype=torch.bfloat16, device=DEV)
    T.swz_gemm_f8(xq, xs, wq, wsc, h, tok, hid, hid)
    ws = u8(T.swz_linear_loss_workspace(tok, v, hid, grad=True))
    loss, lse, zt = (torch.empty(tok, device=DEV) for _ in range(3))
    dh, dw2 = torch.empty_like(h), torch.empty_like(w2)
    up = torch.full((tok,), 1 / tok, device=DEV)
    T.swz_linear_ce(h, w2, target, loss, lse, zt, tok, v, hid, ws)
    T.swz_linear_ce_grad(h, w2, target, lse, zt, up, dh, dw2, tok, v, hid, ws)
    gq, gs, gt, gts = u8(tok, hid), u8(tok, 2), u8(hid, 208), u8(hid, 2)
    T.swz_quant_f8(dh, gq, gs, tok, hid, f8_type=T.F8_E5M2, qt=gt, scale_t=gts)
    dx, dw1 = torch.empty_like(x), torch.empty_like(w1)
    T.swz_gemm_f8(gq, gs, wt, wts, dx, tok, hid, hid, a_type=T.F8_E5M2)
    T.swz_gemm_f8(gt, gts, xt, xts, dw1, hid, hid, tok, a_type=T.F8_E5M2, b_block=T.BLOCK_1X128, c_type=T.C_F32)
    torch.cuda.synchronize()
    hd = h.double().cpu().numpy()
    ref = P.linear_loss(hd, w2.double().cpu().numpy(), target.cpu().numpy(), None, 1.0, np.full(tok, 1 / tok))
    assert np.abs(loss.double().cpu().numpy() - ref["loss"]).max() < 1e-4
    for got, r in ((dh, ref["dh"]), (dw2, ref["dw"])):
        assert np.linalg.norm(got.double().cpu().numpy() - r) <= 2.0 ** -8 * np.linalg.norm(r)
    deq = lambda q, s, c, kind, sq: P.dequantize(q.cpu().numpy()[:, :c], kind, s.cpu().numpy(), sq)  # noqa: E731
    rdx = deq(gq, gs, hid, "e5m2", False) @ deq(wt, wts, hid, "e4m3", True).T
    rdw = deq(gt, gts, tok, "e5m2", False) @ deq(xt, xts, tok, "e4m3", False).T
    assert np.linalg.norm(dx.double().cpu().numpy() - rdx) <= 2.0 ** -8 * np.linalg.norm(rdx)
    assert np.linalg.norm(dw1.double().cpu().numpy() - rdw) <= 2.0 ** -18 * np.linalg.norm(rdw)
