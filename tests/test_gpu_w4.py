"""4-bit weights on the GPU: the quantizer bit for bit, products against 64 bits.

A product's terms are x (16 + code), summed in fp32, less (16 + zero) times the sum of x, times the scale: to first order
(u = 2^-23 bounds an fp32 operation) the result is off by (k + 16) u sum |x| (32 + zero) scale, then by one rounding
(2^-8 bf16, 2^-11 fp16; below their normal ranges 2^-134 and 2^-25).
"""

import numpy as np
import pytest

from oracle import feed_forward as F

import torch

import tiled_movement_amd as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -23
DT = {"bf16": (torch.bfloat16, T.X_BF16, 2.0 ** -8, 2.0 ** -134), "fp16": (torch.float16, T.X_F16, 2.0 ** -11, 2.0 ** -25),
      "fp32": (torch.float32, T.X_F32, None, None)}
ACT = {"silu": T.ACT_SILU, "gelu": T.ACT_GELU, "gelu_tanh": T.ACT_GELU_TANH}


def announce(*what):
    print("case:", *what, flush=True)


def rounder(dt):
    return lambda a: torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DT[dt][0]).float().numpy()


def quantize(w, group, st="bf16", wt="bf16", zero=False):
    """The kernel's (q, scale, zero) of a CPU tensor, in buffers with guards behind them."""
    n, k = w.shape
    groups = -(-k // group)
    q = torch.full((n * k // 2 + 16,), 0xA5, dtype=torch.uint8, device=DEV)
    s = torch.full((n * groups + 8,), 7.0, dtype=DT[st][0], device=DEV)
    z = torch.full((n * groups + 16,), 0xA5, dtype=torch.uint8, device=DEV) if zero else None
    T.swz_quant_w4(w.to(DEV), q, s, n, k, group=group, w_type=DT[wt][1], x_type=DT[st][1], zero=z)
    torch.cuda.synchronize()
    assert bool((q[n * k // 2:] == 0xA5).all()) and bool((s[n * groups:] == 7).all())
    assert z is None or bool((z[n * groups:] == 0xA5).all())
    return q[:n * k // 2].view(n, k // 2), s[:n * groups].view(n, groups), None if z is None else z[:n * groups].view(n, groups)


def check_quantizer(w, group, st, wt, zero):
    q, s, z = (None if t is None else t.cpu() for t in quantize(w, group, st, wt, zero))
    code, scale, zp = F.quant_w4(w.float().numpy(), group, zero, rounder(st))
    assert np.array_equal(s.float().numpy(), scale, equal_nan=True)
    assert np.array_equal(F.unpack_w4(q.numpy()), code)
    assert z is None or np.array_equal(z.numpy(), zp)
    return q, s, z


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("st", ["bf16", "fp16"])
@pytest.mark.parametrize("wt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,k,group", [(1, 32, 32), (1, 32, 128), (3, 96, 64), (7, 160, 128), (130, 352, 32), (65, 1056, 128),
                                       (257, 64, 64)])
def test_quantizer(n, k, group, wt, st, zero):
    announce("quant", n, k, group, wt, st, zero)
    rng = np.random.default_rng(n + k)
    w = torch.from_numpy(rng.standard_normal((n, k)) * 10.0 ** rng.uniform(-2, 1, (n, 1))).to(DT[wt][0])
    w[0, :32] = 0.0  # a group of zeros (or the part of one)
    check_quantizer(w, group, st, wt, zero)


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("st", ["bf16", "fp16"])
@pytest.mark.parametrize("wt", ["bf16", "fp16", "fp32"])
def test_quantizer_on_values_halfway_between_codes(wt, st, zero):
    """Multiples of half a scale: the quotients that a rounding the other way would show."""
    announce("quant halves", wt, st, zero)
    rng = np.random.default_rng(4)
    n, k = 512, 128
    half = torch.from_numpy(2.0 ** rng.integers(-12, 4, (n, 1)) * rng.integers(1, 17, (n, 1)))
    w = half * torch.from_numpy(rng.integers(-14, 15, (n, k)).astype(np.float64))
    w[:, 0], w[:, 64] = 14 * half[:, 0], (-16 if zero else 14) * half[:, 0]
    w = w.to(DT[wt][0])
    check_quantizer(w, 64, st, wt, zero)


@pytest.mark.parametrize("zero", [False, True])
def test_quantizer_far_values(zero):
    """Subnormal and huge groups, infinities and NaN, one sign only, scales that leave fp16."""
    announce("quant far", zero)
    for wt in ("bf16", "fp16", "fp32"):
        big = {"bf16": 3.3e38, "fp16": 6.5e4, "fp32": 3.4e38}[wt]
        small = {"bf16": 1e-40, "fp16": 6e-8, "fp32": 1e-44}[wt]
        rng = np.random.default_rng(6)
        w = torch.from_numpy(rng.uniform(-1, 1, (14, 64)))
        for row, v in enumerate((big, small, 1e-30, 1e30, big / 4, 7e5)):
            w[row] *= v
        w[6] = w[6].abs()
        w[7] = -w[7].abs()
        w[8, 3] = float("inf")
        w[9, 40] = -float("inf")
        w[10, 63] = float("nan")
        w[11] = -0.0
        w = w.to(DT[wt][0])
        for st in ("bf16", "fp16"):
            check_quantizer(w, 32, st, wt, zero)


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("n,k,group", [(1, 32, 32), (5, 96, 64), (33, 416, 128), (100, 288, 32)])
def test_back_to_values(n, k, group, dt, zero):
    announce("dequant", n, k, group, dt, zero)
    rng = np.random.default_rng(k)
    groups = -(-k // group)
    q = torch.from_numpy(rng.integers(0, 256, (n, k // 2), dtype=np.uint8))
    s = torch.from_numpy(rng.standard_normal((n, groups))).to(DT[dt][0])
    z = torch.from_numpy(rng.integers(0, 256, (n, groups), dtype=np.uint8)) if zero else None
    out = torch.full((n * k + 8,), 7.0, dtype=DT[dt][0], device=DEV)
    T.swz_dequant_w4(q.to(DEV), s.to(DEV), out, n, k, group=group, x_type=DT[dt][1], zero=None if z is None else z.to(DEV))
    torch.cuda.synchronize()
    want = torch.from_numpy(F.dequant_w4(q.numpy(), s.double().numpy(), None if z is None else z.numpy(), group)).to(DT[dt][0])
    assert torch.equal(out[:n * k].view(n, k).cpu(), want) and bool((out[n * k:] == 7).all())


class Weights:
    def __init__(self, rng, n, k, group, dt, zero):
        self.n, self.k, self.group = n, k, group
        groups = -(-k // group)
        self.q = torch.from_numpy(rng.integers(0, 256, (n, k // 2), dtype=np.uint8))
        self.s = torch.from_numpy(rng.uniform(0.5, 2, (n, groups)) * rng.choice([1.0, -1.0], (n, groups)) / np.sqrt(k)).to(DT[dt][0])
        self.z = torch.from_numpy(rng.integers(0, 16, (n, groups), dtype=np.uint8)) if zero else None
        self.on = [None if t is None else t.to(DEV) for t in (self.q, self.s, self.z)]

    def product(self, x):
        """(float64 result, first-order bound of its error)."""
        s, z = self.s.double().numpy(), None if self.z is None else self.z.numpy()
        spread = lambda a: np.repeat(np.asarray(a, np.float64), self.group, axis=1)[:, :self.k]  # noqa: E731
        size = np.abs(spread(s)) * (32 + (8 if z is None else spread(z)))
        return x @ F.dequant_w4(self.q.numpy(), s, z, self.group).T, (self.k + 16) * U * (np.abs(x) @ size.T)


def check_gemm(m, n, k, group, dt, zero, act=None, seed=0, x=None, offset=0):
    rng = np.random.default_rng(seed + m + n + k)
    w = [Weights(rng, n, k, group, dt, zero) for _ in range(2 if act else 1)]
    if x is None:
        x = torch.from_numpy(rng.standard_normal((m, k)) * 10.0 ** rng.uniform(-2, 1, (m, 1))).to(DT[dt][0])
    out = torch.full((m * n + 16,), 7.0, dtype=DT[dt][0], device=DEV)
    c = out[offset:offset + m * n].view(m, n)
    if act:
        T.swz_gated_w4(x.to(DEV), *w[0].on[:2], *w[1].on[:2], c, m, n, k, group=group, x_type=DT[dt][1], act=ACT[act],
                       zero_g=w[0].on[2], zero_u=w[1].on[2])
    else:
        T.swz_gemm_w4(x.to(DEV), *w[0].on[:2], c, m, n, k, group=group, x_type=DT[dt][1], zero=w[0].on[2])
    torch.cuda.synchronize()
    assert bool((out[:offset] == 7).all()) and bool((out[offset + m * n:] == 7).all())
    got = c.double().cpu().numpy()
    r, e = w[0].product(x.double().numpy())
    if act:
        u, eu = w[1].product(x.double().numpy())
        a, _ = F.activation(act, r)
        z = np.abs(r) + e
        ea = 1.2 * e + z * (z + 8) * U
        r, e = a * u, np.abs(a) * eu + (np.abs(u) + eu) * ea + 4 * U * np.abs(a * u)
    bound = e + DT[dt][2] * (np.abs(r) + e) + DT[dt][3]
    assert np.all(np.abs(got - r) <= bound), np.max(np.abs(got - r) / bound)
    return got


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 32), (1, 16, 128), (1, 300, 1056), (2, 17, 96), (5, 130, 2080), (16, 40, 224),
                                   (17, 65, 4128), (33, 257, 416), (64, 100, 512), (100, 48, 1184)])
def test_product(m, n, k, dt, group, zero):
    announce("gemm_w4", m, n, k, dt, group, zero)
    check_gemm(m, n, k, group, dt, zero)


@pytest.mark.parametrize("act", F.ACTS)
@pytest.mark.parametrize("dt,zero,group", [("bf16", False, 128), ("fp16", True, 32), ("bf16", True, 64)])
@pytest.mark.parametrize("m,n,k", [(1, 33, 288), (4, 200, 1056), (16, 16, 4096), (30, 70, 352), (70, 33, 128)])
def test_gated_product(m, n, k, dt, zero, group, act):
    announce("gated_w4", m, n, k, dt, group, zero, act)
    check_gemm(m, n, k, group, dt, zero, act)


@pytest.mark.parametrize("offset", [1, 2, 5, 8])
def test_results_at_any_element(offset):
    announce("gemm_w4 offset", offset)
    check_gemm(3, 50, 160, 64, "bf16", False, offset=offset)
    check_gemm(20, 48, 160, 64, "fp16", False, "silu", offset=offset)


def test_rows_are_their_own():
    """Each row's bits are the same whatever stands in the others, NaN and infinities included."""
    announce("gemm_w4 rows")
    rng = np.random.default_rng(3)
    m, n, k = 37, 130, 672
    x = torch.from_numpy(rng.standard_normal((m, k))).to(torch.bfloat16)
    w = Weights(rng, n, k, 64, "bf16", True)

    def run(x):
        c = torch.empty(x.shape[0], n, dtype=torch.bfloat16, device=DEV)
        T.swz_gemm_w4(x.to(DEV), *w.on[:2], c, x.shape[0], n, k, group=64, zero=w.on[2])
        torch.cuda.synchronize()
        return c

    want = run(x)
    y = x.clone()
    y[3, 5], y[20, 671], y[36] = float("nan"), float("inf"), 1e30
    got = run(y)
    keep = [i for i in range(m) if i not in (3, 20, 36)]
    assert torch.equal(got[keep], want[keep])
    assert bool(got[3].isnan().all()) and bool(got[20].isnan().all())
    assert torch.equal(run(x[:16]), want[:16])


def test_nan_scales_reach_their_columns_only():
    announce("gemm_w4 nan scale")
    rng = np.random.default_rng(3)
    w = Weights(rng, 40, 256, 128, "bf16", False)
    x = torch.ones(2, 256, dtype=torch.bfloat16, device=DEV)
    s = w.on[1].clone()
    s[7, 1] = float("nan")
    c = torch.empty(2, 40, dtype=torch.bfloat16, device=DEV)
    T.swz_gemm_w4(x, w.on[0], s, c, 2, 40, 256)
    torch.cuda.synchronize()
    assert bool(c[:, 7].isnan().all()) and int(c.isnan().sum()) == 2


def test_nothing_to_do():
    announce("w4 nothing")
    e = torch.empty(0, dtype=torch.bfloat16, device=DEV)
    c = torch.full((8,), 7.0, dtype=torch.bfloat16, device=DEV)
    w = Weights(np.random.default_rng(0), 4, 64, 32, "bf16", False)
    T.swz_gemm_w4(e, *w.on[:2], c, 0, 4, 64, group=32)
    T.swz_quant_w4(e, w.on[0], w.on[1], 0, 64, group=32)
    torch.cuda.synchronize()
    assert bool((c == 7).all())


def test_weights_behind_2_to_32_bytes():
    """Codes of 4.9 GB, values of 19.7 GB: rows at both ends, quantized, multiplied and turned back."""
    announce("w4 2^32")
    n, k, group = 600001, 16416, 128
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    groups = -(-k // group)
    w = torch.empty(n, k, dtype=torch.bfloat16, device=DEV)
    for i in range(0, n, 50000):
        w[i:i + 50000] = torch.randn(min(50000, n - i), k, generator=g, device=DEV)
    q = torch.empty(n, k // 2, dtype=torch.uint8, device=DEV)
    s = torch.empty(n, groups, dtype=torch.bfloat16, device=DEV)
    T.swz_quant_w4(w, q, s, n, k, group=group)
    x = torch.randn(3, k, generator=g, device=DEV).bfloat16()
    c = torch.empty(3, n, dtype=torch.bfloat16, device=DEV)
    T.swz_gemm_w4(x, q, s, c, 3, n, k, group=group)
    torch.cuda.synchronize()
    rows = [0, 1, 261631, 261632, 261700, 523264, 523300, n - 17, n - 1]
    wr = w[rows].float().cpu().numpy()
    code, scale, _ = F.quant_w4(wr, group, False, rounder("bf16"))
    assert np.array_equal(F.unpack_w4(q[rows].cpu().numpy()), code)
    assert np.array_equal(s[rows].float().cpu().numpy(), scale)
    xd = x.double().cpu().numpy()
    spread = np.repeat(scale.astype(np.float64), group, axis=1)[:, :k]
    r, e = xd @ ((code - 8) * spread).T, (k + 16) * U * (np.abs(xd) @ (40 * spread).T)
    assert np.all(np.abs(c[:, rows].double().cpu().numpy() - r) <= e + 2.0 ** -8 * (np.abs(r) + e))
    T.swz_dequant_w4(q, s, w, n, k, group=group)
    torch.cuda.synchronize()
    want = torch.from_numpy((code - 8) * spread).to(torch.bfloat16)
    assert torch.equal(w[rows].cpu(), want)


def test_streams_and_graphs():
    announce("w4 graph")
    rng = np.random.default_rng(8)
    m, n, k = 9, 200, 1056
    w = [Weights(rng, n, k, 32, "fp16", True) for _ in range(2)]
    src = torch.from_numpy(rng.standard_normal((n, k))).half().to(DEV)
    x = torch.from_numpy(rng.standard_normal((m, k))).half().to(DEV)
    outs = [torch.empty(m, n, dtype=torch.float16, device=DEV) for _ in range(2)]
    q, s = torch.empty(n, k // 2, dtype=torch.uint8, device=DEV), torch.empty(n, k // 32, dtype=torch.float16, device=DEV)
    back = torch.empty_like(src)

    def step():
        T.swz_quant_w4(src, q, s, n, k, group=32, w_type=T.X_F16, x_type=T.X_F16)
        T.swz_gemm_w4(x, q, s, outs[0], m, n, k, group=32, x_type=T.X_F16)
        T.swz_gated_w4(x, *w[0].on[:2], *w[1].on[:2], outs[1], m, n, k, group=32, x_type=T.X_F16, zero_g=w[0].on[2], zero_u=w[1].on[2])
        T.swz_dequant_w4(q, s, back, n, k, group=32, x_type=T.X_F16)

    results = [q, s, back, *outs]
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in results]

    def clear():
        for t in results:
            t.zero_()
        torch.cuda.synchronize()

    clear()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(results, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        clear()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(results, want))
        torch.randn(1000, device=DEV).sum().item()
