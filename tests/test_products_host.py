"""Host-side checks of the 8-bit operand, product and loss calls (no GPU):
refusals return the documented codes before any launch, the workspace is what
the calls take, the binding checks its buffers, and the 64-bit definitions the
GPU tests compare with agree with brute force and with differences."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import products as P

import tiled_movement_amd as T

lib = T.lib
OK, EINVAL, EUNSUP = T.SWZ_OK, T.SWZ_EINVAL, T.SWZ_EUNSUPPORTED
# fake, never dereferenced device addresses, 16 GiB apart
A, B, C, D, E, F, G, H, I, J = (0x700000000000 + i * (1 << 34) for i in range(10))


# ---------------------------------------------------------------- quantizer
QUANT = dict(x=A, x_type=T.X_BF16, rows=100, cols=200, ld_x=200, f8=T.F8_E4M3, block=T.BLOCK_1X128, st=T.SCALE_E8M0, q=B,
             s=C, ld_q=208, qt=D, s_t=E, ld_qt=112)


def quant(**kw):
    a = {**QUANT, **kw}
    return lib.swz_quant_f8(a["x"], a["x_type"], a["rows"], a["cols"], a["ld_x"], a["f8"], a["block"], a["st"], a["q"], a["s"],
                            a["ld_q"], a["qt"], a["s_t"], a["ld_qt"], None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=A + 1), dict(x_type=3), dict(x_type=-1), dict(rows=-1), dict(cols=-1), dict(ld_x=199), dict(f8=2),
    dict(block=2), dict(st=2), dict(q=None, qt=None), dict(s=None), dict(s_t=None), dict(q=B + 8), dict(qt=D + 4),
    dict(ld_q=200), dict(ld_q=192), dict(ld_qt=96), dict(ld_qt=100), dict(st=T.SCALE_F32, s=C + 2),
    dict(st=T.SCALE_F32, s_t=E + 1), dict(q=A + 16), dict(qt=B + 4096), dict(s=B + 100), dict(s_t=D), dict(x=D + 100),
    dict(rows=1 << 62), dict(ld_x=1 << 62), dict(x_type=T.X_F32, x=A + 2), dict(rows=1 << 40, ld_qt=1 << 62),
])
def test_quant_refusals(kw):
    assert quant(**kw) == EINVAL


def test_quant_nothing_to_do_and_too_many_tiles():
    assert quant(rows=0, x=None) == OK
    assert quant(cols=0, ld_x=0, ld_q=0, x=None) == OK
    far = 1 << 50
    assert quant(rows=1 << 31, cols=128, ld_x=128, ld_q=128, ld_qt=1 << 31, q=far, s=2 * far, qt=3 * far, s_t=4 * far) == EUNSUP


# ------------------------------------------------------------------ product
GEMM = dict(a=A, sa=B, b=C, sb=D, c=E, m=100, n=200, k=300, lda=304, ldb=304, at=0, bt=0, ab=0, bb=1, st=T.SCALE_E8M0,
            ct=T.C_BF16)


def gemm(**kw):
    g = {**GEMM, **kw}
    return lib.swz_gemm_f8(*(g[x] for x in ("a", "sa", "b", "sb", "c", "m", "n", "k", "lda", "ldb", "at", "bt", "ab", "bb", "st",
                                            "ct")), None)


@pytest.mark.parametrize("kw", [
    dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(c=None), dict(a=A + 8), dict(b=C + 1), dict(c=E + 1),
    dict(ct=T.C_F32, c=E + 2), dict(m=-1), dict(n=-1), dict(k=-1), dict(lda=296), dict(lda=300), dict(ldb=288), dict(ldb=310),
    dict(at=2), dict(bt=-1), dict(ab=2), dict(bb=-1), dict(st=2), dict(ct=2), dict(st=T.SCALE_F32, sa=B + 2),
    dict(st=T.SCALE_F32, sb=D + 1), dict(c=A + 304 * 99), dict(c=C + 16), dict(c=B + 2), dict(c=D), dict(m=1 << 62),
    dict(n=1 << 62), dict(k=1 << 62, lda=1 << 62, ldb=1 << 62),
])
def test_gemm_refusals(kw):
    assert gemm(**kw) == EINVAL


def test_gemm_limits():
    assert gemm(m=0, c=None) == OK and gemm(n=0, c=None) == OK
    assert gemm(lda=1 << 23) == EUNSUP and gemm(ldb=1 << 23) == EUNSUP
    far = 1 << 50
    assert gemm(n=1 << 26, a=far, sa=2 * far, b=3 * far, sb=4 * far, c=5 * far) == EUNSUP
    assert gemm(m=1 << 20, n=1 << 20, a=far, sa=2 * far, b=3 * far, sb=4 * far, c=5 * far) == EUNSUP


# ------------------------------------------------------------------- losses
def workspace(n, v, k, top=1, grad=1):
    out = ctypes.c_int64(-1)
    return lib.swz_linear_loss_workspace(n, v, k, top, grad, ctypes.byref(out)), out.value


def test_workspace():
    assert workspace(10, 1000, 64)[0] == OK
    for bad in ((-1, 10, 8), (1, 0, 8), (1, 10, 0), (1, 10, 12), (1, 10, 8, 0), (1, 10, 8, 1, 2)):
        assert workspace(*bad)[0] == EINVAL, bad
    for big in ((1 << 22, 10, 8), (1, 1 << 31, 8), (1, 10, 1 << 22), (1, 10, 8, 257), (1 << 21, 1 << 21, 8)):
        assert workspace(*big)[0] == EUNSUP, big
    assert lib.swz_linear_loss_workspace(1, 10, 8, 1, 0, None) == EINVAL
    assert workspace(0, 10, 8, 1, 0) == (OK, 0)
    # far below the logits, and enough for the forward call in the gradient's
    n, v, k = 4096, 131072, 4096
    fwd, both = workspace(n, v, k, 1, 0)[1], workspace(n, v, k, 1, 1)[1]
    assert fwd <= both and fwd * 60 < 4 * n * v and both < 4 * n * v
    assert T.swz_linear_loss_workspace(n, v, k, 1, grad=True) == both
    # every word belongs to a piece, whatever the sizes
    for n in (1, 64, 65, 2000, 4096, 100000):
        for v in (1, 255, 8193, 50001, 128256):
            assert workspace(n, v, 64)[1] > 0


LOSS = dict(h=A, w=B, xt=T.X_BF16, index=C, teacher=D, top=3, tau=2.0, loss=E, lse=F, zt=G, up=H, dh=I, dw=J, n=50, v=700,
            k=64, ws=A + (1 << 40), wsb=None)


def losses(which, **kw):
    a = {**LOSS, **kw}
    top = a["top"] if "distill" in which else 1
    wsb = a["wsb"]
    if wsb is None:
        st, wsb = workspace(max(a["n"], 0), max(a["v"], 1), 64, min(max(top, 1), 256), 1)
    tail = (a["n"], a["v"], a["k"], a["ws"], wsb, None)
    if which == "ce":
        return lib.swz_linear_ce(a["h"], a["w"], a["xt"], a["index"], a["loss"], a["lse"], a["zt"], *tail)
    if which == "ce_grad":
        return lib.swz_linear_ce_grad(a["h"], a["w"], a["xt"], a["index"], a["lse"], a["zt"], a["up"], a["dh"], a["dw"], *tail)
    if which == "distill":
        return lib.swz_linear_distill(a["h"], a["w"], a["xt"], a["index"], a["teacher"], a["top"], a["tau"], a["loss"], a["lse"],
                                      a["zt"], *tail)
    return lib.swz_linear_distill_grad(a["h"], a["w"], a["xt"], a["index"], a["teacher"], a["top"], a["tau"], a["lse"], a["zt"],
                                       a["up"], a["dh"], a["dw"], *tail)


COMMON = [dict(h=None), dict(w=None), dict(h=A + 2), dict(w=B + 8), dict(xt=T.X_F32), dict(xt=7), dict(index=None),
          dict(index=C + 4), dict(lse=None), dict(zt=None), dict(zt=G + 2), dict(n=-1), dict(v=0), dict(k=0), dict(k=60),
          dict(ws=None), dict(ws=A + (1 << 40) + 16), dict(wsb=0), dict(ws=A + 256)]


@pytest.mark.parametrize("which", ["ce", "ce_grad", "distill", "distill_grad"])
def test_loss_refusals(which):
    cases = list(COMMON)
    if "grad" in which:
        cases += [dict(up=None), dict(up=H + 1), dict(dh=None, dw=None), dict(dh=I + 8), dict(dw=J + 2), dict(dh=A + 64),
                  dict(dw=B), dict(dh=J, dw=J), dict(dh=F), dict(wsb=workspace(50, 700, 64, 1, 1)[1] - 4096)]
    else:
        cases += [dict(loss=None), dict(loss=E + 1), dict(loss=F), dict(lse=A), dict(zt=E + 8),
                  dict(wsb=workspace(50, 700, 64, 1, 0)[1] - 1)]
    if "distill" in which:
        cases += [dict(teacher=None), dict(teacher=D + 2), dict(top=0), dict(tau=0.0), dict(tau=-1.0), dict(tau=float("nan")),
                  dict(tau=float("inf"))]
    for kw in cases:
        assert losses(which, **kw) == EINVAL, kw
    for kw in [dict(n=1 << 22, wsb=1 << 45), dict(v=1 << 31, wsb=1 << 45), dict(k=1 << 22, wsb=1 << 45)]:
        assert losses(which, **kw) == EUNSUP, kw
    if "distill" in which:
        assert losses(which, top=257) == EUNSUP
    if "grad" not in which:
        assert losses(which, n=0) == OK


@pytest.mark.parametrize("big", [1 << 31, 1 << 40, 1 << 61, 1 << 62, (1 << 63) - 8])
def test_loss_sizes_of_any_magnitude_are_refused(big):
    """Sizes whose products with an element's bytes leave 64 bits are compared before they are multiplied."""
    for grad in (0, 1):
        assert workspace(1, 10, big, 1, grad)[0] == EUNSUP
        assert workspace(big, 10, 8, 1, grad)[0] == EUNSUP
        assert workspace(1, big, 8, 1, grad)[0] == EUNSUP
        assert workspace(big, big, big, 256, grad)[0] == EUNSUP
    for which in ("ce", "ce_grad", "distill", "distill_grad"):
        for kw in (dict(n=big), dict(v=big), dict(k=big)):
            assert losses(which, wsb=1 << 45, **kw) == EUNSUP, (which, kw)


@pytest.mark.parametrize("which", ["distill", "distill_grad"])
def test_temperatures_at_the_ends_of_the_range(which):
    """Every finite normal temperature is taken (checked with nothing to do), a subnormal one, whose inverse is not, refused."""
    tiny = float(np.finfo(np.float32).tiny)
    nothing = dict(n=0, dw=None) if "grad" in which else dict(n=0)
    for tau in (tiny, 1e-30, 3.4e38, float(np.finfo(np.float32).max)):
        assert losses(which, tau=tau, **nothing) == OK, tau
    for tau in (tiny / 2, 1e-40, float(np.finfo(np.float32).smallest_subnormal)):
        assert losses(which, tau=tau, **nothing) == EINVAL, tau


class FakeCuda:
    is_cuda = True

    def __init__(self, nbytes, esz=2):
        self.nbytes, self.device, self.esz = nbytes, torch.device("cuda:0"), esz

    def is_contiguous(self):
        return True

    def numel(self):
        return self.nbytes // self.esz

    def element_size(self):
        return self.esz

    def data_ptr(self):  # pragma: no cover - reaching here would be a failure of the check
        raise AssertionError("the call reached the library")


def test_binding_checks_its_buffers(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    big = FakeCuda(1 << 24)
    with pytest.raises(ValueError, match="q holds"):
        T.swz_quant_f8(big, FakeCuda(100 * 208 - 16, 1), big, 100, 200)
    with pytest.raises(ValueError, match="scale_t holds"):
        T.swz_quant_f8(big, big, big, 100, 200, qt=big, scale_t=FakeCuda(199, 1))
    with pytest.raises(ValueError, match="scale holds"):
        T.swz_quant_f8(big, big, FakeCuda(100 * 2 * 4 - 4, 4), 100, 200, scale_type=T.SCALE_F32)
    with pytest.raises(ValueError, match="scale_b holds"):
        T.swz_gemm_f8(big, big, big, FakeCuda(5, 1), big, 100, 200, 300)
    with pytest.raises(ValueError, match="c holds"):
        T.swz_gemm_f8(big, big, big, big, FakeCuda(100 * 200 * 2 - 2), 100, 200, 300)
    i64, f32 = FakeCuda(1 << 20, 8), FakeCuda(1 << 20, 4)
    with pytest.raises(ValueError, match="ws holds"):
        T.swz_linear_ce(big, big, i64, f32, f32, f32, 50, 700, 64, FakeCuda(100, 1))
    with pytest.raises(ValueError, match="target has 4-byte elements"):
        T.swz_linear_ce(big, big, f32, f32, f32, f32, 50, 700, 64, big)
    with pytest.raises(ValueError, match="h has 4-byte elements"):
        T.swz_linear_ce_grad(f32, big, i64, f32, f32, f32, None, big, 50, 700, 64, big)
    with pytest.raises(ValueError, match="teacher holds"):
        T.swz_linear_distill(big, big, i64, FakeCuda(596, 4), f32, f32, f32, 50, 700, 64, 3, 1.0, big)
    with pytest.raises(T.SwzError):
        T.swz_linear_ce(big, big, i64, f32, f32, f32, 50, 700, 60, big)


class Typed(FakeCuda):
    """A FakeCuda with an element type."""

    def __init__(self, dtype, nbytes=1 << 24):
        super().__init__(nbytes, dtype.itemsize)
        self.dtype = dtype


BF, HF, FL, F64, BYTE, I16, I32, I64 = (torch.bfloat16, torch.float16, torch.float32, torch.float64, torch.uint8, torch.int16,
                                        torch.int32, torch.int64)
E4, E5, E8 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu


def _call(name, dtypes, **kw):
    """One call of a binding with buffers of the given types, which have to be right but for one."""
    b = {k: None if d is None else Typed(d) for k, d in dtypes.items()}
    if name == "quant":
        T.swz_quant_f8(b["x"], b["q"], b["scale"], 100, 200, qt=b["qt"], scale_t=b["scale_t"], **kw)
    elif name == "gemm":
        T.swz_gemm_f8(b["a"], b["scale_a"], b["b"], b["scale_b"], b["c"], 100, 200, 300, **kw)
    else:
        grad, distill = "grad" in name, "distill" in name
        args = [b["h"], b["w"], b["index" if distill else "target"]] + ([b["teacher"]] if distill else [])
        args += [b["lse"], b["zt"], b["upstream"], b["dh"], b["dw"]] if grad else [b["loss"], b["lse"], b["zt"]]
        args += [50, 700, 64] + ([3, 1.0] if distill else [])
        getattr(T, "swz_linear_" + name)(*args, b["ws"], **kw)


QUANT_T = dict(x=BF, q=BYTE, scale=BYTE, qt=BYTE, scale_t=BYTE)
GEMM_T = dict(a=BYTE, scale_a=BYTE, b=BYTE, scale_b=BYTE, c=BF)
CE_T = dict(h=BF, w=BF, target=I64, loss=FL, lse=FL, zt=FL, ws=BYTE)
CEG_T = dict(h=BF, w=BF, target=I64, lse=FL, zt=FL, upstream=FL, dh=BF, dw=BF, ws=BYTE)
DI_T = dict(h=BF, w=BF, index=I64, teacher=FL, loss=FL, lse=FL, zt=FL, ws=BYTE)
DIG_T = dict(h=BF, w=BF, index=I64, teacher=FL, lse=FL, zt=FL, upstream=FL, dh=BF, dw=BF, ws=BYTE)
WRONG = [("quant", QUANT_T, {}, dict(x=[HF, FL, F64], q=[E5, FL, I16], scale=[FL, HF, I32], qt=[E5, BF], scale_t=[FL, E4])),
         ("quant", QUANT_T, dict(x_type=T.X_F32), dict(x=[BF, HF, F64])),
         ("quant", {**QUANT_T, "x": HF}, dict(x_type=T.X_F16, f8_type=T.F8_E5M2), dict(x=[BF, FL], q=[E4], qt=[E4])),
         ("quant", QUANT_T, dict(scale_type=T.SCALE_F32), dict(scale=[BYTE, HF, F64, E8])),
         ("gemm", GEMM_T, {}, dict(a=[E5, BF, I32], b=[E5, FL], scale_a=[FL, E4, I16], scale_b=[FL], c=[FL, HF, F64])),
         ("gemm", {**GEMM_T, "c": FL}, dict(a_type=T.F8_E5M2, c_type=T.C_F32), dict(a=[E4], c=[BF, F64])),
         ("gemm", {**GEMM_T, "scale_a": FL, "scale_b": FL}, dict(scale_type=T.SCALE_F32), dict(scale_a=[BYTE, F64], scale_b=[E8, HF])),
         ("ce", CE_T, {}, dict(h=[HF, FL, F64], w=[HF, FL], target=[I32, F64, FL], loss=[F64, BF, I64], lse=[F64, HF], zt=[F64])),
         ("ce_grad", CEG_T, {}, dict(h=[HF], w=[HF], target=[I32, F64], lse=[F64], zt=[F64, BF], upstream=[F64, BF, HF], dh=[HF, FL],
                                     dw=[HF, FL])),
         ("ce_grad", {**CEG_T, "h": HF, "w": HF, "dh": HF, "dw": HF}, dict(x_type=T.X_F16), dict(h=[BF], w=[BF], dh=[BF], dw=[BF])),
         ("distill", DI_T, {}, dict(h=[HF], w=[HF], index=[I32, F64], teacher=[F64, BF], loss=[F64], lse=[F64], zt=[F64])),
         ("distill_grad", DIG_T, {}, dict(h=[HF], index=[I32], teacher=[F64], lse=[F64], zt=[F64], upstream=[F64], dh=[HF], dw=[HF]))]


@pytest.mark.parametrize("name,right,kw,wrong", WRONG)
def test_binding_refuses_tensors_of_other_types(monkeypatch, name, right, kw, wrong):
    """A tensor of another type than the call reads there is named, not read as what it is not."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for buf, dtypes in wrong.items():
        for dtype in dtypes:
            types = {**right, buf: dtype}
            if kw.get("scale_type") == T.SCALE_F32:
                types = {**{k: FL for k in right if "scale" in k}, **{k: v for k, v in types.items() if "scale" not in k}, buf: dtype}
            with pytest.raises(ValueError, match=f": {buf} "):
                _call(name, types, **kw)


@pytest.mark.parametrize("name,right,kw,wrong", WRONG)
def test_binding_takes_tensors_of_the_right_types_and_raw_bits(monkeypatch, name, right, kw, wrong):
    """Right types, and integers of their size as raw bits, pass the checks (what comes next, the address, is not asked for)."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    types = {**right}
    if kw.get("scale_type") == T.SCALE_F32:
        types.update({k: FL for k in right if "scale" in k})
    if name == "quant" and kw.get("x_type") == T.X_F32:
        types["x"] = FL
    raw = {1: BYTE, 2: I16, 4: I32, 8: I64}
    f8 = {"q": E4, "qt": E4, "a": E4, "b": E4, "scale": E8, "scale_t": E8, "scale_a": E8, "scale_b": E8}
    named = {k: f8[k] if k in f8 and d == BYTE else d for k, d in types.items()}
    if kw.get("f8_type") == T.F8_E5M2:
        named.update(q=E5, qt=E5)
    if kw.get("a_type") == T.F8_E5M2:
        named["a"] = E5
    for given in (types, {k: raw[d.itemsize] for k, d in types.items()}, named):
        with pytest.raises(AssertionError, match="reached the library"):
            _call(name, given, **kw)


# ---------------------------------------------------------- 64-bit definitions
@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_rounding_picks_the_nearest_value_and_even_on_ties(kind):
    grid = np.unique(P.f8_decode(np.arange(256), kind))
    grid = grid[np.isfinite(grid)]
    assert grid.max() == P.F8[kind][2]
    mids = (grid[1:] + grid[:-1]) / 2
    y = np.concatenate([grid, mids, np.random.default_rng(0).uniform(-1, 1, 4000) * grid.max(),
                        np.random.default_rng(1).standard_normal(4000) * 2.0 ** -8])
    got = P.f8_round(y, kind)
    near = np.abs(grid[None, :] - y[:, None])
    assert np.array_equal(np.abs(got - y), near.min(axis=1))
    codes = {v: c for c, v in enumerate(P.f8_decode(np.arange(128), kind)) if np.isfinite(v)}
    assert all(codes[abs(v)] % 2 == 0 for v in P.f8_round(mids, kind))


def test_blocks_use_the_smallest_scale():
    x = np.random.default_rng(2).standard_normal((130, 300)) * 100
    for kind in P.F8:
        for br in (1, 128):
            q, e = P.quantize(x, kind, br)
            s = np.repeat(np.repeat(2.0 ** e, br, 0)[:130], 128, 1)[:, :300]
            assert np.abs(q).max() <= P.F8[kind][2]
            big = np.array([[np.abs(x[i:i + br, j:j + 128]).max() for j in range(0, 300, 128)] for i in range(0, 130, br)])
            assert np.all(big <= P.F8[kind][2] * 2.0 ** e) and np.all(big > P.F8[kind][2] * 2.0 ** (e - 1))
            step = 2.0 ** -4 if kind == "e4m3" else 2.0 ** -3
            assert np.all(np.abs(q * s - x) <= step * np.abs(x) + s * 2.0 ** (P.F8[kind][1] - P.F8[kind][0] - 1))


@pytest.mark.parametrize("distill", [False, True])
def test_loss_gradients_against_differences(distill):
    rng = np.random.default_rng(3)
    n, v, k = 4, 9, 5
    h, w = rng.standard_normal((n, k)), rng.standard_normal((v, k))
    up = rng.standard_normal(n)
    if distill:
        index, teacher, tau = rng.integers(-1, v + 1, size=(n, 4)), rng.standard_normal((n, 4)), 1.7
        index[0, 1] = index[0, 0] = 2
        index[1] = -1
        teacher[2, 0] = -np.inf
    else:
        index, teacher, tau = np.array([3, -100, 8, 9]), None, 1.0
    f = lambda hh, ww: float(up @ P.linear_loss(hh, ww, index, teacher, tau)["loss"])  # noqa: E731
    g = P.linear_loss(h, w, index, teacher, tau, up)
    eps = 1e-5
    for name, arr, pair in (("dh", h, lambda d: (f(h + d, w), f(h - d, w))), ("dw", w, lambda d: (f(h, w + d), f(h, w - d)))):
        for i in np.ndindex(arr.shape):
            d = np.zeros_like(arr)
            d[i] = eps
            up_, dn = pair(d)
            # the third derivative's part, and the rounding of two losses below 100
            assert abs((up_ - dn) / (2 * eps) - g[name][i]) <= 1e3 * eps ** 2 + 100 * 2.0 ** -52 / eps
