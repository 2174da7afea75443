"""Host checks of the feed-forward calls: every refusal happens before anything reaches the HIP runtime (addresses here
are never dereferenced), the binding's checks of its buffers, and the oracle's own definitions."""

import ctypes
import math
import os

import numpy as np
import pytest

from oracle import feed_forward as F

import torch

import tiled_movement_amd as T

lib = T.lib
OK, EINVAL, EUNSUP = T.SWZ_OK, T.SWZ_EINVAL, T.SWZ_EUNSUPPORTED
A, B, C, D, E, G, H, I, J = (0x7F0000000000 + (i << 32) for i in range(9))
WS = 0x7F0000000000 + (64 << 32)
FAR = 1 << 56
# accepted calls are made only where stand-ins take them
NO_LAUNCH = os.environ.get("SWZ_NO_LAUNCH") == "1"


# -------------------------------------------------------------------- gated
def workspace(n, f, k):
    out = ctypes.c_int64(-1)
    return lib.swz_gated_workspace(n, f, k, ctypes.byref(out)), out.value


GATED = dict(x=A, wg=B, wu=C, xt=T.X_BF16, act=T.ACT_SILU, y=D, pre=E, dy=G, dx=H, dwg=I, dwu=J, n=50, f=70, k=64, ws=WS, wsb=None)


def gated(grad, **kw):
    a = {**GATED, **kw}
    head = (a["x"], a["wg"], a["wu"], a["xt"], a["act"])
    if not grad:
        return lib.swz_gated(*head, a["y"], a["pre"], a["n"], a["f"], a["k"], None)
    wsb = a["wsb"]
    if wsb is None:
        st, wsb = workspace(a["n"], a["f"], a["k"])
        wsb = wsb if st == OK else 1 << 50
    return lib.swz_gated_grad(*head, a["dy"], a["pre"], a["dx"], a["dwg"], a["dwu"], a["n"], a["f"], a["k"], a["ws"], wsb, None)


COMMON = [dict(x=None), dict(wg=None), dict(wu=None), dict(x=A + 8), dict(wg=B + 2), dict(wu=C + 4), dict(xt=T.X_F32), dict(xt=-1),
          dict(act=3), dict(act=-1), dict(n=-1), dict(f=0), dict(k=0), dict(k=60), dict(pre=E + 2)]


def test_gated_refusals():
    for kw in COMMON + [dict(y=None), dict(y=D + 1), dict(y=A), dict(y=B + 64), dict(y=C), dict(pre=D + 50 * 70), dict(pre=A),
                        dict(y=E + 8 * 50 * 70 - 2)]:
        assert gated(False, **kw) == EINVAL, kw
    assert gated(False, n=0, x=None, y=None) == OK


def test_gated_grad_refusals():
    for kw in COMMON + [dict(dy=None), dict(dy=G + 1), dict(dx=None, dwg=None, dwu=None), dict(dx=H + 8), dict(dwg=I + 2),
                        dict(dwu=J + 8), dict(dx=A), dict(dwg=I, dwu=I), dict(dwg=I, dwu=I + 64 * 70), dict(dwg=B), dict(dx=G),
                        dict(dx=E + 160), dict(ws=None), dict(ws=WS + 128), dict(ws=A), dict(ws=I + 256),
                        dict(wsb=workspace(50, 70, 64)[1] - 1), dict(wsb=0)]:
        assert gated(True, **kw) == EINVAL, kw


@pytest.mark.parametrize("big", [(1 << 22) - 8, 1 << 31, 1 << 40, 1 << 62, (1 << 63) - 8])
def test_gated_sizes_of_any_magnitude_are_refused(big):
    for kw in (dict(n=big), dict(f=big), dict(k=big)):
        assert gated(False, **kw) == EUNSUP and gated(True, **kw) == EUNSUP, kw
        sizes = {**dict(n=1, f=1, k=8), **kw}
        assert workspace(**sizes)[0] == EUNSUP


def test_gated_workspace():
    for bad in ((-1, 10, 8), (1, 0, 8), (1, 10, 0), (1, 10, 12)):
        assert workspace(*bad)[0] == EINVAL, bad
    for many in ((1 << 21, 1 << 20, 8), (8, 1 << 20, 1 << 21), (1 << 21, 8, 1 << 21)):
        assert workspace(*many)[0] == EUNSUP, many
    assert lib.swz_gated_workspace(1, 10, 8, None) == EINVAL
    for n in (0, 1, 63, 64, 65, 300, 4096, 100000):
        for f in (1, 127, 4096, 50001):
            for k in (8, 1000, 4096):
                st, b = workspace(n, f, k)
                # dg and du, twice of each for small products, and at most 32 parts of 256 tiles' sums
                terms = 2 if n * f * k <= 1 << 23 else 1
                assert st == OK and 4 * terms * n * f <= b <= 4 * terms * n * (f + 8) + 4 * 32 * 256 * 256 * 256 + 4096
    assert T.swz_gated_workspace(4096, 8192, 4096) == workspace(4096, 8192, 4096)[1]


# ------------------------------------------------------------ 4-bit weights
W4 = dict(w=A, wt=T.X_BF16, n=40, k=96, group=64, xt=T.X_BF16, q=B, s=C, z=D)


def quant(back=False, **kw):
    a = {**W4, **kw}
    if back:
        return lib.swz_dequant_w4(a["q"], a["s"], a["z"], a["n"], a["k"], a["group"], a["xt"], a["w"], None)
    return lib.swz_quant_w4(a["w"], a["wt"], a["n"], a["k"], a["group"], a["xt"], a["q"], a["s"], a["z"], None)


@pytest.mark.parametrize("back", [False, True])
def test_quant_w4_refusals(back):
    cases = [dict(w=None), dict(q=None), dict(s=None), dict(w=A + 8), dict(q=B + 8), dict(s=C + 1), dict(xt=T.X_F32), dict(xt=9),
             dict(n=-1), dict(k=0), dict(k=16), dict(k=80), dict(group=16), dict(group=0), dict(group=256), dict(group=-128),
             dict(q=A), dict(w=C), dict(w=D - 16)]
    # what is written may not overlap; what is only read may
    for kw in cases + ([] if back else [dict(wt=3), dict(wt=-1), dict(z=C + 1), dict(s=B + 2), dict(z=B + 40 * 48 - 1)]):
        assert quant(back, **kw) == EINVAL, kw
    for kw in (dict(n=1 << 30, k=32), dict(n=1 << 62), dict(k=1 << 62), dict(n=1 << 62, k=1 << 62)):
        assert quant(back, **kw) == EUNSUP, kw
    assert quant(back, n=0, w=None, q=None, s=None) == OK


GEMM = dict(x=A, xt=T.X_BF16, act=T.ACT_SILU, q=B, s=C, z=D, q2=E, s2=G, z2=H, group=64, c=I, m=3, n=40, k=96)


def gemm(gated, **kw):
    a = {**GEMM, **kw}
    if gated:
        return lib.swz_gated_w4(a["x"], a["xt"], a["act"], a["q"], a["s"], a["z"], a["q2"], a["s2"], a["z2"], a["group"], a["c"],
                                a["m"], a["n"], a["k"], None)
    return lib.swz_gemm_w4(a["x"], a["xt"], a["q"], a["s"], a["z"], a["group"], a["c"], a["m"], a["n"], a["k"], None)


@pytest.mark.parametrize("two", [False, True])
def test_gemm_w4_refusals(two):
    cases = [dict(x=None), dict(q=None), dict(s=None), dict(c=None), dict(x=A + 2), dict(q=B + 8), dict(s=C + 1), dict(c=I + 1),
             dict(xt=T.X_F32), dict(m=-1), dict(n=-1), dict(k=0), dict(k=48), dict(group=100), dict(c=A), dict(c=B + 2), dict(c=C),
             dict(c=D + 4)]
    if two:
        cases += [dict(q2=None), dict(s2=None), dict(z2=None), dict(z=None), dict(act=7), dict(c=E), dict(c=G), dict(c=H)]
    for kw in cases:
        assert gemm(two, **kw) == EINVAL, kw
    far = dict(x=FAR, q=2 * FAR, s=3 * FAR, z=4 * FAR, q2=5 * FAR, s2=6 * FAR, z2=7 * FAR, c=8 * FAR)
    for kw in (dict(m=1 << 22), dict(m=1 << 62), dict(k=1 << 22), dict(n=1 << 26), dict(n=1 << 62), dict(k=1 << 62),
               dict(n=1 << 25, k=1024)):
        assert gemm(two, **far, **kw) == EUNSUP, kw
    assert gemm(two, m=0, x=None, c=None) == OK and gemm(two, n=0, q=None, c=None) == OK


# --------------------------------------------------------------------- norm
def arrays(at, numel, kind):
    n = len(at)
    return (ctypes.c_void_p * n)(*at), (ctypes.c_int64 * n)(*numel), (ctypes.c_int32 * n)(*kind), n


def norm_workspace(count):
    out = ctypes.c_int64(-1)
    return lib.swz_grad_norm_workspace(count, ctypes.byref(out)), out.value


LIST = ([A, B, C], [100, 7, 5000], [T.X_BF16, T.X_F32, T.X_F16])


def clip(at=LIST[0], numel=LIST[1], kind=LIST[2], out=None, norm=D, ws=WS, wsb=None, max_norm=1.0, which="clip"):
    a = arrays(at, numel, kind)
    if wsb is None:
        wsb = norm_workspace(len(at))[1]
    if which == "norm":
        return lib.swz_grad_norm(*a, norm, ws, wsb, None)
    return lib.swz_clip_grads(a[0], None if out is None else (ctypes.c_void_p * len(out))(*out), *a[1:], max_norm, norm, ws, wsb, None)


@pytest.mark.parametrize("which", ["clip", "norm"])
def test_norm_refusals(which):
    for kw in [dict(at=[A, None, C]), dict(at=[A + 1, B, C]), dict(at=[A, B + 2, C]), dict(numel=[100, -1, 5]), dict(kind=[0, 3, 1]),
               dict(kind=[0, -1, 1]), dict(norm=None), dict(norm=D + 2), dict(ws=None), dict(ws=WS + 4), dict(wsb=16), dict(norm=A + 4),
               dict(norm=WS), dict(ws=A), dict(ws=C + 8)]:
        assert clip(which=which, **kw) == EINVAL, kw
    assert clip(which=which, numel=[1 << 38, 1, 1]) == EUNSUP
    a = arrays(*LIST)
    for i in range(3):
        b = list(a)
        b[i] = None
        assert lib.swz_grad_norm(*b, D, WS, 1 << 30, None) == EINVAL
    for bad in (-1, (1 << 20) + 1):
        assert lib.swz_grad_norm(*a[:3], bad, D, WS, 1 << 30, None) == (EINVAL if bad < 0 else EUNSUP)


def test_clip_refusals():
    for max_norm in (-1.0, float("nan"), -math.inf):
        assert clip(max_norm=max_norm) == EINVAL
    # the same memory twice, whole or in part, in place or to write
    assert clip(at=[A, B, A]) == EINVAL and clip(at=[A, B, A + 198]) == EINVAL
    for out in ([A, A, C], [E, E + 199, G], [E, B + 4, G], [E, G, B], [E, None, G], [E, G + 2, H], [D, G, H], [WS, G, H],
                [A + 16, B, C]):
        assert clip(out=out) == EINVAL, out


@pytest.mark.skipif(not NO_LAUNCH, reason="these calls are accepted: only where stand-ins take them")
def test_accepted_lists():
    assert clip() == OK and clip(which="norm") == OK and clip(max_norm=math.inf) == OK and clip(max_norm=0.0) == OK
    assert clip(out=[A, B, C]) == OK and clip(out=[E, G, H]) == OK and clip(out=[E, B, H]) == OK
    assert clip(which="norm", at=[A, B, A], kind=[0, 2, 0]) == OK  # nothing of it is written
    assert clip(at=[A, B, A + 200]) == OK  # side by side
    assert clip(at=[None, B, C], numel=[0, 7, 5000]) == OK
    assert clip(at=[], numel=[], kind=[], ws=None, wsb=0) == OK
    many = 5000
    assert clip(at=[A + 64 * i for i in range(many)], numel=[16] * many, kind=[2] * many) == OK
    assert clip(at=[A + 64 * i for i in range(many)], numel=[16] * (many - 1) + [17], kind=[2] * many) == OK
    assert clip(at=[A + 64 * (many - i) for i in range(many)], numel=[16] * (many - 1) + [17], kind=[2] * many) == EINVAL


@pytest.mark.skipif(not NO_LAUNCH, reason="these calls are accepted: only where stand-ins take them")
def test_accepted_calls():
    assert gated(False) == OK and gated(False, pre=None) == OK and gated(False, y=D + 2) == OK
    assert gated(True) == OK and gated(True, pre=None) == OK and gated(True, dx=None) == OK and gated(True, dwg=None, dwu=None) == OK
    assert gated(True, n=0, x=None, dy=None, wg=None, wu=None, dx=None) == OK
    assert gated(False, wg=B, wu=B) == OK  # only read
    for back in (False, True):
        assert quant(back) == OK and quant(back, z=None) == OK
    for two in (False, True):
        assert gemm(two) == OK and gemm(two, z=None, z2=None) == OK and gemm(two, m=1000, c=I + 2) == OK
    assert gemm(True, q2=B, s2=C, z2=D) == OK


def test_norm_workspace():
    for count, packs in ((0, 0), (1, 1), (64, 1), (65, 2), (1 << 20, 1 << 14)):
        assert norm_workspace(count) == (OK, packs * 16384)
    assert norm_workspace(-1)[0] == EINVAL and norm_workspace((1 << 20) + 1)[0] == EUNSUP
    assert lib.swz_grad_norm_workspace(1, None) == EINVAL


# ------------------------------------------------------------------ binding
class Typed:
    is_cuda = True

    def __init__(self, dtype, nbytes=1 << 24, device="cuda:0", contiguous=True):
        self.dtype, self.nbytes, self.device, self.contiguous = dtype, nbytes, torch.device(device), contiguous

    def is_contiguous(self):
        return self.contiguous

    def numel(self):
        return self.nbytes // self.dtype.itemsize

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        raise AssertionError("the call reached the library")


class Placed(Typed):
    def __init__(self, at, dtype, nbytes, **kw):
        super().__init__(dtype, nbytes, **kw)
        self.at = at

    def data_ptr(self):
        return self.at


BF, HF, FL, F64, BYTE, I8, I32 = (torch.bfloat16, torch.float16, torch.float32, torch.float64, torch.uint8, torch.int8, torch.int32)
CALLS = {
    "gated": (dict(x=BF, wg=BF, wu=BF, y=BF, pre=FL),
              lambda b, kw: T.swz_gated(b["x"], b["wg"], b["wu"], b["y"], 50, 70, 64, pre=b["pre"], **kw),
              dict(x=2 * 50 * 64, wg=2 * 70 * 64, wu=2 * 70 * 64, y=2 * 50 * 70, pre=8 * 50 * 70)),
    "gated_grad": (dict(x=BF, wg=BF, wu=BF, dy=BF, pre=FL, dx=BF, dwg=BF, dwu=BF, ws=BYTE),
                   lambda b, kw: T.swz_gated_grad(b["x"], b["wg"], b["wu"], b["dy"], b["dx"], b["dwg"], b["dwu"], 50, 70, 64,
                                                  b["ws"], pre=b["pre"], **kw),
                   dict(x=2 * 50 * 64, dy=2 * 50 * 70, pre=8 * 50 * 70, dx=2 * 50 * 64, dwg=2 * 70 * 64, dwu=2 * 70 * 64)),
    "quant_w4": (dict(w=BF, q=BYTE, scale=BF, zero=BYTE),
                 lambda b, kw: T.swz_quant_w4(b["w"], b["q"], b["scale"], 40, 96, group=64, zero=b["zero"], **kw),
                 dict(w=2 * 40 * 96, q=40 * 48, scale=2 * 40 * 2, zero=40 * 2)),
    "dequant_w4": (dict(q=BYTE, scale=BF, w=BF, zero=BYTE),
                   lambda b, kw: T.swz_dequant_w4(b["q"], b["scale"], b["w"], 40, 96, group=64, zero=b["zero"], **kw),
                   dict(w=2 * 40 * 96, q=40 * 48, scale=2 * 40 * 2, zero=40 * 2)),
    "gemm_w4": (dict(x=BF, q=BYTE, scale=BF, c=BF, zero=BYTE),
                lambda b, kw: T.swz_gemm_w4(b["x"], b["q"], b["scale"], b["c"], 3, 40, 96, group=64, zero=b["zero"], **kw),
                dict(x=2 * 3 * 96, q=40 * 48, scale=2 * 40 * 2, c=2 * 3 * 40, zero=40 * 2)),
    "gated_w4": (dict(x=BF, q_g=BYTE, scale_g=BF, q_u=BYTE, scale_u=BF, c=BF, zero_g=BYTE, zero_u=BYTE),
                 lambda b, kw: T.swz_gated_w4(b["x"], b["q_g"], b["scale_g"], b["q_u"], b["scale_u"], b["c"], 3, 40, 96, group=64,
                                              zero_g=b["zero_g"], zero_u=b["zero_u"], **kw),
                 dict(x=2 * 3 * 96, q_g=40 * 48, scale_u=2 * 40 * 2, c=2 * 3 * 40, zero_u=40 * 2)),
}


@pytest.mark.parametrize("name", CALLS)
def test_binding_checks_its_buffers(monkeypatch, name):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    types, call, need = CALLS[name]
    with pytest.raises(AssertionError, match="reached the library"):
        call({k: Typed(t) for k, t in types.items()}, {})
    for buf, size in need.items():
        b = {k: Typed(t) for k, t in types.items()}
        b[buf] = Typed(types[buf], size - types[buf].itemsize)
        with pytest.raises(ValueError, match=f"{buf} holds"):
            call(b, {})
        b[buf] = Typed(types[buf], size)
        with pytest.raises(AssertionError, match="reached the library"):
            call(b, {})
        for wrong in (HF, FL, F64, I32, I8):
            if wrong == types[buf] or (wrong.itemsize == types[buf].itemsize and not wrong.is_floating_point):
                continue
            b[buf] = Typed(wrong)
            with pytest.raises(ValueError, match=f": {buf} "):
                call(b, {})
        b[buf] = Typed(types[buf], device="cuda:1")
        with pytest.raises(ValueError, match="is on cuda|on cuda:1"):
            call(b, {})
        b[buf] = Typed(types[buf], contiguous=False)
        with pytest.raises(ValueError, match="contiguous"):
            call(b, {})
    half = {k: Typed(HF if t == BF else t) for k, t in types.items()}
    if name == "quant_w4":
        half["w"] = Typed(BF)
    with pytest.raises(AssertionError, match="reached the library"):
        call(half, {"x_type": T.X_F16})


def test_binding_reports_the_library():
    with pytest.raises(T.SwzError):
        T.swz_gated_workspace(10, 10, 12)
    with pytest.raises(T.SwzError):
        T.swz_gemm_w4(A, B, C, D, 3, 40, 96, group=48)


def test_binding_checks_tensor_lists(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    ok = [Placed(A, BF, 200), Typed(FL)]
    norm, ws = Typed(FL, 8), Typed(BYTE)
    with pytest.raises(AssertionError, match="reached the library"):
        T.swz_grad_norm(ok, norm, ws)
    for bad, text in ((Typed(F64), "tensor 1 is not"), (Typed(I32), "tensor 1 is not"), (torch.zeros(3), "tensor 1 must be a CUDA"),
                      (Typed(BF, contiguous=False), "tensor 1 must be contiguous"), (Typed(BF, device="cuda:1"), "tensor 1 is on cuda:1"),
                      (A, "tensor 1 is not")):
        for call in (lambda t: T.swz_grad_norm(t, norm, ws), lambda t: T.swz_clip_grads(t, 1.0, norm, ws)):
            with pytest.raises(ValueError, match=text):
                call([ok[0], bad])
    with pytest.raises(ValueError, match="current device"):
        T.swz_grad_norm([Typed(BF, device="cuda:1")], norm, ws)


def test_binding_checks_what_lists_are_written_to(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    ok = [Placed(A, BF, 200), Placed(B, FL, 400)]
    norm, ws = Placed(D, FL, 8), Placed(WS, BYTE, 1 << 20)
    for out, text in (([ok[0]], "1 tensors to write, 2 to read"), ([ok[0], Placed(C, FL, 404)], "tensor 1 to write"),
                      ([Placed(C, HF, 200), ok[1]], "tensor 0 to write"),
                      ([Placed(C, BF, 200, device="cuda:1"), Placed(E, FL, 400, device="cuda:1")], "on cuda:1|current device")):
        with pytest.raises(ValueError, match=text):
            T.swz_clip_grads(ok, 1.0, norm, ws, out=out)
    with pytest.raises(ValueError, match="norm holds"):
        T.swz_clip_grads(ok, 1.0, Placed(D, FL, 4), ws)
    with pytest.raises(ValueError, match="ws holds"):
        T.swz_clip_grads(ok, 1.0, norm, Placed(WS, BYTE, 8))
    with pytest.raises(ValueError, match="norm is on"):
        T.swz_clip_grads(ok, 1.0, Placed(D, FL, 8, device="cuda:1"), ws)
    with pytest.raises(T.SwzError):
        T.swz_clip_grads([ok[0], ok[0]], 1.0, norm, ws, stream=0)


# ------------------------------------------------------------ the definitions
@pytest.mark.parametrize("name", F.ACTS)
def test_activations_and_their_derivatives(name):
    z = np.linspace(-9, 9, 4001)
    a, da = F.activation(name, z)
    e = 1e-5
    diff = (F.activation(name, z + e)[0] - F.activation(name, z - e)[0]) / (2 * e)
    assert np.abs(diff - da).max() < 1e-9
    assert da.max() < 1.13 and da.min() > -0.13  # what the GPU tests' tolerances take
    assert np.abs(np.diff(da) / np.diff(z)).max() < 0.9
    want = {"silu": lambda t: torch.nn.functional.silu(t), "gelu": lambda t: torch.nn.functional.gelu(t),
            "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[name](torch.from_numpy(z))
    assert np.abs(want.numpy() - a).max() < 1e-13


def test_gradient_definition_against_autograd():
    rng = np.random.default_rng(0)
    x, wg, wu, dy = (torch.from_numpy(rng.standard_normal(s)).requires_grad_() for s in ((5, 8), (7, 8), (7, 8), (5, 7)))
    (torch.nn.functional.silu(x @ wg.t()) * (x @ wu.t()) * dy.detach()).sum().backward()
    got = F.gated_grad(*(t.detach().numpy() for t in (x, wg, wu)), "silu", dy.detach().numpy())
    for r, t in zip(got, (x, wg, wu)):
        assert np.abs(r - t.grad.numpy()).max() < 1e-12


def test_quantizer_definition():
    rng = np.random.default_rng(1)
    w = rng.standard_normal((20, 96)).astype(np.float32)
    same = lambda a: a  # noqa: E731
    for zero in (False, True):
        code, s, z = F.quant_w4(w, 64, zero, same)
        assert code.min() >= 0 and code.max() <= 15 and s.shape == (20, 2)
        q = F.pack_w4(code)
        assert np.array_equal(F.unpack_w4(q), code)
        back = F.dequant_w4(q, s, z if zero else None, 64)
        assert np.all(np.abs(back - w) <= 0.5001 * np.repeat(s, 64, axis=1)[:, :96] * (2 if zero else 1))
