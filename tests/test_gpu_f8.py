"""The 8-bit quantizer and product on the GPU against their 64-bit definitions.

The quantizer's one rounding is to the 8-bit grid (its scales are powers of
two), so its values and scales must be equal, not near.  Products of operands
made of small whole numbers are exact in fp32 and must be equal too; random
operands stay within the first-order bound of an fp32 sum
(oracle.products.product_f8_bound) plus, for a bf16 result, half a step
(2^-8 of the value) and what the 8-bit instruction drops: of each eight
consecutive products, up to 2^-13 of the largest from each of the other seven,
so at most 2^-10 of the sum of magnitudes.
"""

import numpy as np
import pytest

from oracle import products as P

import torch

import tiled_movement_amd as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
XT = {"bf16": (torch.bfloat16, T.X_BF16), "fp16": (torch.float16, T.X_F16), "fp32": (torch.float32, T.X_F32)}
KIND = {"e4m3": T.F8_E4M3, "e5m2": T.F8_E5M2}
SENTINEL = 0x5A


def announce(*what):
    print("case:", *what, flush=True)


def up16(n):
    return -(-n // 16) * 16


def quant(x, kind, square, scale_type, rows=True, transposed=True, ld_x=None, x_type=None, **kw):
    """Runs the call on x [R][ld_x] with sentinel-filled outputs; returns host bytes and scales."""
    r = x.shape[0]
    c = kw.pop("cols", x.shape[1])
    sdt = torch.uint8 if scale_type == T.SCALE_E8M0 else torch.float32
    br = 128 if square else 1

    def out(rr, cc):
        return (torch.full((rr, up16(cc) + 16), SENTINEL, dtype=torch.uint8, device=DEV),
                torch.full((-(-rr // br), -(-cc // 128)), 7, dtype=sdt, device=DEV))

    q, s = out(r, c) if rows else (None, None)
    qt, st = out(c, r) if transposed else (None, None)
    T.swz_quant_f8(x, q, s, r, c, x_type=x_type, f8_type=KIND[kind], block=T.BLOCK_128X128 if square else T.BLOCK_1X128,
                   scale_type=scale_type, ld_x=ld_x, ld_q=up16(c) + 16, qt=qt, scale_t=st, ld_qt=up16(r) + 16, **kw)
    torch.cuda.synchronize()
    return [None if t is None else t.cpu().numpy() for t in (q, s, qt, st)]


def check_quant(q, s, x, kind, square):
    ref, ex = P.quantize(x, kind, 128 if square else 1)
    got = P.f8_decode(q[:, :x.shape[1]], kind)
    assert np.array_equal(got, ref, equal_nan=True)
    if s.dtype == np.uint8:
        assert np.array_equal(s, ex + 127)
    else:
        assert np.array_equal(s.astype(np.float64), 2.0 ** ex)
    assert np.all(q[:, x.shape[1]:] == SENTINEL)  # the pitch's padding is left alone


def values(r, c, seed, spread=1.5):
    rng = np.random.default_rng(seed)
    return rng.standard_normal((r, c)) * np.exp(spread * rng.standard_normal((r, 1))) * np.exp(spread * rng.standard_normal((1, c)))


@pytest.mark.parametrize("xt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("r,c", [(1, 8), (1, 1), (3, 129), (130, 256), (128, 128), (257, 120), (65, 391)])
def test_quant_equals_definition(xt, kind, square, r, c):
    announce("quant", xt, kind, square, r, c)
    dt, code = XT[xt]
    x = torch.from_numpy(values(r, c, r * 1000 + c)).to(dt)
    xf = x.double().numpy()
    q, s, qt, st = quant(x.to(DEV), kind, square, T.SCALE_E8M0, x_type=code)
    check_quant(q, s, xf, kind, square)
    check_quant(qt, st, np.ascontiguousarray(xf.T), kind, square)
    # one output at a time, fp32 scales
    q, s, _, _ = quant(x.to(DEV), kind, square, T.SCALE_F32, transposed=False, x_type=code)
    check_quant(q, s, xf, kind, square)
    _, _, qt, st = quant(x.to(DEV), kind, square, T.SCALE_F32, rows=False, x_type=code)
    check_quant(qt, st, np.ascontiguousarray(xf.T), kind, square)


@pytest.mark.parametrize("xt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_every_rounding_and_tie(kind, xt):
    """Every bf16 significand at every distance from the block's largest value."""
    announce("quant ties", kind)
    m = np.arange(128, 256) / 128.0
    rows = []
    for d in range(0, 24 if xt != "fp16" else 7):  # what a fp16 still holds exactly
        rows.append(np.concatenate([[1.75], (m * 2.0 ** -d)[:127]]))
        rows.append(np.concatenate([[-1.0], -(m * 2.0 ** -d)[1:]]) if d else np.concatenate([[-1.9921875], -m[:127]]))
    x = np.stack(rows)
    dt, code = XT[xt]
    t = torch.from_numpy(x).to(dt)
    assert np.array_equal(t.double().numpy(), x)
    q, s, qt, st = quant(t.to(DEV), kind, False, T.SCALE_E8M0, x_type=code)
    check_quant(q, s, x, kind, False)
    check_quant(qt, st, np.ascontiguousarray(x.T), kind, False)


@pytest.mark.parametrize("xt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("square", [False, True])
def test_special_values(kind, square, xt):
    announce("quant special", kind, square, xt)
    dt, code = XT[xt]
    x = values(140, 260, 3, spread=0.5).astype(np.float32)
    x[0, :] = 0
    x[1, 5], x[2, 7], x[3, 130] = np.inf, -np.inf, np.nan
    x[4, :] = np.nan
    x[5, :128] = np.inf
    x[6, :] = {"bf16": 1e-40, "fp16": 1e-7, "fp32": 1e-42}[xt]  # subnormal
    x[7, 3] = {"bf16": 3.3e38, "fp16": 65504.0, "fp32": 3.4e38}[xt]
    x[8, :] = -0.0
    x[9, :128] = 448.0
    x[9, 128:] = np.nextafter(np.float32(448.0), np.float32(1e9))
    x[10, :] = {"bf16": 2.0 ** -126, "fp16": 2.0 ** -24, "fp32": 2.0 ** -149}[xt]
    t = torch.from_numpy(x).to(dt)
    q, s, qt, st = quant(t.to(DEV), kind, square, T.SCALE_E8M0, x_type=code)
    xf = t.double().numpy()
    check_quant(q, s, xf, kind, square)
    check_quant(qt, st, np.ascontiguousarray(xf.T), kind, square)


@pytest.mark.parametrize("off,ld", [(0, 264), (1, 264), (0, 261), (4, 300)])
def test_quant_pitched_and_unaligned_input(off, ld):
    announce("quant pitch", off, ld)
    buf = torch.from_numpy(values(1, 70 * 300 + 8, 9)[0]).to(torch.bfloat16)
    x = buf[off:off + 70 * ld].view(70, ld)
    dev = buf.to(DEV)[off:off + 70 * ld]
    q, s, qt, st = quant(dev.view(70, ld), "e4m3", False, T.SCALE_E8M0, ld_x=ld, x_type=T.X_BF16, cols=256)
    xf = x[:, :256].double().numpy()
    check_quant(q, s, xf, "e4m3", False)
    check_quant(qt, st, np.ascontiguousarray(xf.T), "e4m3", False)


# ------------------------------------------------------------------ product
def operand(r, k, kind, square, scale_type, seed, exact=False):
    """(device bytes [r][ld], device scales, float64 values); bytes behind k are NaN bytes."""
    rng = np.random.default_rng(seed)
    ld = up16(k) + 16
    if exact:
        v = rng.integers(-3, 4, size=(r, k)).astype(np.float64)
        t = torch.from_numpy(v)
    else:
        t = torch.from_numpy(rng.standard_normal((r, k)) * 8)
    f8 = torch.float8_e4m3fn if kind == "e4m3" else torch.float8_e5m2
    bits = t.to(f8).view(torch.uint8).numpy()
    data = np.full((r, ld), 0x7F, dtype=np.uint8)
    data[:, :k] = bits
    shape = (-(-r // 128) if square else r, -(-k // 128))
    if scale_type == T.SCALE_E8M0:
        s = rng.integers(124, 131, size=shape).astype(np.uint8)
    elif exact:
        s = 2.0 ** rng.integers(-3, 4, size=shape).astype(np.float32)
    else:
        s = np.exp(rng.standard_normal(shape)).astype(np.float32)
    val = P.dequantize(bits, kind, s, square)
    return torch.from_numpy(data).to(DEV), torch.from_numpy(s).to(DEV), val


def gemm(a, b, m, n, k, ak, bk, sqa, sqb, scale_type, c_type, pad=0):
    dt = torch.float32 if c_type == T.C_F32 else torch.bfloat16
    c = torch.full((m * n + 2 * pad,), float("nan"), dtype=dt, device=DEV)
    out = c[pad:pad + m * n]
    T.swz_gemm_f8(a[0], a[1], b[0], b[1], out, m, n, k, lda=a[0].shape[1], ldb=b[0].shape[1], a_type=KIND[ak],
                  b_type=KIND[bk], a_block=int(sqa), b_block=int(sqb), scale_type=scale_type, c_type=c_type)
    torch.cuda.synchronize()
    full = c.double().cpu().numpy()
    assert np.all(np.isnan(full[:pad])) and np.all(np.isnan(full[pad + m * n:]))
    return full[pad:pad + m * n].reshape(m, n)


SHAPES = [(1, 1, 1), (1, 300, 128), (3, 17, 1000), (16, 256, 256), (17, 130, 384), (33, 640, 520), (64, 100, 640),
          (65, 257, 129), (130, 48, 4111), (256, 256, 128), (300, 521, 272), (513, 260, 1024)]


@pytest.mark.parametrize("scale_type,sqa,sqb", [(T.SCALE_E8M0, False, True), (T.SCALE_E8M0, False, False),
                                                (T.SCALE_E8M0, True, True), (T.SCALE_F32, False, True),
                                                (T.SCALE_F32, False, False), (T.SCALE_F32, True, False)])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gemm_whole_numbers_equal(m, n, k, scale_type, sqa, sqb):
    announce("gemm exact", m, n, k, scale_type, sqa, sqb)
    a = operand(m, k, "e4m3", sqa, scale_type, m + k, exact=True)
    b = operand(n, k, "e4m3", sqb, scale_type, n + 2 * k, exact=True)
    got = gemm(a, b, m, n, k, "e4m3", "e4m3", sqa, sqb, scale_type, T.C_F32, pad=4)
    # sums of multiples of 2^-6 below 2^17: exact in fp32
    assert np.array_equal(got, P.product_f8(a[2], b[2]))


@pytest.mark.parametrize("ak,bk", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("scale_type,sqb", [(T.SCALE_E8M0, True), (T.SCALE_E8M0, False), (T.SCALE_F32, True),
                                            (T.SCALE_F32, False)])
@pytest.mark.parametrize("m,n,k", [(5, 260, 1000), (40, 200, 700), (300, 264, 1032)])
@pytest.mark.parametrize("c_type", [T.C_F32, T.C_BF16])
def test_gemm_random_within_bound(ak, bk, scale_type, sqb, m, n, k, c_type):
    announce("gemm random", ak, bk, scale_type, sqb, m, n, k, c_type)
    a = operand(m, k, ak, False, scale_type, 1)
    b = operand(n, k, bk, sqb, scale_type, 2)
    got = gemm(a, b, m, n, k, ak, bk, False, sqb, scale_type, c_type)
    ref, bound = P.product_f8(a[2], b[2]), P.product_f8_bound(a[2], b[2])
    if c_type == T.C_BF16:
        bound = bound + 2.0 ** -10 * (np.abs(a[2]) @ np.abs(b[2]).T)
        bound = bound + 2.0 ** -8 * (np.abs(ref) + bound)
    assert np.all(np.abs(got - ref) <= bound)


@pytest.mark.parametrize("pad,n", [(1, 256), (0, 257), (3, 129), (2, 320)])
@pytest.mark.parametrize("m", [2, 70])
def test_gemm_unaligned_result(pad, n, m):
    announce("gemm unaligned", pad, n, m)
    a = operand(m, 256, "e4m3", False, T.SCALE_E8M0, 5, exact=True)
    b = operand(n, 256, "e4m3", True, T.SCALE_E8M0, 6, exact=True)
    ref = P.product_f8(a[2], b[2])
    got = gemm(a, b, m, n, 256, "e4m3", "e4m3", False, True, T.SCALE_E8M0, T.C_F32, pad)
    assert np.array_equal(got, ref)
    got = gemm(a, b, m, n, 256, "e4m3", "e4m3", False, True, T.SCALE_E8M0, T.C_BF16, pad)
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref))


@pytest.mark.parametrize("m", [1, 20, 100])
def test_gemm_empty_k_writes_zeros(m):
    announce("gemm k=0", m)
    z = torch.zeros(1, dtype=torch.uint8, device=DEV)
    c = torch.full((m, 33), float("nan"), dtype=torch.float32, device=DEV)
    T.swz_gemm_f8(z, z, z, z, c, m, 33, 0, lda=0, ldb=0, c_type=T.C_F32)
    torch.cuda.synchronize()
    assert torch.all(c == 0)


@pytest.mark.parametrize("m", [4, 90])
def test_gemm_nan_stays_in_its_row_and_column(m):
    announce("gemm nan", m)
    a = operand(m, 200, "e4m3", False, T.SCALE_E8M0, 8, exact=True)
    b = operand(140, 200, "e4m3", True, T.SCALE_E8M0, 9, exact=True)
    a[0][2, 150] = 0x7F
    b[0][7, 3] = 0xFF
    ref = P.product_f8(a[2], b[2])
    ref[2, :] = np.nan
    ref[:, 7] = np.nan
    got = gemm(a, b, m, 140, 200, "e4m3", "e4m3", False, True, T.SCALE_E8M0, T.C_F32)
    assert np.array_equal(got, ref, equal_nan=True)


@pytest.mark.parametrize("m", [4, 90, 300])
@pytest.mark.parametrize("c_type", [T.C_F32, T.C_BF16])
@pytest.mark.parametrize("scale_type", [T.SCALE_F32, T.SCALE_E8M0])
def test_gemm_nan_scales_and_infinities(m, c_type, scale_type):
    """A NaN scale makes its row (or its 128 rows of B) NaN; an e5m2 infinity its row infinite."""
    announce("gemm nan scale", m, c_type, scale_type)
    n, k = 300, 392
    a = operand(m, k, "e5m2", False, scale_type, 8, exact=True)
    b = operand(n, k, "e4m3", True, scale_type, 9, exact=True)
    b[0][:, 5] = 0x38  # ones where the infinity meets them
    bad = float("nan") if scale_type == T.SCALE_F32 else 255
    a[1][1, 2] = bad
    b[1][1, 3] = bad
    a[0][2, 5] = 0x7C
    got = gemm(a, b, m, n, k, "e5m2", "e4m3", False, True, scale_type, c_type)
    assert np.all(np.isnan(got[1])) and np.all(np.isnan(got[:, 128:256]))
    rest = np.r_[0:128, 256:n]
    assert np.all(np.isposinf(got[2, rest]))
    rows = np.array([r for r in range(m) if r not in (1, 2)])
    assert np.all(np.isfinite(got[np.ix_(rows, rest)]))


@pytest.mark.parametrize("m", [4, 90])
@pytest.mark.parametrize("ea,eb", [(1, 200), (253, 60), (30, 30), (127, 127)])
def test_gemm_far_scales(m, ea, eb):
    """E8M0 scales far from one (their values times them stay normal bf16 numbers): exact where the result is normal."""
    announce("gemm far scales", m, ea, eb)
    n, k = 140, 256
    a = operand(m, k, "e4m3", False, T.SCALE_E8M0, 8, exact=True)
    b = operand(n, k, "e4m3", True, T.SCALE_E8M0, 9, exact=True)
    raw = P.product_f8(P.f8_decode(a[0].cpu().numpy()[:, :k], "e4m3"), P.f8_decode(b[0].cpu().numpy()[:, :k], "e4m3"))
    a[1].fill_(ea)
    b[1].fill_(eb)
    ref = raw * 2.0 ** (ea + eb - 254)
    got = gemm(a, b, m, n, k, "e4m3", "e4m3", False, True, T.SCALE_E8M0, T.C_F32)
    if ea + eb - 254 > -120:
        assert np.array_equal(got, ref)
    else:  # products below the normal range of fp32: nothing but zero or the rounded value
        assert np.all(np.abs(got - ref) <= 2.0 ** -126 * k)


# ------------------------------------------------------------- as they are used
def test_training_layer_with_its_gradients():
    """x -> quantize -> y = x w^T; dy -> dx = dy w, dw = dy^T x, all of 8-bit operands, chained as a training step
    does.  Each product is compared with the 64-bit product of the operands it was given."""
    announce("layer")
    rng = np.random.default_rng(20)
    tok, nin, nout = 300, 520, 390
    x = torch.from_numpy(rng.standard_normal((tok, nin))).to(torch.bfloat16).to(DEV)
    w = torch.from_numpy(rng.standard_normal((nout, nin)) * 0.05).to(torch.float32).to(DEV)
    dy = torch.from_numpy(rng.standard_normal((tok, nout)) * 1e-3).to(torch.bfloat16).to(DEV)

    def q(t, r, c, code, square, kind):
        br = 128 if square else 1
        new = lambda *s: torch.empty(s, dtype=torch.uint8, device=DEV)  # noqa: E731
        o = (new(r, up16(c)), new(-(-r // br), -(-c // 128)), new(c, up16(r)), new(-(-c // br), -(-r // 128)))
        T.swz_quant_f8(t, o[0], o[1], r, c, x_type=code, f8_type=KIND[kind], block=int(square), qt=o[2], scale_t=o[3])
        return o

    def val(b, s, r, c, square, kind):
        return P.dequantize(b.cpu().numpy()[:, :c], kind, s.cpu().numpy(), square)

    xq, wq, gq = q(x, tok, nin, T.X_BF16, False, "e4m3"), q(w, nout, nin, T.X_F32, True, "e4m3"), q(dy, tok, nout, T.X_BF16, False, "e5m2")
    y = torch.empty(tok, nout, dtype=torch.bfloat16, device=DEV)
    dx = torch.empty(tok, nin, dtype=torch.bfloat16, device=DEV)
    dw = torch.empty(nout, nin, dtype=torch.float32, device=DEV)
    T.swz_gemm_f8(xq[0], xq[1], wq[0], wq[1], y, tok, nout, nin)
    T.swz_gemm_f8(gq[0], gq[1], wq[2], wq[3], dx, tok, nin, nout, a_type=T.F8_E5M2)
    T.swz_gemm_f8(gq[2], gq[3], xq[2], xq[3], dw, nout, nin, tok, a_type=T.F8_E5M2, b_block=T.BLOCK_1X128, c_type=T.C_F32)
    torch.cuda.synchronize()
    for got, a, b, half in (
            (y, val(xq[0], xq[1], tok, nin, False, "e4m3"), val(wq[0], wq[1], nout, nin, True, "e4m3"), True),
            (dx, val(gq[0], gq[1], tok, nout, False, "e5m2"), val(wq[2], wq[3], nin, nout, True, "e4m3"), True),
            (dw, val(gq[2], gq[3], nout, tok, False, "e5m2"), val(xq[2], xq[3], nin, tok, False, "e4m3"), False)):
        ref, bound = P.product_f8(a, b), P.product_f8_bound(a, b)
        if half:
            bound = bound + 2.0 ** -10 * (np.abs(a) @ np.abs(b).T)
            bound = bound + 2.0 ** -8 * (np.abs(ref) + bound)
        assert np.all(np.abs(got.double().cpu().numpy() - ref) <= bound)
    # and the layer is the layer: 8-bit rounding (half a step of each operand, 2^-4 e4m3 and 2^-3 e5m2, below the
    # normal range 2^-10 and 2^-17 of a scale of at most 2^-8 and 2^-15 of twice the block's largest value)
    xf, wf, gf = x.double().cpu().numpy(), w.double().cpu().numpy(), dy.double().cpu().numpy()
    ex, ew, eg = (s * np.abs(t) + 2.0 ** -17 * np.abs(t).max() for s, t in ((2.0 ** -4, xf), (2.0 ** -4, wf), (2.0 ** -3, gf)))
    for got, (a, ea), (b, eb) in ((y, (xf, ex), (wf.T, ew.T)), (dx, (gf, eg), (wf, ew)), (dw, (gf.T, eg.T), (xf, ex))):
        bound = ea @ (np.abs(b) + eb) + np.abs(a) @ eb
        assert np.all(np.abs(got.double().cpu().numpy() - a @ b) <= bound + 2.0 ** -7 * (np.abs(a) @ np.abs(b)))


@pytest.mark.parametrize("m", [3, 100, 700])
def test_streams_and_graphs_give_the_same_bits(m):
    announce("graph", m)
    n, k = 520, 1000
    x = torch.from_numpy(values(m, k, 4, 0.3)).to(torch.bfloat16).to(DEV)
    b = operand(n, k, "e4m3", True, T.SCALE_E8M0, 7)
    q = torch.empty(m, up16(k), dtype=torch.uint8, device=DEV)
    s = torch.empty(m, 8, dtype=torch.uint8, device=DEV)
    c = {t: torch.empty(m, n, dtype=d, device=DEV) for t, d in ((T.C_F32, torch.float32), (T.C_BF16, torch.bfloat16))}

    def work():
        T.swz_quant_f8(x, q, s, m, k)
        for t in c:
            T.swz_gemm_f8(q, s, b[0], b[1], c[t], m, n, k, ldb=b[0].shape[1], c_type=t)

    def clear():
        q.zero_()
        s.zero_()
        for t in c.values():
            t.fill_(float("nan"))
        torch.cuda.synchronize()

    work()
    torch.cuda.synchronize()
    want = {t: v.clone() for t, v in c.items()}
    side = torch.cuda.Stream()
    clear()
    with torch.cuda.stream(side):
        work()
    side.synchronize()
    assert all(torch.equal(c[t], want[t]) for t in c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for _ in range(3):
        clear()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(c[t], want[t]) for t in c)
        torch.randn(100, device=DEV).sum().item()


@pytest.mark.parametrize("m", [3, 20, 300])
def test_rows_behind_2_to_32_bytes(m):
    """B of 4.6 GB: whole-number operands, the last rows against the 64-bit product."""
    announce("gemm 2^32", m)
    n, k = 70000, 65536
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    b = torch.randint(0, 2, (n, k), generator=g, device=DEV, dtype=torch.uint8) * 0x38  # 0 or 1
    a = torch.randint(0, 2, (m, k), generator=g, device=DEV, dtype=torch.uint8) * 0x38
    sa = torch.full((m, k // 128), 127, dtype=torch.uint8, device=DEV)
    sb = torch.full((-(-n // 128), k // 128), 127, dtype=torch.uint8, device=DEV)
    c = torch.empty(m, n, dtype=torch.float32, device=DEV)
    T.swz_gemm_f8(a, sa, b, sb, c, m, n, k, c_type=T.C_F32)
    rows = torch.tensor([0, 1, 32767, 65535, 65536, 65537, 69998, 69999], device=DEV)
    ref = (a != 0).double().cpu().numpy() @ (b[rows] != 0).double().cpu().numpy().T
    assert np.array_equal(c[:, rows].double().cpu().numpy(), ref)


def test_quant_behind_2_to_32_bytes():
    announce("quant 2^32")
    r, c = 33001, 65544
    x = torch.empty(r, c, dtype=torch.bfloat16, device=DEV)
    x.copy_((torch.arange(c, device=DEV) % 251 - 125).to(torch.bfloat16))
    x *= (torch.arange(r, device=DEV) % 7 + 1).to(torch.bfloat16)[:, None]
    q, s = torch.empty(r, up16(c), dtype=torch.uint8, device=DEV), torch.empty(r, -(-c // 128), dtype=torch.uint8, device=DEV)
    qt, st = torch.empty(c, up16(r), dtype=torch.uint8, device=DEV), torch.empty(c, -(-r // 128), dtype=torch.uint8, device=DEV)
    T.swz_quant_f8(x, q, s, r, c, qt=qt, scale_t=st)
    rows = torch.tensor([0, 32767, 32768, 33000], device=DEV)
    ref, ex = P.quantize(x[rows].double().cpu().numpy(), "e4m3", 1)
    assert np.array_equal(P.f8_decode(q[rows].cpu().numpy()[:, :c], "e4m3"), ref) and np.array_equal(s[rows].cpu().numpy(), ex + 127)
    cols = torch.tensor([0, 65535, 65536, 65543], device=DEV)
    ref, ex = P.quantize(x[:, cols].t().double().cpu().numpy(), "e4m3", 1)
    assert np.array_equal(P.f8_decode(qt[cols].cpu().numpy()[:, :r], "e4m3"), ref) and np.array_equal(st[cols].cpu().numpy(), ex + 127)
    q2 = torch.empty_like(q)
    T.swz_quant_f8(x, q2, s, r, c)
    torch.cuda.synchronize()
    assert torch.equal(q2[:, :c], q[:, :c])
