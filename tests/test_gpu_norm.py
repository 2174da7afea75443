"""The norm of many tensors and the clipping by it, on the GPU.

Squares and sums are taken in 64 bits: the norm is off by its rounding to fp32 (2^-24) and count additions of 2^-53, the
factor, a quotient in 64 bits, by one rounding.  A clipped value is one fp32 product of the value and the factor, rounded
once to its type: the same bits as on the host, given the factor.
"""

import math

import numpy as np
import pytest

from oracle import feed_forward as F

import torch

import tiled_movement_amd as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def announce(*what):
    print("case:", *what, flush=True)


def make(sizes, seed=0, types=TYPES, scale=1.0):
    rng = np.random.default_rng(seed)
    return [torch.from_numpy(rng.standard_normal(n) * scale).to(types[i % len(types)]) for i, n in enumerate(sizes)]


def workspace(ts):
    return torch.full((max(1, T.swz_grad_norm_workspace(ts)),), 0xFF, dtype=torch.uint8, device=DEV)


def check(host, max_norm, out=False):
    dev = [t.to(DEV) for t in host]
    ws, got = workspace(dev), torch.full((2,), float("nan"), device=DEV)
    alone = torch.full((1,), float("nan"), device=DEV)
    T.swz_grad_norm(dev, alone, ws)
    to = [torch.full_like(t, 7.0) for t in dev] if out else None
    T.swz_clip_grads(dev, max_norm, got, ws, out=to)
    torch.cuda.synchronize()
    n, f = got.tolist()
    want = F.norm([t.double().numpy() for t in host])
    assert alone.item() == n and abs(n - want) <= 2.0 ** -23 * want
    factor = np.float32(max_norm / want) if want > max_norm else np.float32(1)
    assert abs(f - factor) <= 2.0 ** -23 * factor
    for h, d, o in zip(host, dev, to or dev):
        assert torch.equal(o.cpu(), (h.float() * f).to(h.dtype))
        if out:
            assert torch.equal(d.cpu(), h)
    return n, f


SIZES = [[1], [7], [8, 9], [1, 2, 3, 4, 5], [16383, 16384, 16385, 8191, 8192, 8193], [100000, 1, 333333, 17],
         [1000] * 64, [1000] * 65, list(range(1, 200)), [0, 5, 0, 0, 12, 0], [5000000, 3]]


@pytest.mark.parametrize("out", [False, True])
@pytest.mark.parametrize("sizes", SIZES, ids=[str(i) for i in range(len(SIZES))])
def test_norm_and_clipping(sizes, out):
    announce("norm", sizes[:6], len(sizes), out)
    host = make(sizes, seed=len(sizes))
    whole = F.norm([t.double().numpy() for t in host])
    for max_norm in (whole / 3, whole * 2, 0.0, math.inf):
        check(host, max_norm, out)


def test_no_tensors():
    announce("norm of nothing")
    for host in ([], [torch.empty(0)]):
        dev = [t.to(DEV) for t in host]
        got = torch.full((2,), float("nan"), device=DEV)
        T.swz_clip_grads(dev, 1.0, got, None)
        torch.cuda.synchronize()
        assert got.tolist() == [0.0, 1.0]


@pytest.mark.parametrize("dtype", TYPES)
def test_any_alignment(dtype):
    """Tensors at every element from a 16-byte boundary, written where they stand and at another offset."""
    announce("norm alignment", dtype)
    per = 16 // dtype.itemsize
    for n in (1, 5, 8, 40, 16400):
        base = torch.randn(n + 4 * per).to(dtype)
        for a in range(per):
            for b in (None, (a + 3) % per, a):
                d = base.to(DEV)
                o = torch.full((n + 4 * per,), 7.0, dtype=dtype, device=DEV)
                t = d[a:a + n]
                to = None if b is None else [o[b:b + n]]
                got = torch.empty(2, device=DEV)
                T.swz_clip_grads([t], 0.25, got, workspace([t]), out=to)
                torch.cuda.synchronize()
                h = base[a:a + n]
                f = got[1].item()
                want = (h.float() * f).to(dtype)
                assert abs(got[0].item() - F.norm([h.double().numpy()])) <= 2.0 ** -23 * got[0].item()
                if b is None:
                    assert torch.equal(t.cpu(), want)
                    assert torch.equal(d[:a].cpu(), base[:a]) and torch.equal(d[a + n:].cpu(), base[a + n:])
                else:
                    assert torch.equal(o[b:b + n].cpu(), want) and torch.equal(d.cpu(), base)
                    assert bool((o[:b] == 7).all()) and bool((o[b + n:] == 7).all())


def test_squares_that_leave_fp32():
    """Values of 1e30 and 1e-30: their squares are no fp32 numbers."""
    announce("norm far")
    n, f = check([torch.full((1000,), 1e30), torch.full((10,), 3.0)], 1.0)
    assert abs(n - 1e30 * math.sqrt(1000)) <= 1e24 and f > 0
    n, _ = check([torch.full((1000,), 1e-30)], 1e-31)
    assert abs(n - 1e-30 * math.sqrt(1000)) <= 1e-36
    # a norm over fp32's largest number is told as infinite, and still clips
    d = [torch.full((4096,), 3e38, device=DEV)]
    got = torch.empty(2, device=DEV)
    T.swz_clip_grads(d, 1e38, got, workspace(d))
    torch.cuda.synchronize()
    assert got[0].item() == math.inf and abs(got[1].item() - 1e38 / (3e38 * 64)) <= 1e-9
    assert abs(d[0][0].item() - 1e38 / 64) <= 1e31


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("out", [False, True])
def test_tensors_that_are_not_finite_stay(bad, out):
    announce("norm not finite", bad, out)
    host = make([100, 20000, 3], seed=2)
    host[1][777] = bad
    d = [t.to(DEV) for t in host]
    to = [torch.zeros_like(t) for t in d] if out else None
    got = torch.empty(2, device=DEV)
    T.swz_clip_grads(d, 1.0, got, workspace(d), out=to)
    torch.cuda.synchronize()
    assert not math.isfinite(got[0].item()) and got[1].item() == 1.0
    for h, o in zip(host, to or d):
        assert torch.equal(o.cpu().view(torch.uint8), h.view(torch.uint8))


def test_tensor_behind_2_to_32_elements():
    announce("norm 2^32")
    n = (1 << 32) + 12345
    t = torch.full((n,), 0.5, dtype=torch.bfloat16, device=DEV)
    small = torch.full((9,), 2.0, device=DEV)
    t[-1], t[1 << 32], t[(1 << 31) + 1] = 1024.0, 2048.0, 512.0
    want = math.sqrt((n - 3) * 0.25 + 1024.0 ** 2 + 2048.0 ** 2 + 512.0 ** 2 + 36.0)
    got = torch.empty(2, device=DEV)
    T.swz_clip_grads([t, small], want / 4, got, workspace([t, small]))
    torch.cuda.synchronize()
    assert abs(got[0].item() - want) <= 2.0 ** -23 * want and abs(got[1].item() - 0.25) <= 2.0 ** -24
    f = got[1].item()
    as_type = lambda v: torch.tensor(v * f).to(torch.bfloat16).item()  # noqa: E731
    assert t[-1].item() == as_type(1024.0) and t[1 << 32].item() == as_type(2048.0) and t[(1 << 31) + 1].item() == as_type(512.0)
    for a in range(0, n, 1 << 30):
        piece = t[a:a + (1 << 30)]
        assert int((piece != as_type(0.5)).sum()) == sum(a <= i < a + (1 << 30) for i in (n - 1, 1 << 32, (1 << 31) + 1))


def test_same_bits_on_streams_and_in_graphs():
    announce("norm graph")
    host = make([3000] * 70 + [400000, 5], seed=4)
    src = [t.to(DEV) for t in host]
    d = [t.clone() for t in src]
    ws, got = workspace(d), torch.empty(2, device=DEV)
    T.swz_clip_grads(d, 10.0, got, ws)
    torch.cuda.synchronize()
    want, norm = [t.clone() for t in d], got.tolist()

    def again(run):
        for t, s in zip(d, src):
            t.copy_(s)
        ws.fill_(0xFF)
        got.fill_(float("nan"))
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        assert got.tolist() == norm and all(torch.equal(a, b) for a, b in zip(d, want))

    side = torch.cuda.Stream()

    def on_side():
        with torch.cuda.stream(side):
            T.swz_clip_grads(d, 10.0, got, ws)

    again(on_side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        T.swz_clip_grads(d, 10.0, got, ws)
    for _ in range(3):
        again(graph.replay)
        torch.randn(1000, device=DEV).sum().item()
