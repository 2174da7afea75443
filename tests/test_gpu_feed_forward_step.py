"""The feed-forward calls together, as a program runs them: a training step from the block through an output layer's loss
and back to clipped gradients, and the same block served with 4-bit weights.

Each stage is held to its 64-bit definition on what the stage before it really wrote, so a stage's own rounding is all
that may differ: 2^-8 of a bf16 result (relative to its norm, since every value is off by at most that), twice that where
dg and du are rounded on the way, and fp32 sums of at most 1111 products (2^-13 of sums of magnitudes, far below).
"""

import math

import numpy as np
import pytest

from oracle import feed_forward as F
from oracle import products as P

import torch

import tiled_movement_amd as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def near(got, want, tol):
    return np.linalg.norm(got.double().cpu().numpy() - want) <= tol * np.linalg.norm(want)


def test_training_step():
    print("case: training step", flush=True)
    rng = np.random.default_rng(40)
    n, k, f, v = 160, 128, 224, 1111
    make = lambda *s, by=1.0: torch.from_numpy(rng.standard_normal(s) * by).bfloat16().to(DEV)  # noqa: E731
    new = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    byte = lambda b: torch.empty(b, dtype=torch.uint8, device=DEV)  # noqa: E731
    x, wg, wu, wd, wo = make(n, k), make(f, k, by=0.1), make(f, k, by=0.1), make(k, f, by=0.07), make(v, k, by=0.1)
    target = torch.from_numpy(rng.integers(0, v, n)).to(DEV)
    up = torch.full((n,), 1 / n, device=DEV)
    y, h, dh, dy, dx = new(n, f), new(n, k), new(n, k), new(n, f), new(n, k)
    dwg, dwu, dwd, dwo = torch.empty_like(wg), torch.empty_like(wu), torch.empty_like(wd), torch.empty_like(wo)
    wdt, dht, yt = new(f, k), new(k, n), new(f, n)
    pre, loss, lse, zt = (torch.empty(s, device=DEV) for s in ((2, n, f), n, n, n))
    ws, ws_loss = byte(T.swz_gated_workspace(n, f, k)), byte(T.swz_linear_loss_workspace(n, v, k, grad=True))
    grads = [dwg, dwu, dwd, dwo]
    ws_norm, norm = byte(T.swz_grad_norm_workspace(grads)), torch.empty(2, device=DEV)
    max_norm = 0.05

    def step():
        T.swz_gated(x, wg, wu, y, n, f, k, pre=pre)
        T.swz_gemm_ex(y, wd, h, n, k, f, c_type=T.C_BF16)
        T.swz_linear_ce(h, wo, target, loss, lse, zt, n, v, k, ws_loss)
        T.swz_linear_ce_grad(h, wo, target, lse, zt, up, dh, dwo, n, v, k, ws_loss)
        T.swz_transpose(wd, wdt, k, f, 2)
        T.swz_gemm_ex(dh, wdt, dy, n, f, k, c_type=T.C_BF16)
        T.swz_transpose(dh, dht, n, k, 2)
        T.swz_transpose(y, yt, n, f, 2)
        T.swz_gemm_ex(dht, yt, dwd, k, f, n, c_type=T.C_BF16)
        T.swz_gated_grad(x, wg, wu, dy, dx, dwg, dwu, n, f, k, ws, pre=pre)

    step()
    torch.cuda.synchronize()
    whole = [g.clone() for g in grads]
    T.swz_clip_grads(grads, max_norm, norm, ws_norm)
    torch.cuda.synchronize()
    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    assert near(y, F.gated(host(x), host(wg), host(wu), "silu")[0], 2.0 ** -8)
    assert near(h, host(y) @ host(wd).T, 2.0 ** -8)
    ref = P.linear_loss(host(h), host(wo), target.cpu().numpy(), None, 1.0, np.full(n, 1 / n))
    assert np.abs(host(loss) - ref["loss"]).max() < 1e-4
    assert near(dh, ref["dh"], 2.0 ** -8) and near(whole[3], ref["dw"], 2.0 ** -8)
    assert near(dy, host(dh) @ host(wd), 2.0 ** -8) and near(whole[2], host(dh).T @ host(y), 2.0 ** -8)
    rdx, rdwg, rdwu, _, _ = F.gated_grad(host(x), host(wg), host(wu), "silu", host(dy))
    for got, want in ((dx, rdx), (whole[0], rdwg), (whole[1], rdwu)):
        assert near(got, want, 2.0 ** -7)
    total = F.norm([host(g) for g in whole])
    assert total > max_norm and abs(norm[0].item() - total) <= 2.0 ** -23 * total
    for g, w in zip(grads, whole):
        assert torch.equal(g.cpu(), (w.cpu().float() * norm[1].item()).bfloat16())
    # a smaller step along the clipped gradient is a captured program's whole loop
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
        T.swz_clip_grads(grads, max_norm, norm, ws_norm)
    want = [g.clone() for g in grads] + [dx.clone(), norm.clone()]
    for _ in range(3):
        for t in grads + [dx, y, h]:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(grads + [dx, norm], want))
        torch.randn(1000, device=DEV).sum().item()


@pytest.mark.parametrize("m", [1, 11, 40])
def test_served_with_4_bit_weights(m):
    print("case: served", m, flush=True)
    rng = np.random.default_rng(41 + m)
    k, f = 288, 416
    make = lambda *s, by=1.0: torch.from_numpy(rng.standard_normal(s) * by).bfloat16().to(DEV)  # noqa: E731
    x, wg, wu, wd = make(m, k), make(f, k, by=0.06), make(f, k, by=0.06), make(k, f, by=0.05)

    def quantized(w):
        n, cols = w.shape
        groups = -(-cols // 128)
        q = torch.empty(n, cols // 2, dtype=torch.uint8, device=DEV)
        s, z = torch.empty(n, groups, dtype=torch.bfloat16, device=DEV), torch.empty(n, groups, dtype=torch.uint8, device=DEV)
        T.swz_quant_w4(w, q, s, n, cols, zero=z)
        return q, s, z

    (qg, sg, zg), (qu, su, zu), (qd, sd, zd) = quantized(wg), quantized(wu), quantized(wd)
    y, out = torch.empty(m, f, dtype=torch.bfloat16, device=DEV), torch.empty(m, k, dtype=torch.bfloat16, device=DEV)
    T.swz_gated_w4(x, qg, sg, qu, su, y, m, f, k, zero_g=zg, zero_u=zu)
    T.swz_gemm_w4(y, qd, sd, out, m, k, f, zero=zd)
    # a prompt takes the weights turned back
    back = [torch.empty_like(w) for w in (wg, wu)]
    T.swz_dequant_w4(qg, sg, back[0], f, k, zero=zg)
    T.swz_dequant_w4(qu, su, back[1], f, k, zero=zu)
    y2 = torch.empty_like(y)
    T.swz_gated(x, *back, y2, m, f, k)
    torch.cuda.synchronize()
    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    values = lambda q, s, z: F.dequant_w4(q.cpu().numpy(), host(s), z.cpu().numpy(), 128)  # noqa: E731
    want, g, u = F.gated(host(x), values(qg, sg, zg), values(qu, su, zu), "silu")
    # fp32 sums of k terms of up to 48 scales, carried through the product
    assert near(y, want, 2.0 ** -8)
    assert near(out, host(y) @ values(qd, sd, zd).T, 2.0 ** -8)
    # the values' rounding to bf16, and what it moves the activation by
    size = np.abs(host(x)) @ np.abs(values(qg, sg, zg)).T, np.abs(host(x)) @ np.abs(values(qu, su, zu)).T
    tol = 2.0 ** -8 * (1.2 * size[0] * (np.abs(u) + 2.0 ** -8 * size[1]) + np.abs(F.activation("silu", g)[0]) * size[1] + np.abs(want))
    assert np.all(np.abs(host(y2) - want) <= 1.02 * tol + 1e-6)
    # and the weights themselves are theirs to within a step of their group
    for w, (q, s, z) in ((wg, (qg, sg, zg)), (wu, (qu, su, zu)), (wd, (qd, sd, zd))):
        step = np.repeat(host(s), 128, axis=1)[:, :w.shape[1]]
        assert np.all(np.abs(values(q, s, z) - host(w)) <= 1.03 * step) and math.isfinite(step.max())
