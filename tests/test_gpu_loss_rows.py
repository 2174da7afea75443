"""What one row of a loss call may not do to another, and what a row's loss owes to its own logits."""

import numpy as np
import pytest
import torch

from test_gpu_loss import DT, U, Case

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def announce(*what):
    print("case:", *what, flush=True)


def check_rows(c, d):
    """c's losses and gradients in d against their 64-bit values with the tolerances of test_gpu_loss.py, but each row's dz
    by its own upstream: rounding to fp16, 2^-11 of the value, below the normal range 2^-25 of what 2^14 times at least
    half the upstream stands for, so 2^-38 of it.  Operands widened to fp16: 2^-25 where the largest is at least 2^14."""
    t = {x: torch.as_tensor(np.asarray(getattr(c, x))).to(DEV) for x in ("index", "upstream")}
    h, w, tau, top = c.h.to(DEV).double(), c.w.to(DEV).double(), c.tau, max(c.top, 1)
    here = (t["index"] >= 0) & (t["index"] < c.v)
    at = torch.where(here, t["index"], 0)
    z = h @ w.t() / tau
    lse = torch.logsumexp(z, dim=1)
    entropy = torch.zeros(c.n, dtype=torch.float64, device=DEV)
    teach = torch.zeros(c.n, dtype=torch.float64, device=DEV)
    if c.top:
        teacher = torch.from_numpy(c.teacher).to(DEV).double() / tau
        here &= teacher > -np.inf
        at = torch.where(here, t["index"], 0)
        p = torch.softmax(teacher.masked_fill(~here, -np.inf), dim=1).nan_to_num(0.0)
        entropy = -torch.special.entr(p).sum(dim=1)
        teach = (6 * torch.where(here, teacher.abs(), 0.0).amax(dim=1) + top + 16) * U
    else:
        p = here.double()
    counts = here.any(dim=1)
    y = torch.zeros_like(z).scatter_add_(1, at, p * here)
    loss = torch.where(counts, tau * tau * (entropy + lse * y.sum(dim=1) - (y * z).sum(dim=1)), 0.0)
    ez = (c.k + 2) * U * (h.abs() @ w.abs().t()) / tau
    size = z.abs().amax(dim=1) + lse.abs()
    elog = ez.amax(dim=1) + 4 * U * size + 520 * U
    assert bool(((d["lse"].double() - lse).abs() <= elog).all())
    eloss = tau * tau * (elog + ez.amax(dim=1) + 4 * U * size + teach * (2 * size + 2 + np.log(top)))
    assert bool(((d["loss"].double() - loss).abs() <= torch.where(counts, eloss, 0.0)).all())
    step, tiny = DT[c.dt][2], DT[c.dt][3]
    up = t["upstream"].double().abs() * tau * counts
    sm = torch.exp(z - lse[:, None])
    off = (sm - y).abs()
    edz = 2.0 ** -11 * off + (1 + 2.0 ** -11) * (((elog + 4 * U * size)[:, None] + ez + 8 * U) * sm + teach[:, None] * y + 4 * U * off)
    edz = (edz + 2.0 ** -38) * counts[:, None]  # of a row's own upstream
    dz = (sm - y) * (t["upstream"].double() * tau * counts)[:, None]
    wide_w = 2.0 ** -39 * w.abs().max() if c.dt == "bf16" else 0.0
    wide_h = 2.0 ** -39 * (h.abs().amax(dim=1) * counts).max()
    results = {"dh": (dz @ w, (up[:, None] * edz) @ w.abs() + (up[:, None] * (off + edz)) @ (wide_w + (c.v + 24) * U * w.abs())),
               "dw": (dz.t() @ h, (up[:, None] * edz).t() @ h.abs() + (up[:, None] * (off + edz)).t() @ ((c.n + 24) * U * h.abs())
                      + (up.max() * (off + edz) * counts[:, None]).sum(dim=0)[:, None] * wide_h)}
    for name, (ref, bound) in results.items():
        bound = bound + step * (ref.abs() + bound) + tiny
        err = (d[name].double() - ref).abs()
        assert bool((err <= bound).all()), (name, float((err / bound.clamp(min=1e-300)).max()))
    assert bool((d["dh"][~counts] == 0).all())


@pytest.mark.parametrize("top", [0, 5])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_values_of_rows_that_do_not_count_change_nothing(dt, top):
    """A padding row may hold any number: the gradients are those with zeros in it, to the bit."""
    announce("huge ignored row", dt, top)
    c = Case(40, 300, 64, dt, top=top, seed=21, absent=0.0)
    c.index[[3, 17]] = -100
    d = c.device()
    want = {}
    for fill in (0.0, 3e38 if dt == "bf16" else 65504.0):
        d["h"][[3, 17]] = fill
        c.forward(d)
        c.backward(d)
        torch.cuda.synchronize()
        got = {x: d[x].clone() for x in ("loss", "dh", "dw")}
        want = want or got
        assert all(torch.equal(got[x], want[x]) for x in want), [x for x in want if not torch.equal(got[x], want[x])]


@pytest.mark.parametrize("dt,decades", [("bf16", 60), ("bf16", 20), ("fp16", 20)])
@pytest.mark.parametrize("top,tau", [(0, 1.0), (6, 0.6)])
@pytest.mark.parametrize("n,v,k", [(41, 3000, 64), (200, 5000, 136)])
def test_upstreams_far_apart(n, v, k, top, tau, dt, decades):
    """Weights of the rows from 2^0 down to 2^-decades in one call: every row of dH keeps its own digits."""
    announce("upstreams", n, v, k, top, dt, decades)
    c = Case(n, v, k, dt, top=top, tau=tau, seed=22, absent=0.1)
    rng = np.random.default_rng(23)
    c.w = (c.w.double() + 0.3).to(c.w.dtype)  # softmax part and target part of a row of dH do not cancel
    c.upstream = (rng.choice([-1.0, 1.0], n) * rng.uniform(1, 2, n) * 2.0 ** -np.linspace(0, decades, n)).astype(np.float32)
    if dt == "fp16":
        c.upstream *= 2.0 ** 10  # results of the smallest rows stay normal numbers
    d = c.device()
    c.forward(d)
    c.backward(d)
    torch.cuda.synchronize()
    check_rows(c, d)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("top,tau,z", [(0, 1.0, 90.0), (1, 1.0, 90.0), (1, 2.0, 180.0), (1, 0.7, 63.0)])
@pytest.mark.parametrize("n,v,k", [(40, 600, 256), (300, 16500, 128), (600, 33000, 128), (33, 700, 1000)])
def test_certain_rows_have_no_loss(n, v, k, top, tau, z, dt):
    """The target's logit over tau is 90 and the others' are below 45 (asserted): their exponentials vanish beside one in
    fp32, so lse is the target's own logit over tau, the loss zero and no gradient left; nothing is negative."""
    announce("certain rows", n, v, k, top, tau, dt)
    c = Case(n, v, k, dt, top=top, tau=tau, seed=24, absent=0.0, scale=0.1)
    c.index[:, 0] = np.random.default_rng(25).permutation(v)[:n]
    h = c.h.double()
    w = c.w.double()
    w[torch.from_numpy(c.index[:, 0])] = z * h / (h * h).sum(dim=1, keepdim=True)
    c.w = w.to(c.w.dtype)
    c.upstream = np.ones(n, np.float32)
    zz = c.h.to(DEV).double() @ c.w.to(DEV).double().t() / tau
    at = torch.from_numpy(c.index).to(DEV)
    others = zz.scatter(1, at, -np.inf)
    assert float(zz.gather(1, at).min()) > 88 and float(others.max()) < 45
    d = c.device()
    c.forward(d)
    c.backward(d)
    torch.cuda.synchronize()
    for x in ("loss", "dh", "dw"):
        assert bool((d[x] == 0).all()), (x, float(d[x].double().abs().max()))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("n,v,k", [(70, 900, 72), (300, 16500, 200), (600, 33000, 136), (5, 300, 4104)])
def test_listed_logits_are_the_same_number_in_both_losses(n, v, k, dt):
    """A logit is one number, whichever call reports it: cross entropy's at the target and distillation's at an entry."""
    announce("logits", n, v, k, dt)
    c = Case(n, v, k, dt, top=19, seed=26, absent=0.0)
    c.teacher = np.random.default_rng(27).standard_normal(c.teacher.shape).astype(np.float32)
    d = c.device()
    c.forward(d)
    for j in (0, 7, 18):
        e = Case(1, 1, 8, dt)
        e.n, e.v, e.k, e.h, e.w, e.index, e.upstream = n, v, k, c.h, c.w, c.index[:, j:j + 1].copy(), c.upstream
        f = e.device()
        e.forward(f)
        torch.cuda.synchronize()
        assert torch.equal(f["zt"][:, 0], d["zt"][:, j])
        assert torch.equal(f["lse"], d["lse"])


@pytest.mark.parametrize("tau", [1e-25, 1e-8, 1e-5])
@pytest.mark.parametrize("n,v,k", [(50, 700, 64), (300, 16500, 64)])
def test_temperatures_that_leave_one_word(n, v, k, tau):
    """H rows pick one feature and W holds multiples of 1/16: the row's largest logit is 1/16 or more above the others,
    hundreds and more over tau, so both softmaxes are one word each.  Then lse is the largest logit over tau, the loss
    tau times the distance of the two words' logits, and a row of dH the difference of two rows of W (multiples of 1/16
    up to 32: a difference is exact in fp32, so one rounding to bf16, 2^-8)."""
    announce("temperature", n, v, k, tau)
    rng = np.random.default_rng(28)
    c = Case(n, v, k, "bf16", top=8, tau=float(np.float32(tau)), seed=28, absent=0.0)
    feature = rng.integers(0, k, n)
    h = np.zeros((n, k))
    h[np.arange(n), feature] = 1.0
    w = rng.integers(-256, 240, size=(v, k)) / 16.0
    best = rng.permutation(v)[:k]
    w[best, np.arange(k)] = 15.0 + 1.0 / 16  # the largest of its column
    c.h, c.w = torch.from_numpy(h).bfloat16(), torch.from_numpy(w).bfloat16()
    w = c.w.double().numpy()
    z = h @ w.T
    two = np.sort(z, axis=1)[:, -2:]
    assert np.all(two[:, 1] - two[:, 0] >= 1 / 16)
    c.index = np.stack([rng.permutation(v)[:8] for _ in range(n)])
    c.teacher = np.stack([rng.permutation(8) for _ in range(n)]).astype(np.float32)
    c.upstream = np.full(n, 1 / c.tau, np.float32)
    d = c.device()
    c.forward(d)
    c.backward(d)
    torch.cuda.synchronize()
    top = z.argmax(axis=1)
    word = c.index[np.arange(n), c.teacher.argmax(axis=1)]
    # two roundings of z / tau and one of the sum, and their differences scaled back
    m = z.max(axis=1) / c.tau
    assert np.all(np.abs(d["lse"].double().cpu().numpy() - m) <= 3 * U * np.abs(m))
    loss = c.tau * (z[np.arange(n), top] - z[np.arange(n), word])
    assert np.all(np.abs(d["loss"].double().cpu().numpy() - loss) <= c.tau * 8 * U * np.abs(z).max(axis=1))
    # the two 1 / tau of upstream and of 1 / tau times tau: one within 2 U
    ref = np.where((top == word)[:, None], 0.0, w[top] - w[word])
    assert np.all(np.abs(d["dh"].double().cpu().numpy() - ref) <= (2.0 ** -8 + 2.0 ** -11 + 4 * U) * np.abs(ref) + 2.0 ** -20)


@pytest.mark.parametrize("tau", [0.1, 0.3, 0.77, 1.3, 3.0, 7.1, 11.0])
def test_certain_rows_at_any_temperature(tau):
    """Whatever the inverse of tau rounds to, lse and a listed logit take the same product (the rows of
    test_certain_rows_have_no_loss, logits of 90 and below 45 over tau)."""
    announce("certain rows at", tau)
    n, v, k = 60, 900, 256
    c = Case(n, v, k, "bf16", top=1, tau=tau, seed=29, absent=0.0, scale=0.1 * tau)
    c.index[:, 0] = np.random.default_rng(30).permutation(v)[:n]
    h, w = c.h.double(), c.w.double()
    w[torch.from_numpy(c.index[:, 0])] = 90.0 * tau * h / (h * h).sum(dim=1, keepdim=True)
    c.w = w.to(c.w.dtype)
    zz = c.h.to(DEV).double() @ c.w.to(DEV).double().t() / tau
    at = torch.from_numpy(c.index).to(DEV)
    assert float(zz.gather(1, at).min()) > 88 and float(zz.scatter(1, at, -np.inf).max()) < 45
    d = c.device()
    c.forward(d)
    c.backward(d)
    torch.cuda.synchronize()
    for x in ("loss", "dh", "dw"):
        assert bool((d[x] == 0).all()), (x, float(d[x].double().abs().max()))
