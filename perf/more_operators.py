"""The library's feed-forward and 4-bit operators as measured cases.

Four operators, each in its plain form (elementary torch operations in fp32)
and as a program calls it of ``tiled_movement_amd``:

* ``gated``  -- y = act(x Wg^T) * (x Wu^T), a gated feed-forward block's two
                projections with the activation and the product, and its
                gradients;
* ``quant4`` -- weights to 4 bits with a scale (and on request a zero point)
                per group along k, and back;
* ``gemm4``  -- C = X W^T of such weights for a few rows of X, and the gated
                block of two of them;
* ``clip``   -- the norm of all gradients of a model together, and the
                gradients scaled down to a largest norm.

Sizes are generic ones and those of the library's own workloads (4096, 8192).
"""

from __future__ import annotations

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token through a feed-forward block while serving: reads both weights
        {"name": "gated 1x4096 to 8192", "op": "gated", "n": 1, "k": 4096, "f": 8192, "x": "bf16", "act": "silu", "grad": False},
        # a ragged batch of tokens, odd widths
        {"name": "gated 77x2056 to 5000", "op": "gated", "n": 77, "k": 2056, "f": 5000, "x": "fp16", "act": "gelu_tanh",
         "grad": False},
        # a prompt
        {"name": "gated 4096x4096 to 8192", "op": "gated", "n": 4096, "k": 4096, "f": 8192, "x": "bf16", "act": "silu",
         "grad": False},
        # a small training step of odd sizes, fp16 results
        {"name": "gated step 333x1000 to 2777", "op": "gated", "n": 333, "k": 1000, "f": 2777, "x": "fp16", "act": "gelu",
         "grad": True},
        # a training step: the block forward, then back to its input and both weights
        {"name": "gated step 4096x4096 to 8192", "op": "gated", "n": 4096, "k": 4096, "f": 8192, "x": "bf16", "act": "silu",
         "grad": True},
        # a layer's weights to 4 bits for serving, symmetric
        {"name": "quant4 8192x4096", "op": "quant4", "n": 8192, "k": 4096, "w": "bf16", "s": "bf16", "group": 128, "zero": False},
        # fp32 master weights of odd sizes, short groups with zero points
        {"name": "quant4 5001x6048 zero points", "op": "quant4", "n": 5001, "k": 6048, "w": "fp32", "s": "fp16", "group": 32,
         "zero": True},
        # one token through a layer of 4-bit weights: latency and the weights' bytes
        {"name": "gemm4 1x8192x4096", "op": "gemm4", "m": 1, "n": 8192, "k": 4096, "x": "bf16", "group": 128, "zero": False,
         "gated": False, "act": "silu"},
        # some sequences decoded together, odd widths, short groups with zero points
        {"name": "gemm4 19x5000x4160 zero points", "op": "gemm4", "m": 19, "n": 5000, "k": 4160, "x": "fp16", "group": 32,
         "zero": True, "gated": False, "act": "silu"},
        # a decoded batch through the gated block of 4-bit weights
        {"name": "gemm4 gated 8x8192x8192", "op": "gemm4", "m": 8, "n": 8192, "k": 8192, "x": "bf16", "group": 128,
         "zero": False, "gated": True, "act": "silu"},
        # a small model's gradients of odd sizes and mixed types: latency
        {"name": "clip 40 tensors to 60000", "op": "clip", "count": 40, "smallest": 1, "largest": 60000, "mix": True,
         "over": 3.0},
        # a block's gradients, bf16 with some fp32: bytes
        {"name": "clip 32 tensors to 33554432", "op": "clip", "count": 32, "smallest": 4096, "largest": 33554432, "mix": True,
         "over": 3.0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated", "gated", "quant4", "gemm4", "gemm4", "clip"])
    if op == "gated":
        return {"op": op, "n": _log_int(rng, 1, 4096), "k": 8 * _log_int(rng, 8, 512), "f": _log_int(rng, 64, 8192),
                "x": rng.choice(["bf16", "bf16", "fp16"]), "act": rng.choice(["silu", "silu", "gelu", "gelu_tanh"]),
                "grad": rng.random() < 0.5}
    if op == "quant4":
        return {"op": op, "n": _log_int(rng, 1, 8192), "k": 32 * _log_int(rng, 2, 128),
                "w": rng.choice(["bf16", "fp16", "fp32"]), "s": rng.choice(["bf16", "fp16"]),
                "group": rng.choice([32, 64, 128]), "zero": rng.random() < 0.5}
    if op == "gemm4":
        return {"op": op, "m": _log_int(rng, 1, 64), "n": _log_int(rng, 64, 8192), "k": 32 * _log_int(rng, 4, 256),
                "x": rng.choice(["bf16", "fp16"]), "group": rng.choice([32, 64, 128, 128]), "zero": rng.random() < 0.4,
                "gated": rng.random() < 0.4, "act": rng.choice(["silu", "gelu", "gelu_tanh"])}
    return {"op": op, "count": rng.randint(1, 48), "smallest": 1, "largest": _log_int(rng, 100, 1 << 24),
            "mix": rng.random() < 0.6, "over": rng.choice([0.5, 3.0, 40.0])}


# ----------------------------------------------------------------- inputs
def _groups(w, group, fill):
    """[n][k] as [n][groups][group], the last group filled up."""
    k = w.shape[1]
    return torch.nn.functional.pad(w, (0, -k % group), value=fill).unflatten(1, (-1, group))


def _quant4(w, group, zero, stype):
    """Codes 0..15 as int32 [n][k], scales of stype [n][groups], zero points uint8 [n][groups] or None, of an fp32 matrix."""
    k = w.shape[1]
    b = _groups(w, group, 0.0)
    if zero:
        lo, hi = b.amin(dim=2).clamp(max=0.0), b.amax(dim=2).clamp(min=0.0)
        s = ((hi - lo) / 15.0).to(stype)
        step = torch.where(s > 0, s.float(), 1.0)
        z = torch.round(-lo / step).clamp(0, 15)
    else:
        s = (b.abs().amax(dim=2) / 7.0).to(stype)
        step = torch.where(s > 0, s.float(), 1.0)
        z = torch.full_like(step, 8.0)
    code = (torch.round(b / step[:, :, None]) + z[:, :, None]).clamp(0, 15)
    code = torch.where((s > 0)[:, :, None], code, z[:, :, None])
    return code.flatten(1)[:, :k].to(torch.int32), s, z.to(torch.uint8) if zero else None


def _pack4(code):
    """Two codes a byte, the even column's in the low half."""
    return (code[:, 0::2] | code[:, 1::2] << 4).to(torch.uint8)


def _unpack4(q):
    return torch.stack((q & 15, q >> 4), dim=2).flatten(1).to(torch.int32)


def _values4(q, s, z, group, k):
    """fp32 [n][k] of packed codes."""
    code = _groups(_unpack4(q).float(), group, 0.0)
    z = 8.0 if z is None else z.float()[:, :, None]
    return ((code - z) * s.float()[:, :, None]).flatten(1)[:, :k]


def _sizes(case):
    """Sizes of a model's gradients: from the smallest to the largest over their logarithm, odd ones among them."""
    n, lo, hi = case["count"], math.log(case["smallest"]), math.log(case["largest"])
    if n == 1:
        return [case["largest"]]
    return [max(1, int(round(math.exp(lo + (hi - lo) * i / (n - 1))))) for i in range(n)]


def _kinds(case):
    return ["bf16" if not case["mix"] else ("bf16", "bf16", "fp32", "fp16")[i % 4] for i in range(case["count"])]


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 29)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = dict(case)
    if case["op"] == "gated":
        n, k, f, t = case["n"], case["k"], case["f"], TYPES[case["x"]]
        s["xs"] = randn(n, k).to(t)
        s["wg"] = (randn(f, k) * (1.2 / math.sqrt(k))).to(t)
        s["wu"] = (randn(f, k) * (1.0 / math.sqrt(k))).to(t)
        if case["grad"]:
            # gradients of tokens of different weight, under a loss scale
            s["dy"] = (randn(n, f) * torch.exp(0.5 * randn(n, 1)) * 0.05).to(t)
    elif case["op"] == "quant4":
        w = randn(case["n"], case["k"]) * 0.02 * torch.exp(0.3 * randn(case["n"], 1))
        s["ws"] = w.to(TYPES[case["w"]])
    elif case["op"] == "gemm4":
        t = TYPES[case["x"]]
        s["xs"] = (randn(case["m"], case["k"]) * torch.exp(0.3 * randn(case["m"], 1))).to(t)
        for i in range(2 if case["gated"] else 1):
            w = randn(case["n"], case["k"]) * (1.0 / math.sqrt(case["k"]))
            code, s["s%d" % i], s["z%d" % i] = _quant4(w, case["group"], case["zero"], t)
            s["q%d" % i] = _pack4(code)
    else:
        s["grads"] = [(randn(n) * math.exp(0.1 * (i % 7))).to(TYPES[t])
                      for i, (n, t) in enumerate(zip(_sizes(case), _kinds(case)))]
        s["clipped"] = [torch.empty_like(t) for t in s["grads"]]
        s["max_norm"] = math.sqrt(sum(_sizes(case))) * 1.4 / case["over"]
    return s


# ------------------------------------------------------------ plain forms
def _act(name, z):
    """(act(z), its derivative)."""
    if name == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        th = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * z * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * z * (1.0 - th * th) * c * (1.0 + 3 * 0.044715 * z * z)
    sg = 1.0 / (1.0 + torch.exp(-z))
    return z * sg, sg * (1.0 + z * (1.0 - sg))


def _plain_gated(s):
    x, wg, wu, t = s["xs"].float(), s["wg"].float(), s["wu"].float(), s["xs"].dtype
    gate, up = torch.mm(x, wg.t()), torch.mm(x, wu.t())
    a, da = _act(s["act"], gate)
    out = {"y": (a * up).to(t)}
    if s["grad"]:
        dy = s["dy"].float()
        dg, du = dy * up * da, dy * a
        out["dx"] = (torch.mm(dg, wg) + torch.mm(du, wu)).to(t)
        out["dwg"], out["dwu"] = torch.mm(dg.t(), x).to(t), torch.mm(du.t(), x).to(t)
    return out


def _plain_quant4(s):
    code, sc, z = _quant4(s["ws"].float(), s["group"], s["zero"], TYPES[s["s"]])
    out = {"scale": sc, "w": _values4(_pack4(code), sc, z, s["group"], s["k"]).to(sc.dtype)}
    if z is not None:
        out["zero"] = z
    return out


def _plain_gemm4(s):
    x = s["xs"].float()
    c = torch.mm(x, _values4(s["q0"], s["s0"], s["z0"], s["group"], s["k"]).t())
    if s["gated"]:
        c = _act(s["act"], c)[0] * torch.mm(x, _values4(s["q1"], s["s1"], s["z1"], s["group"], s["k"]).t())
    return {"c": c.to(s["xs"].dtype)}


def _plain_clip(s):
    norm = torch.stack([t.double().square().sum() for t in s["grads"]]).sum().sqrt()
    factor = (s["max_norm"] / norm).clamp(max=1.0).float()
    return {"norm": norm.float().reshape(1), "grads": [(t.float() * factor).to(t.dtype) for t in s["grads"]]}


# ------------------------------------------------- the library's operators
def _own_gated(s):
    import tiled_movement_amd as T

    x, n, f, k = s["xs"], s["n"], s["f"], s["k"]
    kw = {"x_type": {"bf16": T.X_BF16, "fp16": T.X_F16}[s["x"]],
          "act": {"silu": T.ACT_SILU, "gelu": T.ACT_GELU, "gelu_tanh": T.ACT_GELU_TANH}[s["act"]]}
    y = torch.empty(n, f, dtype=x.dtype, device=x.device)
    out = {"y": y}
    if s["grad"]:
        kw["pre"] = torch.empty(2, n, f, dtype=torch.float32, device=x.device)
    T.swz_gated(x, s["wg"], s["wu"], y, n, f, k, **kw)
    if s["grad"]:
        ws = torch.empty(T.swz_gated_workspace(n, f, k), dtype=torch.uint8, device=x.device)
        dx, dwg, dwu = torch.empty_like(x), torch.empty_like(s["wg"]), torch.empty_like(s["wu"])
        T.swz_gated_grad(x, s["wg"], s["wu"], s["dy"], dx, dwg, dwu, n, f, k, ws, **kw)
        out.update(dx=dx, dwg=dwg, dwu=dwu)
    return out


def _own_quant4(s):
    import tiled_movement_amd as T

    w, n, k, group = s["ws"], s["n"], s["k"], s["group"]
    stype, groups = {"bf16": T.X_BF16, "fp16": T.X_F16}[s["s"]], -(-k // group)
    q = torch.empty(n, k // 2, dtype=torch.uint8, device=w.device)
    sc = torch.empty(n, groups, dtype=TYPES[s["s"]], device=w.device)
    z = torch.empty(n, groups, dtype=torch.uint8, device=w.device) if s["zero"] else None
    T.swz_quant_w4(w, q, sc, n, k, group=group, w_type={"bf16": T.X_BF16, "fp16": T.X_F16, "fp32": T.X_F32}[s["w"]], x_type=stype,
                   zero=z)
    back = torch.empty(n, k, dtype=sc.dtype, device=w.device)
    T.swz_dequant_w4(q, sc, back, n, k, group=group, x_type=stype, zero=z)
    out = {"scale": sc, "w": back}
    if z is not None:
        out["zero"] = z
    return out


def _own_gemm4(s):
    import tiled_movement_amd as T

    x, m, n, k = s["xs"], s["m"], s["n"], s["k"]
    c = torch.empty(m, n, dtype=x.dtype, device=x.device)
    xt = {"bf16": T.X_BF16, "fp16": T.X_F16}[s["x"]]
    if s["gated"]:
        T.swz_gated_w4(x, s["q0"], s["s0"], s["q1"], s["s1"], c, m, n, k, group=s["group"], x_type=xt, zero_g=s["z0"], zero_u=s["z1"],
                       act={"silu": T.ACT_SILU, "gelu": T.ACT_GELU, "gelu_tanh": T.ACT_GELU_TANH}[s["act"]])
    else:
        T.swz_gemm_w4(x, s["q0"], s["s0"], c, m, n, k, group=s["group"], x_type=xt, zero=s["z0"])
    return {"c": c}


def _own_clip(s):
    import tiled_movement_amd as T

    dev = s["grads"][0].device
    ws = torch.empty(T.swz_grad_norm_workspace(s["grads"]), dtype=torch.uint8, device=dev)
    norm = torch.empty(2, dtype=torch.float32, device=dev)
    T.swz_clip_grads(s["grads"], s["max_norm"], norm, ws, out=s["clipped"])
    return {"norm": norm[:1], "grads": s["clipped"]}


def run(state):
    if own:
        return {"gated": _own_gated, "quant4": _own_quant4, "gemm4": _own_gemm4, "clip": _own_clip}[state["op"]](state)
    return {"gated": _plain_gated, "quant4": _plain_quant4, "gemm4": _plain_gemm4, "clip": _plain_clip}[state["op"]](state)


# -------------------------------------------------- what each has to do
def work(case):
    if case["op"] == "gated":
        n, k, f = case["n"], case["k"], case["f"]
        if not case["grad"]:
            return {"bytes": 2 * (n * k + 2 * f * k + n * f), "flops": 4 * n * f * k}
        # both projections, and two products as large for each of x and the weights
        return {"bytes": 2 * (2 * n * k + 4 * f * k + 2 * n * f), "flops": 12 * n * f * k}
    if case["op"] == "quant4":
        n, k = case["n"], case["k"]
        side = n * -(-k // case["group"]) * (3 if case["zero"] else 2)
        # to 4 bits, and from there back to 16
        return {"bytes": n * k * (TYPES[case["w"]].itemsize + 0.5) + n * k * 2.5 + 2 * side, "flops": 0}
    if case["op"] == "gemm4":
        m, n, k, both = case["m"], case["n"], case["k"], 2 if case["gated"] else 1
        side = n * -(-k // case["group"]) * (3 if case["zero"] else 2)
        return {"bytes": 2 * m * k + both * (n * k / 2 + side) + 2 * m * n, "flops": 2 * both * m * n * k}
    held = sum(n * TYPES[t].itemsize for n, t in zip(_sizes(case), _kinds(case)))
    return {"bytes": 2 * held + 4, "flops": 0}


# ------------------------------------------------------------ in 64 bits
def _act64(name, z):
    """act(z) in 64 bits, as a function that can be differentiated."""
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gated":
        x, wg, wu = s["xs"].double(), s["wg"].double(), s["wu"].double()
        gate, up = (x @ wg.t()).requires_grad_(case["grad"]), x @ wu.t()
        a = _act64(case["act"], gate)
        out = {"y": (a * up).detach()}
        if case["grad"]:
            dy = s["dy"].double()
            dg = torch.autograd.grad(a, gate, dy * up)[0]
            du = dy * a.detach()
            out.update(dx=dg @ wg + du @ wu, dwg=dg.t() @ x, dwu=du.t() @ x)
        return out
    if case["op"] == "quant4":
        w, group, t = s["ws"].double(), case["group"], TYPES[case["s"]]
        n, k = w.shape
        pad = torch.zeros(n, -(-k // group) * group, dtype=torch.float64, device=w.device)
        pad[:, :k] = w
        b = pad.view(n, -1, group)
        if case["zero"]:
            low, high = -(-b).amax(dim=2).clamp(min=0.0), b.amax(dim=2).clamp(min=0.0)
            unrounded = (high - low) / 15.0
        else:
            low, unrounded = None, b.abs().amax(dim=2) / 7.0
        step = unrounded.float().to(t).double()
        lowest = (low / step).round().nan_to_num(0.0) if case["zero"] else torch.full_like(step, -8.0)
        lowest = lowest.clamp(-15.0, 0.0)
        code = (b / step[:, :, None]).round().nan_to_num(0.0)
        code = torch.minimum(torch.maximum(code, lowest[:, :, None]), lowest[:, :, None] + 15.0)
        return {"scale": unrounded, "w": (code * step[:, :, None]).flatten(1)[:, :k], **({"zero": None} if case["zero"] else {})}
    if case["op"] == "gemm4":
        def weights(i):
            q, sc, z = s["q%d" % i].long(), s["s%d" % i].double(), s["z%d" % i]
            low, high = q % 16, q // 16
            code = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.float64, device=q.device)
            code[:, 0::2], code[:, 1::2] = low.double(), high.double()
            code -= 8.0 if z is None else z.double().repeat_interleave(case["group"], dim=1)[:, :case["k"]]
            return code * sc.repeat_interleave(case["group"], dim=1)[:, :case["k"]]

        c = s["xs"].double() @ weights(0).t()
        if case["gated"]:
            c = _act64(case["act"], c) * (s["xs"].double() @ weights(1).t())
        return {"c": c}
    norm = math.sqrt(sum(torch.dot(t.double(), t.double()).item() for t in s["grads"]))
    factor = min(1.0, s["max_norm"] / norm)
    return {"norm": torch.full((1,), norm, dtype=torch.float64), "grads": [t.double() * factor for t in s["grads"]]}
