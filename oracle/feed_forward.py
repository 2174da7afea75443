"""Plain definitions of the gated feed-forward block, 4-bit weights and the
norm of many tensors.  TEST INFRASTRUCTURE ONLY, like the rest of this package:
NumPy in float64 (the quantizer's quotients in float32, as it is defined), no
code shared with the product.
"""

from __future__ import annotations

import math

import numpy as np

__all__ = ["ACTS", "activation", "gated", "gated_grad", "quant_w4", "pack_w4", "unpack_w4", "dequant_w4", "norm"]

ACTS = ("silu", "gelu", "gelu_tanh")

_erf = np.vectorize(math.erf, otypes=[np.float64])


def activation(name: str, z: np.ndarray):
    """(act(z), its derivative)."""
    if name == "silu":
        s = 0.5 * (1 + np.tanh(z / 2))
        return z * s, s * (1 + z * (1 - s))
    if name == "gelu":
        cdf = 0.5 * (1 + _erf(z / math.sqrt(2)))
        return z * cdf, cdf + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    q = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    t = np.tanh(q)
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)


def gated(x, wg, wu, act):
    """(y, g, u) of float64 operands."""
    g, u = x @ wg.T, x @ wu.T
    return activation(act, g)[0] * u, g, u


def gated_grad(x, wg, wu, act, dy):
    """(dx, dwg, dwu, dg, du)."""
    _, g, u = gated(x, wg, wu, act)
    a, da = activation(act, g)
    dg, du = dy * u * da, dy * a
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dg, du


def quant_w4(w: np.ndarray, group: int, zero: bool, to_type):
    """float32 [n][k] -> (codes [n][k], scales float32 [n][groups], zero points [n][groups]).  to_type: rounds a float32
    array to the scales' type (as float32; what leaves it becomes infinite)."""
    n, k = w.shape
    groups = -(-k // group)
    code, scale, zp = np.zeros((n, k), np.int64), np.zeros((n, groups), np.float32), np.full((n, groups), 0 if zero else 8)
    for j in range(groups):
        b = w[:, j * group:(j + 1) * group].astype(np.float32)
        with np.errstate(all="ignore"):
            if zero:
                lo, hi = np.minimum(b.min(axis=1), 0), np.maximum(b.max(axis=1), 0)
                s = (hi - lo) * np.float32(1 / np.float32(15))
            else:
                s = np.abs(b).max(axis=1) * np.float32(1 / np.float32(7))
            s = to_type(s.astype(np.float32))
            bad = ~np.isfinite(b).all(axis=1) | ~np.isfinite(s)
            s = np.where(bad, np.float32(np.nan), s).astype(np.float32)
            some = s > 0
            step = np.where(some, s, np.float32(1)).astype(np.float32)
            if zero:
                zp[:, j] = np.where(some, np.clip(np.rint(np.where(some, -lo, 0) / step), 0, 15), 0)
            q = np.rint(np.where(some[:, None], b, 0) / step[:, None]) + zp[:, j:j + 1]
        code[:, j * group:(j + 1) * group] = np.where(some[:, None], np.clip(q, 0, 15), zp[:, j:j + 1])
        scale[:, j] = s
    return code, scale, zp


def pack_w4(code):
    return (code[:, 0::2] | code[:, 1::2] << 4).astype(np.uint8)


def unpack_w4(q):
    return np.stack([q & 15, q >> 4], axis=2).reshape(q.shape[0], -1).astype(np.int64)


def dequant_w4(q, scale, zero, group):
    """float64 [n][k] of packed codes; zero None: 8."""
    code = unpack_w4(q).astype(np.float64)
    k = code.shape[1]
    spread = lambda a: np.repeat(np.asarray(a, np.float64), group, axis=1)[:, :k]  # noqa: E731
    return (code - (8 if zero is None else spread(zero))) * spread(scale)


def norm(tensors):
    return math.sqrt(sum(float(np.sum(np.square(np.asarray(t, np.float64)))) for t in tensors))
