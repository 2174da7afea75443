"""Plain 64-bit definitions of the block-scaled 8-bit operands, their product
and the output-layer losses.  TEST INFRASTRUCTURE ONLY, like the rest of this
package: NumPy in float64, no code shared with the product.

``F8``: (mantissa bits, smallest normal exponent, largest value) of the two
8-bit formats of the OCP specification "OCP 8-bit Floating Point (OFP8)".
"""

from __future__ import annotations

import numpy as np

__all__ = ["F8", "f8_round", "f8_decode", "quantize", "scale_values", "dequantize", "product_f8", "product_f8_bound",
           "linear_loss"]

F8 = {"e4m3": (3, -6, 448.0), "e5m2": (2, -14, 57344.0)}


def f8_round(y: np.ndarray, kind: str) -> np.ndarray:
    """float64 -> the nearest 8-bit value (ties to even) as float64, |y| <= the largest value."""
    mant, emin, _ = F8[kind]
    a = np.abs(y)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.where(a > 0, np.floor(np.log2(np.where(a > 0, a, 1.0))), emin)
    e = np.where(np.ldexp(1.0, e.astype(int)) > a, e - 1, e)  # a logarithm rounded up to a whole number
    step = np.ldexp(1.0, (np.maximum(e, emin) - mant).astype(int))
    return np.copysign(np.rint(a / step) * step, y)


def f8_decode(bits: np.ndarray, kind: str) -> np.ndarray:
    """Bytes -> float64."""
    mant, emin, _ = F8[kind]
    b = np.asarray(bits, dtype=np.uint8).astype(np.int64)
    e, m = (b & 127) >> mant, b & ((1 << mant) - 1)
    v = np.where(e == 0, np.ldexp(m.astype(float), emin - mant), np.ldexp((m + (1 << mant)).astype(float), e - 1 + emin - mant))
    if kind == "e4m3":
        v = np.where((b & 127) == 127, np.nan, v)
    else:
        v = np.where((b & 127) == 124, np.inf, np.where((b & 127) > 124, np.nan, v))
    return np.where(b >> 7, -v, v)


def quantize(x: np.ndarray, kind: str, block_rows: int):
    """x float64 [R][C] -> (values float64 [R][C], exponents int [ceil(R/block_rows)][ceil(C/128)])."""
    r, c = x.shape
    fmax = F8[kind][2]
    nr, nc = -(-r // block_rows), -(-c // 128)
    q = np.zeros_like(x, dtype=np.float64)
    ex = np.zeros((nr, nc), dtype=np.int64)
    for i in range(nr):
        for j in range(nc):
            s = (slice(i * block_rows, (i + 1) * block_rows), slice(128 * j, 128 * j + 128))
            blk = x[s].astype(np.float64)
            fin = np.isfinite(blk)
            a = np.max(np.abs(blk[fin]), initial=0.0)
            e = 0
            if a > 0:
                e = -127
                while a > fmax * 2.0 ** e:
                    e += 1
            ex[i, j] = e
            out = np.full(blk.shape, np.nan)
            out[fin] = f8_round(blk[fin] * 2.0 ** -e, kind)
            if kind == "e5m2":
                out = np.where(np.isinf(blk), blk, out)
            q[s] = out
    return q, ex


def scale_values(scale: np.ndarray, rows: int, k: int, square: bool) -> np.ndarray:
    """Stored scales (uint8 exponents or floats) -> float64 [rows][k]."""
    s = 2.0 ** (scale.astype(np.float64) - 127) if scale.dtype == np.uint8 else scale.astype(np.float64)
    return np.repeat(np.repeat(s, 128 if square else 1, axis=0)[:rows], 128, axis=1)[:, :k]


def dequantize(bits, kind, scale, square):
    v = f8_decode(bits, kind)
    return v * scale_values(scale, v.shape[0], v.shape[1], square)


def product_f8(a: np.ndarray, b: np.ndarray) -> np.ndarray:
    return a @ b.T


def product_f8_bound(a: np.ndarray, b: np.ndarray) -> np.ndarray:
    """First-order bound of an fp32 evaluation in any order: each of the k - 1
    additions, and the three multiplications a block scale may take, is off by
    at most one unit in the last place (2^-23; half that where it rounds to
    nearest) of a partial sum that the sum of magnitudes bounds."""
    k = a.shape[1]
    return (k + 3) * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)


def linear_loss(h, w, index, weight_logits=None, tau=1.0, upstream=None):
    """Cross entropy (index [n], weight_logits None) or distillation (index
    [n][T], teacher logits [n][T]) of the logits h w^T, in float64, with the
    gradients if `upstream` [n] is given.  Entries outside [0, v) are absent."""
    h, w = np.asarray(h, np.float64), np.asarray(w, np.float64)
    n, v = h.shape[0], w.shape[0]
    z = (h @ w.T) / tau
    top = z.max(axis=1, keepdims=True)
    lse = np.log(np.exp(z - top).sum(axis=1)) + top[:, 0]
    index = np.asarray(index).reshape(n, -1)
    loss = np.zeros(n)
    target = np.zeros((n, v))
    mass = np.zeros(n)
    for i in range(n):
        here = (index[i] >= 0) & (index[i] < v)
        if weight_logits is not None:
            here &= np.asarray(weight_logits)[i] > -np.inf
        if not here.any():
            continue
        if weight_logits is None:
            p = np.ones(1)
        else:
            t = np.asarray(weight_logits, np.float64)[i][here] / tau
            p = np.exp(t - t.max())
            p /= p.sum()
        ids = index[i][here]
        logp = np.log(np.where(p > 0, p, 1.0))
        loss[i] = tau * tau * np.sum(p * (logp - (z[i, ids] - lse[i])))
        np.add.at(target[i], ids, p)
        mass[i] = 1.0
    out = {"loss": loss, "lse": lse, "target": target}
    if upstream is not None:
        dz = tau * np.asarray(upstream, np.float64)[:, None] * (mass[:, None] * np.exp(z - lse[:, None]) - target)
        out.update(dz=dz, dh=dz @ w, dw=dz.T @ h)
    return out
