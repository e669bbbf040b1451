"""Plain 64-bit definitions of the feed-forward network's operators and of the
combine with dropout.

Test infrastructure, written from the formulas; nothing is shared with the
CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

ACTIVATIONS = ("none", "relu", "gelu", "silu", "swiglu")

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def cdf(x):
    return 0.5 * _erfc(-np.asarray(x, np.float64) / math.sqrt(2.0))


def activation(z, act: str):
    if act == "relu":
        return np.where(z < 0, 0.0, z)
    if act == "gelu":
        return z * cdf(z)
    if act == "silu":
        return z * sigmoid(z)
    if act == "swiglu":
        f = z.shape[-1] // 2
        return z[..., :f] * sigmoid(z[..., :f]) * z[..., f:]
    return np.array(z)


def slope(z, act: str):
    """Derivative of the activations that take one value."""
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "gelu":
        return cdf(z) + z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "silu":
        s = sigmoid(z)
        return s * (1 + z * (1 - s))
    return np.ones_like(z)


def activation_backward(z, d_out, act: str):
    if act != "swiglu":
        return d_out * slope(z, act)
    f = z.shape[-1] // 2
    g, u = z[..., :f], z[..., f:]
    return np.concatenate([d_out * u * slope(g, "silu"), d_out * g * sigmoid(g)], -1)


def sensitivity(z, act: str, err):
    """How far act(z) can move, to first order, when z is off by at most err."""
    if act != "swiglu":
        return np.abs(slope(z, act)) * err
    f = z.shape[-1] // 2
    g, u = z[..., :f], z[..., f:]
    return np.abs(u * slope(g, "silu")) * err[..., :f] + np.abs(g * sigmoid(g)) * err[..., f:]


def philox(seed: int, offset: int, groups: np.ndarray) -> np.ndarray:
    """Philox4x32-10 of the counters (group, offset): uint32 [..., 4]."""
    low = np.uint64(0xFFFFFFFF)
    g = np.asarray(groups, np.uint64)
    c = [g & low, g >> np.uint64(32), np.full_like(g, offset & 0xFFFFFFFF),
         np.full_like(g, (offset >> 32) & 0xFFFFFFFF)]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, -1).astype(np.uint32)


def dropout_factor(n: int, p: float, seed: int, offset: int) -> np.ndarray:
    """What each of n elements (a multiple of 8) is multiplied by: 0 or 1 / (1 - p'), p' = p in 65536ths."""
    cut = math.floor(65536 * p + 0.5)
    w = philox(seed, offset, np.arange(n // 8))
    numbers = np.stack([w & np.uint32(0xFFFF), w >> np.uint32(16)], -1).reshape(-1)
    return np.where(numbers >= cut, 65536.0 / (65536 - cut), 0.0)


def combine_dropout(y, dst, gates, residual, factor):
    """y [N][Hp], dst and gates [T][K], factor [T][Hp]."""
    total = (y[dst] * gates[..., None]).sum(1)
    out = np.where(factor != 0, total * factor, 0.0)
    return out if residual is None else out + residual


def combine_dropout_backward(y, dst, gates, d_out, factor):
    """What was dropped counts as 0 whatever y, the gate and d_out are."""
    kept = (factor != 0)[:, None]
    with np.errstate(invalid="ignore"):
        d = (d_out * factor)[:, None]
        d_y = np.zeros_like(y)
        d_y[dst] = np.where(kept, gates[..., None] * d, 0.0)
        return d_y, np.where(kept, y[dst] * d, 0.0).sum(-1)
