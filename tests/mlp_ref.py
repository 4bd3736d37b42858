"""64-bit forms of the operators around an MLP's products, and their error bounds.

NumPy in double throughout, written from the definitions; nothing here calls the library.
"""

from __future__ import annotations

import numpy as np
from scipy.special import ndtr

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
GELU_C = np.sqrt(2.0 / np.pi)
U32 = 2.0 ** -23     # one unit in the last place of an FP32 in [1, 2)


def act(z, name):
    if name == "none":
        return z
    if name == "relu":
        return np.where(z > 0, z, 0.0 * z)
    if name == "gelu":
        return z * ndtr(z)
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(GELU_C * (z + 0.044715 * z ** 3)))
    return z / (1.0 + np.exp(-z))


def slope(z, name):
    if name == "none":
        return np.ones_like(z)
    if name == "relu":
        return np.where(z > 0, 1.0, 0.0)
    if name == "gelu":
        return ndtr(z) + z * np.exp(-0.5 * z * z) / np.sqrt(2.0 * np.pi)
    if name == "gelu_tanh":
        t = np.tanh(GELU_C * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * GELU_C * (1.0 + 3 * 0.044715 * z * z)
    s = 1.0 / (1.0 + np.exp(-z))
    return s + z * s * (1.0 - s)


def act_error(z, name):
    """FP32 evaluation of act or act' at an FP32 z. none and relu are exact; the others combine a
    polynomial or rational form (2e-7 of 1 + |z| by their fits and a few roundings of 6e-8), and two
    special-function results of 2 ulp: below 1e-6 (1 + |z|)."""
    return 0.0 * z if name in ("none", "relu") else 1e-6 * (1.0 + np.abs(z))


def product(a, b, k, chunk=None):
    """(op(A) op(B), bound of the FP32 accumulation's error). The tensor core adds K = 16 products at a
    time and truncates: at most one ulp of the running sum, itself at most sum |a b|, per step; the
    chunks of K (FP32 outputs) are then added with one more rounding each."""
    ref = a @ b
    mag = np.abs(a) @ np.abs(b)
    steps = -(-k // 16) if chunk is None else -(-min(k, chunk) // 16) + -(-k // chunk)
    return ref, (steps + 16) * U32 * mag   # 16: rounding inside a step's own sum


def rounding(x, bf16):
    """Half an ulp of the stored type, at x's size or at the smallest normal's."""
    return np.maximum(np.abs(x), 2.0 ** -126) * (2.0 ** -8 if bf16 else 2.0 ** -24)


# ------------------------------------------------------------------ MXFP8
def e4m3_values():
    code = np.arange(256)
    e, f = (code >> 3) & 15, code & 7
    v = np.where(e == 0, f * 2.0 ** -9, (1 + f / 8.0) * 2.0 ** (e - 7.0))
    v = np.where(code >> 7 == 1, -v, v)
    return np.where(code & 127 == 127, np.nan, v)


def scale_offsets(rows, cols):
    r = np.arange(rows)[:, None]
    g = np.arange(-(-cols // 32))[None, :]
    return ((r // 128) * -(-cols // 128) + g // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + g % 4


def tile_scales(s, rows, cols, fill=0):
    """Row-major scale codes [rows, ceil(cols / 32)] in the library's layout."""
    out = np.full(-(-rows // 128) * -(-cols // 128) * 512, fill, np.uint8)
    out[scale_offsets(rows, cols)] = s
    return out


def decode(q, s_tiled, rows, cols):
    s = s_tiled[scale_offsets(rows, cols)].astype(np.float64)
    scale = np.where(s == 255, np.nan, 2.0 ** (s - 127.0))
    return e4m3_values()[q[:rows, :cols]] * np.repeat(scale, 32, axis=1)[:, :cols]


def quantize(z):
    """(codes, row-major scale codes) of z by the MX rule, groups of 32 along the rows."""
    rows, cols = z.shape
    groups = -(-cols // 32)
    pad = np.zeros((rows, groups * 32))
    pad[:, :cols] = z
    pad = pad.reshape(rows, groups, 32)
    bad = ~np.isfinite(pad).all(axis=2)
    clean = np.where(np.isfinite(pad), pad, 0.0)
    amax = np.abs(clean).max(axis=2)
    _, ex = np.frexp(amax)                       # amax = f 2^ex, f in [1/2, 1)
    e = np.where(amax > 0, np.clip(ex - 1 - 8, -127, 127), -127)
    x = clean / 2.0 ** e[:, :, None]
    positive = e4m3_values()[:127]               # codes 0 .. 126 are 0 .. 448
    mid = (positive[1:] + positive[:-1]) / 2
    a = np.minimum(np.abs(x), 448.0)
    code = np.searchsorted(mid, a, side="left")  # below the midpoint of code and code + 1
    tie = (code < 126) & (a == mid[np.minimum(code, 125)])
    code = np.where(tie & (code % 2 == 1), code + 1, code)
    code = code + np.where(np.signbit(x), 128, 0)
    code = np.where(bad[:, :, None], 127, code).reshape(rows, -1)[:, :cols].astype(np.uint8)
    return code, np.where(bad, 255, e + 127).astype(np.uint8)


# ------------------------------------------------------------------ layer norm
def layernorm(x, gamma, beta, eps):
    mean = x.mean(axis=1, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - mean) ** 2).mean(axis=1, keepdims=True) + eps)
    return (x - mean) * rstd * gamma + beta, mean[:, 0], rstd[:, 0]


def layernorm_backward(dy, x, gamma, mean, rstd):
    xh = (x - mean[:, None]) * rstd[:, None]
    u = dy * gamma
    dx = rstd[:, None] * (u - u.mean(axis=1, keepdims=True) - xh * (u * xh).mean(axis=1, keepdims=True))
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)
