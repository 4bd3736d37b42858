"""64-bit forms of a gated MLP's products and of the Newton-Schulz update, and their error bounds.

NumPy in double throughout, written from the definitions; nothing here calls the library.
"""

from __future__ import annotations

import numpy as np

import mlp_ref as ref

STEP = (3.4445, -4.7750, 2.0315)
HALF16 = 2.0 ** -11   # half a step of fp16, relative
SUB16 = 2.0 ** -25    # half a step of fp16's subnormal values
SCALE = 256.0         # X is held times this


def glu(a, bg, bu, k, alpha, act):
    """(H, G, U) and the bounds of their errors before rounding. g and u carry the FP32 accumulation's error and
    alpha's rounding; |act'| <= 1.13 takes g's on, and the product takes both."""
    (pg, eg), (pu, eu) = ref.product(a, bg, k), ref.product(a, bu, k)
    g, u = alpha * pg, alpha * pu
    eg, eu = np.abs(alpha) * eg + ref.U32 * np.abs(g), np.abs(alpha) * eu + ref.U32 * np.abs(u)
    h = ref.act(g, act)
    eh = 1.2 * eg + ref.act_error(g, act)
    return (h * u, g, u), (eh * np.abs(u) + np.abs(h) * eu + eh * eu + ref.U32 * np.abs(h * u), eg, eu)


def dglu(a, b, k, alpha, g, u, act):
    """(dG, dU, H) and the bounds of their errors before rounding, for exact g and u."""
    p, e = ref.product(a, b, k)
    dh = alpha * p
    e = np.abs(alpha) * e + ref.U32 * np.abs(dh)
    h, s, ea = ref.act(g, act), ref.slope(g, act), ref.act_error(g, act)
    dg, du = dh * u * s, dh * h
    return ((dg, du, h * u),
            (np.abs(u) * (np.abs(s) * e + (np.abs(dh) + e) * ea) + 2 * ref.U32 * np.abs(dg),
             np.abs(h) * e + (np.abs(dh) + e) * ea + ref.U32 * np.abs(du),
             np.abs(u) * ea + ref.U32 * np.abs(h * u)))


def newton_schulz(x, coeffs, eps=1e-7):
    """X after one polynomial (a, b, c) for each of `coeffs`."""
    x = x / (np.linalg.norm(x) + eps)
    wide = x.shape[0] <= x.shape[1]
    for a, b, c in coeffs:
        gram = x @ x.T if wide else x.T @ x
        poly = b * gram + c * (gram @ gram)
        x = a * x + (poly @ x if wide else x @ poly)
    return x


def one_step_bound(x, coeffs, eps=1e-7):
    """Bound, element by element, of one step's error before rounding to bf16: the operands are rounded to fp16
    (the high half of X; A and B off their diagonals), what multiplies a and the diagonals is not, and each sum of
    K products in FP32 is off by at most (K / 16 + 16) units of its absolute sum."""
    (a, b, c), = coeffs
    x = x / (np.linalg.norm(x) + eps)
    if x.shape[0] > x.shape[1]:
        return one_step_bound(x.T, coeffs, 0.0).T
    s, n = x.shape

    def units(k):
        return (k / 16 + 16) * ref.U32

    ax = np.abs(x)
    ex = HALF16 * ax + SUB16 / SCALE          # of the high half
    gram, mag = x @ x.T, ax @ ax.T
    off = 1.0 - np.eye(s)
    eg = 2 * (ex @ ax.T + ax @ ex.T) + units(n) * mag                      # of A before it is rounded
    eo = eg + off * (HALF16 * (np.abs(gram) + eg) + SUB16)                 # and of what is kept
    ag = np.abs(gram)
    poly = b * gram + c * (gram @ gram)
    e2 = eo @ ag + ag @ eo + eo @ eo + units(s) * (ag @ ag)
    ep = np.abs(b) * eo + np.abs(c) * e2 + 8 * ref.U32 * (np.abs(b) * ag + np.abs(c) * ag @ ag)
    eb = ep + off * (HALF16 * (np.abs(poly) + ep) + SUB16)
    ap = np.abs(poly)
    # the diagonal multiplies 22 bits of X, the rest its high half
    diag = np.abs(np.diag(poly))[:, None]
    exact = (2.0 ** -21 * ax + SUB16 / SCALE) * (np.abs(a) + diag)
    return (exact + eb @ (ax + ex) + (ap * off) @ ex + units(s) * (ap @ ax)
            + 4 * ref.U32 * (np.abs(a) + diag) * ax + 2.0 ** -22 * (np.abs(a) * ax + ap @ ax))  # (X0's own scaling)


def rounded_steps(x, coeffs, eps=1e-7):
    """newton_schulz with the library's rounding points, everything else in 64 bits: what their error is made of."""
    def fp16(v):
        return v.astype(np.float16).astype(np.float64)

    wide = x.shape[0] <= x.shape[1]
    x = x if wide else x.T
    x = SCALE * x / (np.linalg.norm(x) + eps)
    hi = fp16(x)
    lo = fp16(x - hi)
    for a, b, c in coeffs:
        gram = hi @ hi.T / SCALE ** 2
        d = np.diag(gram).copy()
        o = fp16(gram - np.diag(d))
        poly = b * (o + np.diag(d)) + c * (o @ o + (d[:, None] + d[None, :]) * o + np.diag(d * d))
        e = np.diag(poly).copy()
        x = (a + e)[:, None] * (hi + lo) + fp16(poly - np.diag(e)) @ hi
        hi = fp16(x)
        lo = fp16(x - hi)
    x = x / SCALE
    return x if wide else x.T
