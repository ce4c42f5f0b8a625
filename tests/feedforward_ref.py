"""Plain 64-bit forms of the gated feed-forward operators and of the 8-bit
integer ones, for the tests, with what their results may be off by.

Nothing here shares code with the library.
"""
import numpy as np

import experts_ref as ref

U = 2.0 ** -24           # half a binary32 step, relative
TINY = 2.0 ** -120       # results below the normal numbers may become zero
ZERO = 2.0 ** -125       # and so may a sigmoid

SILU, GELU = 0, 1
C = 2 * np.sqrt(2 / np.pi)


def logistic(act, g):
    """t(g), its derivative, sigmoid(t) and 1 - sigmoid(t)."""
    if act == SILU:
        t, dt = g, np.ones_like(g)
    else:
        t, dt = C * (g + 0.044715 * g ** 3), C * (1 + 3 * 0.044715 * g ** 2)
    e = np.exp(-np.abs(t))
    big, small = 1 / (1 + e), e / (1 + e)
    return t, dt, np.where(t >= 0, big, small), np.where(t >= 0, small, big)


def act_of(act, g):
    return g * logistic(act, g)[2]


def slope_of(act, g):
    _, dt, s, r = logistic(act, g)
    return s + g * s * r * dt


def sigmoid_error(act, g):
    """The relative error of the library's sigmoid: exp2's argument takes four
    roundings (the coefficients', g^2's, an fma's and a product's), each a half step of
    |t| / ln 2, so the exponential is off by 4 |t| half steps, and 2 for the
    instruction; the sum 1 and the reciprocal 2 more."""
    return (4 * np.minimum(np.abs(logistic(act, g)[0]), 90) + 6) * U


def product(a, sa, b, sb, ends, kind):
    """y (M, N) and what its binary32 sums may be off by, before a rounding to the output's type."""
    if kind == "i8":
        y, mag = mm_i8(a, sa, b, sb, ends)
        # the sum's own rounding, two reciprocals and two products
        return y, np.abs(y) * 6 * U
    y, mag = ref.mm_block128(a, sa, b, sb, ends)
    tol = ref.mm_tolerance(np.zeros_like(y), mag, a.shape[1], "f32", kind == "fast")
    return y, tol + np.abs(y) * 2 * U


def mm_i8(a, sa, b, sb, ends):
    """y (M, N) of int8 rows, the sum being exact, and it again as whole numbers."""
    y = np.zeros((a.shape[0], b.shape[1]))
    whole = np.zeros(y.shape)
    first = 0
    for e, end in enumerate(ends):
        if end > first:
            whole[first:end] = a[first:end].astype(np.float64) @ b[e].astype(np.float64).T     # exact below 2^53
            y[first:end] = whole[first:end] / (sa[first:end, None].astype(np.float64) * sb[e].astype(np.float64))
        first = max(first, end)
    return y, whole


def quant_rows_i8(bits):
    """q int8 and scales of bf16 rows, each step in binary32 as defined."""
    x = ref.bf16_to_f64(bits).astype(np.float32)
    amax = np.abs(x).max(-1)
    s = np.float32(127) / np.maximum(amax, np.float32(1e-12))
    assert s.dtype == np.float32
    return np.rint(x * s[..., None]).astype(np.int8), s


def half(y, tol, out="bf16"):
    """tol with the result's one rounding to the output's type."""
    return tol + (np.abs(y) + tol) * ref.HALF_STEP[out] * 1.01 + TINY


def gated(a, sa, b, sb, ends, act, kind):
    """h and gu (both with their tolerances) of b (2 E, N, K)."""
    g, dg = product(a, sa, b[0::2], sb[0::2], ends, kind)
    u, du = product(a, sa, b[1::2], sb[1::2], ends, kind)
    _, dt, s, _ = logistic(act, g)
    p = np.abs(act_of(act, g))
    # |act'| is at most 1.1 (silu) or 1.13 (gelu); the sigmoid's error and three products
    dp = 1.13 * dg + p * (sigmoid_error(act, np.abs(g) + dg) + 2 * U)
    tol = dp * np.abs(u) + (p + dp) * du + np.abs(p * u) * U + np.abs(g * u) * ZERO
    h = act_of(act, g) * u
    gu = np.concatenate([g, u], 1)
    return (h, half(h, tol)), (gu, half(gu, np.concatenate([dg, du], 1)))


def gated_grad(dy, sa, b, sb, gu, ends, act, kind):
    """dgu and h (both with their tolerances); gu (M, 2 N) values of the kept
    bf16. Rows of no group are zeros."""
    N = b.shape[1]
    dh, tol = product(dy, sa, b, sb, ends, kind)
    gu = np.where(np.arange(len(gu))[:, None] < max([0, *ends]), gu, 0.0)
    g, u = gu[:, :N], gu[:, N:]
    _, dt, s, r = logistic(act, g)
    es = sigmoid_error(act, g)
    p = g * s
    ep = np.abs(p) * (es + U)
    du, dg = dh * p, dh * u * slope_of(act, g)
    # the slope s + p (1 - s) t': errors of s in both terms (1 - s also its own rounding), t' 3
    # half steps of its sum of magnitudes, which for both activations is t' itself, and 3 products and sums
    es_slope = es * s + np.abs(g * s * dt) * (es + s * es + 8 * U) + 2 * U * s
    tol_du = tol * (np.abs(p) + ep) + np.abs(dh) * ep + np.abs(du) * U + np.abs(dh * g) * ZERO
    slope = np.abs(slope_of(act, g))
    tol_dg = np.abs(u) * (tol * (slope + es_slope) + np.abs(dh) * es_slope) + np.abs(dg) * 2 * U
    tol_dg = tol_dg + np.abs(dh * u) * (1 + np.abs(g * dt)) * ZERO
    dgu = np.concatenate([dg, du], 1)
    h = p * u
    return (dgu, half(dgu, np.concatenate([tol_dg, tol_du], 1))), (h, half(h, ep * np.abs(u) + np.abs(h) * U + np.abs(g * u) * ZERO))
