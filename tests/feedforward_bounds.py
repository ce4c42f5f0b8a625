"""The gated feed-forward formulas in 64 bits on the GPU, for whole outputs of
large sizes and over the activation's range, each with what a call's result
may be off by. Nothing here shares code with the library.

A sigmoid is computed as 1 / (1 + exp2(x)): x takes four roundings, each a half
step of |t| / ln 2, and the instruction two half steps of the result, so that
e^-t is off by (4 |t| + 2) half steps of itself, the sigmoid s by 1 - s of that,
and by four more in the sum and the reciprocal. Where e^-t is below half a step
of 1, s is 1 (the reciprocal of 1), and where exp2 passes the type's range it
is 0: exactly, so that 1 - s and act are.
"""
import numpy as np
import torch

import experts_ref as ref

U = 2.0 ** -24                # half a step of binary32, relative
TINY, ZERO = 2.0 ** -120, 2.0 ** -125       # results, and sigmoids, below the normal numbers may be zero
SILU, GELU = 0, 1
C = 2 * (2 / np.pi) ** 0.5


def activation(act, g):
    """act(g), its derivative, and what each may be off by for an exact g."""
    if act == SILU:
        t, dt = g, torch.ones_like(g)
    else:
        t, dt = C * (g + 0.044715 * g ** 3), C * (1 + 3 * 0.044715 * g ** 2)
    e = torch.exp(-t.abs())
    big, small = 1 / (1 + e), e / (1 + e)
    s, r = torch.where(t >= 0, big, small), torch.where(t >= 0, small, big)
    one, none = t > 20, t < -200
    es = torch.where(one, r, (r * (4 * t.abs().clamp(max=200) + 2) + 4) * U)
    er = torch.where(one, r, s * es + U)
    a = g * s
    ea = a.abs() * (es + U) + g.abs() * ZERO
    slope = s + g * s * r * dt
    eslope = s * es + (g * dt).abs() * (s * es * r + s * er) * 1.01 + (g * s * r * dt).abs() * 8 * U
    eslope = eslope + 2 * U * (slope.abs() + s) + (1 + (g * dt).abs()) * ZERO
    zero = torch.zeros_like(g)
    return (torch.where(none, zero, a), torch.where(none, zero, slope), torch.where(none, zero, ea),
            torch.where(none, zero, eslope))


def half(y, tol):
    """tol and the result's rounding to bf16."""
    return tol + (y.abs() + tol) * ref.HALF_STEP["bf16"] * 1.01 + TINY


def gated(act, g, eg, u, eu):
    """h, its tolerance, of projections g and u off by eg and eu."""
    a, _, ea, _ = activation(act, g)
    ea = 1.13 * eg + ea * 1.05           # |act'| is at most 1.13
    h = a * u
    return h, half(h, ea * u.abs() + (a.abs() + ea) * eu + h.abs() * U)


def gated_grad(act, dh, edh, g, u):
    """dg, du and h with their tolerances, of dh off by edh and exact g and u."""
    a, slope, ea, eslope = activation(act, g)
    dg, du, h = dh * u * slope, dh * a, a * u
    tol_g = u.abs() * (edh * (slope.abs() + eslope) + dh.abs() * eslope) + 2 * U * dg.abs()
    tol_u = edh * (a.abs() + ea) + dh.abs() * ea + U * du.abs()
    return (dg, half(dg, tol_g)), (du, half(du, tol_u)), (h, half(h, ea * u.abs() + U * h.abs()))


def sum_error(y, mag, K, fast):
    """Of a block-128 product before its rounding (experts_ref.mm_tolerance), with the blocks' chains of instructions."""
    tol = mag * ((128 + 4 * -(-K // 128) + 16 + 6) * 2.0 ** -23 + (8 * 2.0 ** -13 if fast else 0.0))
    return tol + y.abs() * 2 * U


DECODED = np.nan_to_num(ref.DECODE)


def spread(s, rows, cols):
    s = s.double()
    if s.shape[0] != rows:
        s = s.repeat_interleave(128, 0)[:rows]
    return s.repeat_interleave(128, 1)[:, :cols]


def products(a, sa, b, sb, ends, matrices, first_matrix, ints):
    """Of every group's rows with its matrix first_matrix of `matrices`: y (M, N) and the sum of magnitudes."""
    M, N, K = a.shape[0], b.shape[1], a.shape[1]
    table = torch.from_numpy(DECODED).cuda()
    y = torch.zeros((M, N), dtype=torch.float64, device="cuda")
    mag, first = torch.zeros_like(y), 0
    for e, end in enumerate(ends):
        if end > first:
            w = e * matrices + first_matrix
            if ints:
                y[first:end] = (a[first:end].double() @ b[w].double().t()) / sa[first:end, None].double() / sb[w].double()
            else:
                av = table[a[first:end].long()] / spread(sa[first:end], end - first, K)
                bv = table[b[w].long()] / spread(sb[w], N, K)
                y[first:end] = av @ bv.t()
                mag[first:end] = av.abs() @ bv.abs().t()
        first = max(first, end)
    return y, mag


def differ(got, want, tol):
    """How many results are off by more than tol (or not a number), and the first."""
    bad = ~((got.double() - want).abs() <= tol)
    n = int(bad.sum())
    return (n, torch.nonzero(bad)[0].tolist() if n else None)
