"""Plain 64-bit forms of the mixture-of-experts operators, for the tests.

Nothing here shares code with the library. The casts' bytes and scales come
from the CPU oracle's cast, whose own pins are in tests/test_oracle_*.py.
"""
import numpy as np

import oracle
from group_scaling_fp8_amd import workloads as wl

DECODE = oracle.e4m3_decode_table().astype(np.float64)

# A rounding to the nearest is off by at most half a step of the value.
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def bf16_to_f64(bits):
    return wl.bf16_bits_to_f32(bits).astype(np.float64)


def order(ids, E, align):
    """Offsets, rows and slots of the sorted tokens, slot by slot."""
    T, k = ids.shape
    n = T * k
    P = (n + min(E, n) * (align - 1)) // align * align
    members = [[] for _ in range(E)]
    for i, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < E:
            members[e].append(i)
    rows, slots, offsets = np.full(n, -1, np.int32), [], []
    for mine in members:
        for i in mine:
            rows[i] = len(slots)
            slots.append(i)
        slots += [-1] * (-len(mine) % align)
        offsets.append(len(slots))
    slots += [-1] * (P - len(slots))
    return np.array(offsets, np.int32), rows.reshape(T, k), np.array(slots, np.int32)


def permuted(x_bits, slots, k):
    xp = np.zeros((len(slots), x_bits.shape[1]), np.uint16)
    held = slots >= 0
    xp[held] = x_bits[slots[held] // k]
    return xp


def block_ends(K):
    return np.array([min(b + 128, K) for b in range(0, K, 128)], np.int32)


def rows128(x_bits, pow2=False):
    """One scale for each row and 128 columns: the rowwise cast with those
    groups. Columns are filled up with zeros to a multiple of 16, which no
    amax and no byte of the others depends on."""
    M, K = x_bits.shape
    wide = np.zeros((M, -(-K // 16) * 16), np.uint16)
    wide[:, :K] = x_bits
    q, s = oracle.quant_groups_dim1(wide, block_ends(wide.shape[1]), pow2)
    return np.ascontiguousarray(q[:, :K]), s


def blocks128(w_bits, pow2=False):
    """One scale for each 128 x 128: every block laid out as one row."""
    E, N, K = w_bits.shape
    nb, kb = -(-N // 128), -(-K // 128)
    full = np.zeros((E, nb * 128, kb * 128), np.uint16)
    full[:, :N, :K] = w_bits
    flat = full.reshape(E, nb, 128, kb, 128).transpose(0, 1, 3, 2, 4).reshape(E * nb * kb, 128 * 128)
    q, s = oracle.quant_groups_dim1(np.ascontiguousarray(flat), np.array([128 * 128], np.int32), pow2)
    q = q.reshape(E, nb, kb, 128, 128).transpose(0, 1, 3, 2, 4).reshape(E, nb * 128, kb * 128)
    return np.ascontiguousarray(q[:, :N, :K]), s.reshape(E, nb, kb)


def clean_ends(offsets, M, align=1):
    """Group ends as the calls read them."""
    return np.maximum.accumulate(np.clip(np.asarray(offsets, np.int64), 0, M) // align * align)


def mm_block128(a, sa, b, sb, ends):
    """y (M, N) and the sum of its terms' magnitudes, in 64 bits."""
    M, K = a.shape
    N = b.shape[1]
    av = DECODE[a] / np.repeat(sa.astype(np.float64), 128, 1)[:, :K]
    y, mag = np.zeros((M, N)), np.zeros((M, N))
    first = 0
    for e, end in enumerate(ends):
        if end > first:
            s = np.repeat(np.repeat(sb[e].astype(np.float64), 128, 0)[:N], 128, 1)[:, :K]
            bv = DECODE[b[e]] / s
            y[first:end] = av[first:end] @ bv.T
            mag[first:end] = np.abs(av[first:end]) @ np.abs(bv).T
        first = max(first, end)
    return y, mag


def mm_wgrad(a_t, sa, b_t, sb, ends):
    N, K = a_t.shape[0], b_t.shape[0]
    dw, mag = np.zeros((len(ends), N, K)), np.zeros((len(ends), N, K))
    first = 0
    for g, end in enumerate(ends):
        if end > first:
            av = DECODE[a_t[:, first:end]] / sa[:, g:g + 1].astype(np.float64)
            bv = DECODE[b_t[:, first:end]] / sb[:, g:g + 1].astype(np.float64)
            dw[g] = av @ bv.T
            mag[g] = np.abs(av) @ np.abs(bv).T
        first = max(first, end)
    return dw, mag


def mm_tolerance(y, mag, length, out, fast=False):
    """What a product may be off by. A sum of n terms in binary32, in any
    order, is within n steps of 2^-23 (an addition in the matrix core may cut
    off instead of rounding) of the sum of magnitudes: at most 128 + (blocks)
    additions lie between a term and the result when a contraction is summed
    block by block or in a chain of instructions over 128, at most 16 more when
    parts of it are joined, and 6 roundings are in the scales and their
    reciprocals and products. Then one rounding to the output type. The fast
    form drops, of each of up to eight products, what lies below 2^-13 of the
    largest of them: eight times that of the magnitudes' sum at most."""
    blocks = -(-length // 128)
    tol = mag * (128 + blocks + 16 + 6) * 2.0 ** -23 + np.abs(y) * HALF_STEP[out] * 1.01
    return tol + mag * 8 * 2.0 ** -13 if fast else tol


def combine(yp, rows, weights):
    """y (T, D) and the sum of magnitudes."""
    T, k = rows.shape
    y, mag = np.zeros((T, yp.shape[1])), np.zeros((T, yp.shape[1]))
    for t in range(T):
        for s in range(k):
            if 0 <= rows[t, s] < yp.shape[0]:
                v = yp[rows[t, s]] * float(weights[t, s])
                y[t] += v
                mag[t] += np.abs(v)
    return y, mag


def combine_grad(dy, yp, rows, weights):
    """dyp, dw and the magnitudes of dw's sums."""
    T, k = rows.shape
    dyp, dw, mag = np.zeros(yp.shape), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for s in range(k):
            p = rows[t, s]
            if 0 <= p < yp.shape[0]:
                dyp[p] = dy[t] * float(weights[t, s])
                dw[t, s] = dy[t] @ yp[p]
                mag[t, s] = np.abs(dy[t]) @ np.abs(yp[p])
    return dyp, dw, mag
