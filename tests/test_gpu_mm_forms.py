"""Values of the products in the forms that large and mid sizes take
(tests/mm_form_cases.py), whole outputs against 64-bit sums, with workgroups
that walk several tiles, ragged and empty groups, rows that belong to none,
and contractions of one to a hundred steps.

Two kinds of operands. Codes of every exponent, within a bound counted from
the roundings. Small whole multiples of 1/2 with scales 1/2, 1 and 2, whose
products and sums are exact in either form (a product that is not 0 is at least
2^-4 of the largest of its eight; sums are multiples of 2^-4 below 2^18), so
that the result is the exact sum rounded once: equal, bit for bit."""
import numpy as np
import pytest
import torch

import experts_ref as ref
import group_scaling_fp8_amd as mgs
from gpu_util import Guarded, to_dev
from mm_form_cases import BLOCK128, WGRAD
from test_gpu_mm import OUT, codes, ends_of, scales

pytestmark = pytest.mark.gpu

HALVES = np.array([0x00, 0x30, 0x38, 0x3C, 0x40, 0x80, 0xB0, 0xB8, 0xBC, 0xC0], np.uint8)   # 0, +-0.5, 1, 1.5, 2


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mgs.lib()


def operand(rng, kind, shape):
    return codes(rng, shape) if kind == "codes" else rng.choice(HALVES, shape)


def factors(rng, kind, shape):
    return scales(rng, shape) if kind == "codes" else np.exp2(rng.integers(-1, 2, shape)).astype(np.float32)


def decoded(q):
    return to_dev(np.nan_to_num(ref.DECODE))[q.long()]


def spread(s, rows, cols):
    """Scales of blocks of 128 (or of single rows) as one for each value."""
    s = s.double()
    if s.shape[0] != rows:
        s = s.repeat_interleave(128, 0)[:rows]
    return s.repeat_interleave(128, 1)[:, :cols]


def tolerance(want, mag, length, out, fast):
    """A binary32 sum is off by at most one step of 2^-23 of the magnitudes for
    each addition between a term and the result: up to 128 in an instruction,
    four instructions a block of 128, 16 where parts are joined; and 6 roundings
    in scales, reciprocals and products. The fast form drops of each of eight
    products what lies below 2^-13 of the largest."""
    steps = 128 + 4 * -(-length // 128) + 16 + 6
    tol = mag * (steps * 2.0 ** -23 + (8 * 2.0 ** -13 if fast else 0.0))
    return tol.add_(want.abs(), alpha=ref.HALF_STEP[out] * 1.01)


def compare(got, want, mag, length, out, fast, kind, what):
    if kind == "codes":
        bad = ~((got.double() - want).abs() <= tolerance(want, mag, length, out, fast))
    else:
        bad = got != want.to(got.dtype)
    assert not bool(bad.any()), (what, int(bad.sum()), torch.nonzero(bad)[0].tolist())


@pytest.mark.parametrize("case", BLOCK128, ids=lambda c: "-".join(str(v) for v in c[:5]))
@pytest.mark.parametrize("kind", ["codes", "halves"])
@pytest.mark.parametrize("fast", [True, False])
def test_block128(case, kind, fast):
    M, N, K, G, which = case[:5]
    rng = np.random.default_rng(M + N + K)
    off = ends_of(which, M, G, rng)
    ends = ref.clean_ends(off if off is not None else [M], M)
    a, b = operand(rng, kind, (M, K)), operand(rng, kind, (G, N, K))
    sa, sb = factors(rng, kind, (M, -(-K // 128))), factors(rng, kind, (G, -(-N // 128), -(-K // 128)))
    a[ends[-1]:] = 0x7F          # what no group holds is not a number
    sa[ends[-1]:] = np.nan
    a, b, sa, sb = to_dev(a), to_dev(b), to_dev(sa), to_dev(sb)
    want = torch.zeros((M, N), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(want)
    first = 0
    for e, end in enumerate(ends):
        if end > first:
            av = decoded(a[first:end]) / spread(sa[first:end], end - first, K)
            bv = decoded(b[e]) / spread(sb[e], N, K)
            want[first:end] = av @ bv.t()
            if kind == "codes":
                mag[first:end] = av.abs() @ bv.abs().t()
        first = max(first, end)
    for out in OUT:
        y = Guarded((M, N), OUT[out])
        mgs.mgs_mm_block128(a, sa, b, sb, None if off is None else to_dev(off), OUT[out], fast, y=y.view)
        torch.cuda.synchronize()
        y.check()
        compare(y.view, want, mag, K, out, fast, kind, (case, out))


@pytest.mark.parametrize("case", WGRAD, ids=lambda c: "-".join(str(v) for v in c[:5]))
@pytest.mark.parametrize("kind", ["codes", "halves"])
@pytest.mark.parametrize("fast", [True, False])
def test_wgrad(case, kind, fast):
    M, N, K, G, which = case[:5]
    rng = np.random.default_rng(M + N + K)
    off = ends_of(which, M, G, rng)
    if which != "bad":
        off = off // 16 * 16
    ends = ref.clean_ends(off, M, 16)
    a, b = operand(rng, kind, (N, M)), operand(rng, kind, (K, M))
    sa, sb = factors(rng, kind, (N, G)), factors(rng, kind, (K, G))
    a[:, ends[-1]:], b[:, ends[-1]:] = 0x7F, 0xFF
    first = 0
    for g, end in enumerate(ends):       # the scales of an empty group are not read as values
        if end <= first:
            sa[:, g], sb[:, g] = np.nan, 0.0
        first = max(first, end)
    a, b, sa, sb, off = to_dev(a), to_dev(b), to_dev(sa), to_dev(sb), to_dev(off)
    want = torch.zeros((G, N, K), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(want)
    first = 0
    for g, end in enumerate(ends):
        if end > first:
            av = decoded(a[:, first:end]) / sa[:, g:g + 1].double()
            bv = decoded(b[:, first:end]) / sb[:, g:g + 1].double()
            want[g] = av @ bv.t()
            if kind == "codes":
                mag[g] = av.abs() @ bv.abs().t()
        first = max(first, end)
    for out in ("bf16", "f32", "accumulate"):
        f32 = out != "bf16"
        dw = Guarded((G, N, K), torch.float32 if f32 else torch.bfloat16)
        before = None
        if out == "accumulate":
            before = (torch.arange(N * K, device="cuda") % 7 - 3).float().view(N, K).expand(G, N, K).contiguous()
            dw.view.copy_(before)
        mgs.mgs_mm_wgrad(a, sa, b, sb, off, OUT["f32" if f32 else "bf16"], fast, dw=dw.view,
                         accumulate=out == "accumulate")
        torch.cuda.synchronize()
        dw.check()
        total = want if before is None else want + before
        # one more addition where the result is added to what was there
        more = mag if before is None else mag + total.abs() * 2.0 ** -8
        compare(dw.view, total, more, M, "f32" if f32 else "bf16", fast, kind, (case, out))


@pytest.mark.parametrize("fast", [True, False])
def test_repeats_are_identical_in_the_large_forms(fast):
    M, N, K, G = 8200, 4000, 656, 6
    rng = np.random.default_rng(5)
    off = to_dev(ends_of("tail", M, G, rng) // 16 * 16)
    a, b = to_dev(codes(rng, (M, K))), to_dev(codes(rng, (G, N, K)))
    sa, sb = to_dev(scales(rng, (M, 6))), to_dev(scales(rng, (G, 32, 6)))
    ys = [mgs.mgs_mm_block128(a, sa, b, sb, off, torch.float32, fast) for _ in range(4)]
    assert all(torch.equal(ys[0], y) for y in ys)
    M, N, K = 1040, 2064, 2064
    off = to_dev(ends_of("even", M, 16, rng) // 16 * 16)
    a, b = to_dev(codes(rng, (N, M))), to_dev(codes(rng, (K, M)))
    sa, sb = to_dev(scales(rng, (N, 16))), to_dev(scales(rng, (K, 16)))
    ds = [mgs.mgs_mm_wgrad(a, sa, b, sb, off, fast_accum=fast) for _ in range(4)]
    assert all(torch.equal(ds[0], d) for d in ds)
