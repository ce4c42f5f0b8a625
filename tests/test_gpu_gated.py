"""The gated feed-forward calls against forms in 64 bits, with tolerances from
the number of roundings (feedforward_ref)."""
import numpy as np
import pytest
import torch

import experts_ref as ref
import feedforward_ref as ff
import group_scaling_fp8_amd as mgs
from feedforward_cases import GATED, ROWS
from group_scaling_fp8_amd import feedforward, workloads as wl
from gpu_util import Guarded, to_dev
from test_gpu_mm import check, codes, ends_of

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mgs.lib()


def scales(rng, shape, K):
    """Scales over a few binades that bring sums of K products of random codes,
    which are about 2^7 in their mean square, to between 1 and 100."""
    return np.exp2(rng.uniform(-2, 2, size=shape) + 5.5 + 0.25 * np.log2(K)).astype(np.float32)


def operands(rng, M, K, W, N, ends):
    kb = -(-K // 128)
    a, b = codes(rng, (M, K)), codes(rng, (W, N, K))
    sa, sb = scales(rng, (M, kb), K), scales(rng, (W, -(-N // 128), kb), K)
    last = max([0, *ends])
    clean = [v.copy() for v in (a, sa)]
    a[last:] = 0x7F              # what no group holds is not a number
    sa[last:] = np.nan
    clean[0][last:], clean[1][last:] = 0, 1
    return (a, sa, b, sb), (*clean, b, sb)


def groups(rng, kind, M, G):
    off = ends_of(kind, M, G, rng)
    return off, ref.clean_ends(off if off is not None else [M], M)


@pytest.mark.parametrize("case", GATED, ids=str)
@pytest.mark.parametrize("act,fast,keep", [(ff.SILU, True, True), (ff.GELU, False, False)])
def test_gated(case, act, fast, keep):
    M, F, K, G, kind, *_ = case
    rng = np.random.default_rng(M * 7 + F + K)
    off, ends = groups(rng, kind, M, G)
    held, clean = operands(rng, M, K, 2 * G, F, ends)
    h, gu = Guarded((M, F), BF16), Guarded((M, 2 * F), BF16) if keep else None
    feedforward.mgs_mm_gated_block128(*[to_dev(v) for v in held], None if off is None else to_dev(off), act, fast,
                                      h=h.view, gu=gu.view if keep else None)
    torch.cuda.synchronize()
    h.check()
    (want, tol), (want_gu, tol_gu) = ff.gated(*clean, ends, act, "fast" if fast else "exact")
    check(h.view.float().cpu().numpy(), want, tol, (case, "h"))
    if keep:
        gu.check()
        check(gu.view.float().cpu().numpy(), want_gu, tol_gu, (case, "gu"))


@pytest.mark.parametrize("case", ROWS, ids=str)
@pytest.mark.parametrize("act,fast,hidden", [(ff.GELU, True, True), (ff.SILU, False, False)])
def test_gated_grad(case, act, fast, hidden):
    M, F, D, G, kind, *_ = case
    rng = np.random.default_rng(M * 11 + F + D)
    off, ends = groups(rng, kind, M, G)
    held, clean = operands(rng, M, D, G, F, ends)
    gu = wl.f32_to_bf16_bits(rng.standard_normal((M, 2 * F)).astype(np.float32) * 2)
    values = ref.bf16_to_f64(gu)
    gu[max([0, *ends]):] = 0x7FC0            # rows of no group need not be numbers
    dgu, h = Guarded((M, 2 * F), BF16), Guarded((M, F), BF16) if hidden else None
    feedforward.mgs_mm_gated_grad_block128(*[to_dev(v) for v in held], to_dev(gu), None if off is None else to_dev(off),
                                           act, fast, dgu=dgu.view, h=h.view if hidden else None)
    torch.cuda.synchronize()
    dgu.check()
    (want, tol), (want_h, tol_h) = ff.gated_grad(*clean, values, ends, act, "fast" if fast else "exact")
    check(dgu.view.float().cpu().numpy(), want, tol, (case, "dgu"))
    if hidden:
        h.check()
        check(h.view.float().cpu().numpy(), want_h, tol_h, (case, "h"))


def one_code():
    return int(np.argmin(np.abs(np.nan_to_num(ref.DECODE, nan=9) - 1)))


@pytest.mark.parametrize("act", [ff.SILU, ff.GELU])
@pytest.mark.parametrize("M", [3, 40, 300])
def test_activation_over_its_range(act, M):
    """Projections of exactly known values: one code of 1 in a row, one in a
    weight's row, the scales make the rest. Every result is within the rounding
    of its binary32 steps, from the linear parts to where the sigmoid is 0 or 1."""
    F, K = 512, 128
    g = np.concatenate([np.linspace(-100, 100, 201), np.geomspace(1e-30, 1e30, 55), -np.geomspace(1e-30, 1e30, 55)])
    g = np.resize(g, M)
    a, b = np.zeros((M, K), np.uint8), np.zeros((2, F, K), np.uint8)
    a[:, 5] = b[:, :, 5] = one_code()
    a[g < 0, 5] |= 0x80
    b[1] = b[0]
    sa = np.where(g == 0, 1e30, 1 / np.abs(np.where(g == 0, 1, g))).astype(np.float32)[:, None]
    sb = np.ones((2, 4, 1), np.float32)
    sb[1] = 2.0 ** np.array([0, -4, 8, 30])[:, None]
    h, gu = feedforward.mgs_mm_gated_block128(*[to_dev(v) for v in (a, sa, b, sb)], None, act, keep=True)
    (want, tol), (want_gu, tol_gu) = ff.gated(a, sa, b, sb, [M], act, "exact")
    small = np.abs(want) < 3e38              # larger ones pass the type's range
    check(np.where(small, h.float().cpu().numpy(), 0), np.where(small, want, 0), tol, (act, M))
    check(gu.float().cpu().numpy(), want_gu, tol_gu, (act, M))


@pytest.mark.parametrize("act", [ff.SILU, ff.GELU])
def test_values_that_are_not_finite(act):
    """A projection that is not a number or infinite gives what the formula gives and reaches its own column only."""
    rng = np.random.default_rng(4)
    M, F, K = 24, 144, 128
    held, _ = operands(rng, M, K, 2, F, [M])
    clean = feedforward.mgs_mm_gated_block128(*[to_dev(v) for v in held], None, act).float().cpu().numpy()
    held[2][0, 17] = 0x7F
    held[2][1, 140] = 0xFF
    got = feedforward.mgs_mm_gated_block128(*[to_dev(v) for v in held], None, act).float().cpu().numpy()
    bad = np.zeros((M, F), bool)
    bad[:, [17, 140]] = True
    assert np.isnan(got[bad]).all() and np.array_equal(got[~bad], clean[~bad])
    dy, _ = operands(rng, M, K, 1, F, [M])
    gu = rng.standard_normal((M, 2 * F)).astype(np.float32)
    gu[1, 3], gu[2, 5], gu[3, F + 7] = np.nan, np.inf, np.inf
    dgu, h = (t.float().cpu().numpy() for t in feedforward.mgs_mm_gated_grad_block128(
        *[to_dev(v) for v in dy], to_dev(wl.f32_to_bf16_bits(gu)), None, act, hidden=True))
    assert np.isnan(h[1, 3]) and np.isnan(dgu[1, [3, F + 3]]).all()
    assert np.isinf(h[2, 5]) and np.isinf(h[3, 7])
    ok = np.ones((M, F), bool)
    ok[[1, 2, 3], [3, 5, 7]] = False
    assert np.isfinite(h[ok]).all() and np.isfinite(dgu[np.concatenate([ok, ok], 1)]).all()


def test_rows_do_not_depend_on_others():
    """A row that is not a number leaves the others alone, as does another expert's weight."""
    rng = np.random.default_rng(78)
    M, F, K, G = 150, 272, 272, 3
    off = to_dev(np.array([50, 90, 150], np.int32))
    held, _ = operands(rng, M, K, 2 * G, F, [M])
    clean = feedforward.mgs_mm_gated_block128(*[to_dev(v) for v in held], off).float().cpu().numpy()
    held[0][[0, 49, 60, 149]] = 0x7F
    held[2][2:4] = 0xFF
    got = feedforward.mgs_mm_gated_block128(*[to_dev(v) for v in held], off).float().cpu().numpy()
    keep = np.ones(M, bool)
    keep[[0, 49, 149]] = False
    keep[50:90] = False
    assert np.array_equal(got[keep], clean[keep]) and np.isnan(got[~keep]).all()


def test_empty_sizes():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    f32 = lambda *s: torch.ones(s, dtype=torch.float32, device="cuda")  # noqa: E731
    h, gu = feedforward.mgs_mm_gated_block128(u8(0, 64), f32(0, 1), u8(2, 32, 64), f32(2, 1, 1), keep=True)
    assert h.shape == (0, 32) and gu.shape == (0, 64)
    h, gu = feedforward.mgs_mm_gated_block128(u8(5, 0), f32(5, 0), u8(2, 32, 0), f32(2, 1, 0), keep=True)
    assert not h.any() and not gu.any()
    empty = torch.zeros((5, 64), dtype=BF16, device="cuda")
    with pytest.raises(mgs.MgsError):
        feedforward.mgs_mm_gated_grad_block128(u8(5, 0), f32(5, 0), u8(1, 32, 0), f32(1, 1, 0), empty)
    dgu = feedforward.mgs_mm_gated_grad_block128(u8(0, 64), f32(0, 1), u8(1, 32, 64), f32(1, 1, 1), empty[:0])
    assert dgu.shape == (0, 64)
