"""The activation and its derivative over their whole range, in the form for few
rows and in every form of tiles, and projections that are infinite or not
numbers."""
import numpy as np
import pytest
import torch

import feedforward_bounds as fb
import group_scaling_fp8_amd as mgs
from group_scaling_fp8_amd import feedforward
from test_gpu_gated import one_code

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
F = 512
# rows, the forms that a pair of twice F columns takes (tests/test_long_cases.py checks them): few rows, two sets of
# waves, tiles of 128 and of 256; the gradient's F columns take twice the rows
ROWS = [24, 1100, 5000, 8300]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mgs.lib()


def wide_range(n):
    """n values of both signs: the linear parts, the bends, and far out; powers of two near the clamp of the argument."""
    some = np.concatenate([np.linspace(-30, 30, 241), np.linspace(-120, 120, 97), np.geomspace(1e-30, 1e30, 61),
                           -np.geomspace(1e-30, 1e30, 61), [8191, 8192, 8193, -8191, -8192, -8193, 0, -0.0]])
    return np.resize(np.random.default_rng(3).permutation(some), n)


def units(M, W, K=128):
    """Rows and weights with one code of 1 each, at the same place: products are 1 over the scales."""
    a, b = torch.zeros((M, K), dtype=torch.uint8, device="cuda"), torch.zeros((W, F, K), dtype=torch.uint8, device="cuda")
    a[:, 5], b[:, :, 5] = one_code(), one_code()
    return a, b


@pytest.mark.parametrize("act", [fb.SILU, fb.GELU])
@pytest.mark.parametrize("fast", [True, False])
@pytest.mark.parametrize("M", ROWS)
def test_forward(act, fast, M):
    """g of each row, u = g times a power of two for each block of columns."""
    a, b = units(M, 2)
    g = wide_range(M)
    a[torch.from_numpy(g < 0).cuda(), 5] |= 0x80
    # what the scales make of it, rounded as the call rounds: 1 / sa times 1 / sb
    sa = torch.from_numpy(np.where(g == 0, 1e30, 1 / np.abs(np.where(g == 0, 1, g))).astype(np.float32)).cuda()[:, None]
    sb = torch.ones((2, 4, 1), device="cuda")
    sb[1] = torch.tensor([1, 2.0 ** -4, 2.0 ** 8, 2.0 ** 30], device="cuda")[:, None]
    h, gu = feedforward.mgs_mm_gated_block128(a, sa, b, sb, None, act, fast, keep=True)
    alone = feedforward.mgs_mm_gated_block128(a, sa, b, sb, None, act, fast)
    assert torch.equal(h.view(torch.int16), alone.view(torch.int16))
    sign = torch.from_numpy(np.where(g < 0, -1.0, 1.0)).cuda()[:, None]
    true_g = (sign / sa.double()).expand(M, F)
    true_u = true_g / sb[1, :, 0].double().repeat_interleave(128)
    want, tol = fb.gated(act, true_g, true_g.abs() * 2 * fb.U, true_u, true_u.abs() * 2 * fb.U)
    held = want.abs() < 3e38                  # larger ones pass the type's range
    assert fb.differ(torch.where(held, h.double(), 0.0), torch.where(held, want, 0.0), tol) == (0, None)
    both = torch.cat([true_g, true_u], 1)
    held = both.abs() < 3e38
    assert fb.differ(torch.where(held, gu.double(), 0.0), torch.where(held, both, 0.0), fb.half(both, both.abs() * 2 * fb.U)) \
        == (0, None)


@pytest.mark.parametrize("act", [fb.SILU, fb.GELU])
@pytest.mark.parametrize("fast", [True, False])
@pytest.mark.parametrize("M", [2 * m for m in ROWS])
def test_gradient(act, fast, M):
    """g over the range in every row and column, dh and u of a few magnitudes."""
    dy, b = units(M, 1)
    rng = np.random.default_rng(M)
    dh = 2.0 ** rng.integers(-6, 7, (M, 1))
    sa = torch.from_numpy((1 / dh).astype(np.float32)).cuda()
    sb = torch.from_numpy(2.0 ** np.array([0, 3, -2, 5])).float().cuda()[None, :, None]
    gu = torch.from_numpy(np.concatenate([wide_range(M * F).reshape(M, F),
                                          2.0 ** rng.integers(-8, 9, (M, F)) * rng.choice([-1, 1], (M, F))], 1)).to(BF16).cuda()
    g, u = gu[:, :F].double(), gu[:, F:].double()
    dgu, h = feedforward.mgs_mm_gated_grad_block128(dy, sa, b, sb, gu, None, act, fast, hidden=True)
    alone = feedforward.mgs_mm_gated_grad_block128(dy, sa, b, sb, gu, None, act, fast)
    assert torch.equal(dgu.view(torch.int16), alone.view(torch.int16))
    true = torch.from_numpy(dh).cuda() / sb[0, :, 0].double().repeat_interleave(128)          # powers of two: exact
    (dg, tg), (du, tu), (want, tol) = fb.gated_grad(act, true, torch.zeros_like(true), g, u)
    for got, v, t in ((dgu[:, :F], dg, tg), (dgu[:, F:], du, tu), (h, want, tol)):
        held = v.abs() < 3e38
        assert fb.differ(torch.where(held, got.double(), 0.0), torch.where(held, v, 0.0), t) == (0, None)
    # where the sigmoid is 1, the derivative is exactly 1 and act is g; where it is 0, both are
    t = g if act == fb.SILU else fb.C * (g + 0.044715 * g ** 3)
    for where, d, x in ((t > 60, true * u, true * g), (t < -200, 0 * u, 0 * u)):
        assert torch.equal(dgu[:, :F][where], d.to(BF16)[where]) and torch.equal(dgu[:, F:][where], x.to(BF16)[where])


NAN, INF = float("nan"), float("inf")
# g, u; du over dh > 0, dg over dh > 0, h, as the formulas give them in fp32: silu(-inf) is -inf * 0
SPECIAL = [
    (INF, 2.0, INF, NAN, INF), (INF, -2.0, INF, NAN, -INF), (-INF, 2.0, NAN, NAN, NAN), (NAN, 2.0, NAN, NAN, NAN),
    (30.0, INF, 30.0, INF, INF), (30.0, -INF, 30.0, -INF, -INF), (30.0, NAN, 30.0, NAN, NAN), (-1e30, INF, 0.0, NAN, NAN),
]


@pytest.mark.parametrize("act", [fb.SILU, fb.GELU])
@pytest.mark.parametrize("fast", [True, False])
@pytest.mark.parametrize("M", [2 * m for m in ROWS])
def test_gradient_of_projections_that_are_not_finite(act, fast, M):
    dy, b = units(M, 1)
    sa, sb = torch.ones((M, 1), device="cuda"), torch.ones((1, 4, 1), device="cuda")
    gu = torch.randn((M, 2 * F), device="cuda").to(BF16)
    clean, clean_h = feedforward.mgs_mm_gated_grad_block128(dy, sa, b, sb, gu, None, act, fast, hidden=True)
    at = [(r, c) for r in (0, 7, M - 1) for c in (0, 130, F - 9)]
    for r, c in at:
        for i, (g, u, *_) in enumerate(SPECIAL):
            gu[r, c + i], gu[r, F + c + i] = g, u
    dgu, h = feedforward.mgs_mm_gated_grad_block128(dy, sa, b, sb, gu, None, act, fast, hidden=True)
    same = torch.ones((M, F), dtype=torch.bool, device="cuda")
    for r, c in at:
        for i, (_, _, du, dg, hidden) in enumerate(SPECIAL):
            got = [float(dgu[r, F + c + i]), float(dgu[r, c + i]), float(h[r, c + i])]
            assert np.array_equal(np.float64(got), np.float64([du, dg, hidden]), equal_nan=True), (r, c, i, got)
            same[r, c + i] = False
    assert torch.equal(h[same], clean_h[same]) and torch.equal(dgu[torch.cat([same, same], 1)], clean[torch.cat([same, same], 1)])


@pytest.mark.parametrize("act", [fb.SILU, fb.GELU])
@pytest.mark.parametrize("M", ROWS)
def test_projections_that_are_not_numbers(act, M):
    """A weight's byte that is not a number makes its own column of h NaN, in either matrix."""
    a, b = units(M, 2)
    sa, sb = torch.ones((M, 1), device="cuda"), torch.ones((2, 4, 1), device="cuda")
    clean = feedforward.mgs_mm_gated_block128(a, sa, b, sb, None, act)
    b[0, 17, 9], b[1, 300, 100] = 0x7F, 0xFF
    for fast in (True, False):
        h = feedforward.mgs_mm_gated_block128(a, sa, b, sb, None, act, fast)
        bad = torch.zeros((M, F), dtype=torch.bool, device="cuda")
        bad[:, [17, 300]] = True
        assert torch.equal(torch.isnan(h), bad) and torch.equal(h[~bad], clean[~bad])
