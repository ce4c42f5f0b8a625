"""The gated pair, its gradient and the integer products in every kind of their
kernels (faster or binary32 sums; with and without what is stored beside) on
tiles that run many steps: whole outputs against 64 bits.

Two kinds of operands, as in test_gpu_mm_forms: codes of every exponent within
a bound counted from the roundings, and halves of whole numbers with scales
that are powers of two, whose products and sums are exact in either form, so
that kept projections are the exact sums rounded once."""
import numpy as np
import pytest
import torch

import experts_ref as ref
import feedforward_bounds as fb
import group_scaling_fp8_amd as mgs
from feedforward_long_cases import LONG, half_columns
from group_scaling_fp8_amd import feedforward
from gpu_util import Guarded, to_dev
from test_gpu_mm import ends_of
from test_gpu_mm_forms import HALVES

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mgs.lib()


def generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def codes(gen, kind, shape):
    """E4M3 bytes without NaN."""
    if kind == "halves":
        return to_dev(HALVES)[torch.randint(0, len(HALVES), shape, generator=gen, device="cuda")]
    sign = torch.randint(0, 2, shape, generator=gen, device="cuda", dtype=torch.uint8) * 128
    return torch.randint(0, 127, shape, generator=gen, device="cuda", dtype=torch.uint8) | sign


def scales(gen, kind, shape, K):
    """That bring sums of K products to between 1 and 100 (codes, whose products are about 2^14 in their mean square) or
    to about 1 (halves, 2^0.5)."""
    at = 0.25 * np.log2(K)
    if kind == "halves":
        return torch.exp2(torch.randint(-1, 2, shape, generator=gen, device="cuda") + round(at + 0.25)).float()
    return torch.exp2(torch.rand(shape, generator=gen, device="cuda") * 4 - 2 + 5.5 + at)


def groups(case):
    M, G, kind = case[0], case[3], case[4]
    off = ends_of(kind, M, G, np.random.default_rng(M + G))
    return None if off is None else to_dev(off), ref.clean_ends(off if off is not None else [M], M)


def operands(gen, kind, M, K, W, N, ends):
    kb = -(-K // 128)
    a, b = codes(gen, kind, (M, K)), codes(gen, kind, (W, N, K))
    sa, sb = scales(gen, kind, (M, kb), K), scales(gen, kind, (W, -(-N // 128), kb), K)
    a[ends[-1]:], sa[ends[-1]:] = 0x7F, float("nan")        # of no group
    return a, sa, b, sb


def summed(held, ends, matrices, first, kind, fast):
    """A product and its error."""
    y, mag = fb.products(*held, ends, matrices, first, False)
    return y, torch.zeros_like(y) if kind == "halves" else fb.sum_error(y, mag, held[0].shape[1], fast)


@pytest.mark.parametrize("case", LONG, ids=str)
@pytest.mark.parametrize("kind", ["codes", "halves"])
@pytest.mark.parametrize("fast,act", [(True, fb.SILU), (False, fb.GELU)])
def test_gated(case, kind, fast, act):
    M, N, K, G = case[:4]
    F = half_columns(N)
    off, ends = groups(case)
    held = operands(generator(M + F), kind, M, K, 2 * G, F, ends)
    (g, eg), (u, eu) = (summed(held, ends, 2, j, kind, fast) for j in (0, 1))
    want, tol = fb.gated(act, g, eg, u, eu)
    for keep in (True, False):
        h, gu = Guarded((M, F), BF16), Guarded((M, 2 * F), BF16) if keep else None
        feedforward.mgs_mm_gated_block128(*held, off, act, fast, h=h.view, gu=gu.view if keep else None)
        torch.cuda.synchronize()
        h.check()
        assert fb.differ(h.view, want, tol) == (0, None), keep
        if keep:
            gu.check()
            both, e = torch.cat([g, u], 1), torch.cat([eg, eu], 1)
            if kind == "halves":
                assert torch.equal(gu.view, both.to(BF16))
            else:
                assert fb.differ(gu.view, both, fb.half(both, e)) == (0, None)


@pytest.mark.parametrize("case", LONG, ids=str)
@pytest.mark.parametrize("kind", ["codes", "halves"])
@pytest.mark.parametrize("fast,act", [(True, fb.GELU), (False, fb.SILU)])
def test_gated_grad(case, kind, fast, act):
    M, F, D, G = case[:4]
    off, ends = groups(case)
    gen = generator(M + F + 1)
    held = operands(gen, kind, M, D, G, F, ends)
    gu = (torch.randn((M, 2 * F), generator=gen, device="cuda") * 2).to(BF16)
    gu[ends[-1]:] = 0
    dh, edh = summed(held, ends, 1, 0, kind, fast)
    (dg, tg), (du, tu), (want, tol) = fb.gated_grad(act, dh, edh, gu[:, :F].double(), gu[:, F:].double())
    gu[ends[-1]:] = float("nan")
    for hidden in (True, False):
        dgu, h = Guarded((M, 2 * F), BF16), Guarded((M, F), BF16) if hidden else None
        feedforward.mgs_mm_gated_grad_block128(*held, gu, off, act, fast, dgu=dgu.view, h=h.view if hidden else None)
        torch.cuda.synchronize()
        dgu.check()
        assert fb.differ(dgu.view, torch.cat([dg, du], 1), torch.cat([tg, tu], 1)) == (0, None), hidden
        if hidden:
            h.check()
            assert fb.differ(h.view, want, tol) == (0, None)


@pytest.mark.parametrize("case", LONG, ids=str)
def test_integers(case):
    """Products bit for bit (the exact sum to fp32, times both reciprocals), the gated pair within its roundings."""
    M, N, K, G = case[:4]
    off, ends = groups(case)
    gen = generator(M + N + 2)
    F = half_columns(N)
    a = torch.randint(-128, 128, (M, K), generator=gen, device="cuda", dtype=torch.int8)
    b = torch.randint(-128, 128, (2 * G, max(N, F), K), generator=gen, device="cuda", dtype=torch.int8)
    near = 0.25 * np.log2(K) + 6                # sums near 1
    sa = torch.exp2(torch.rand((M,), generator=gen, device="cuda") * 2 - 1 + near)
    sb = torch.exp2(torch.rand((2 * G, max(N, F)), generator=gen, device="cuda") * 2 - 1 + near)
    sa[ends[-1]:] = float("nan")
    one = [t[:G, :N].contiguous() for t in (b, sb)]
    total = torch.zeros((M, N), device="cuda")
    first = 0
    for e, end in enumerate(ends):
        if end > first:
            s = (a[first:end].double() @ one[0][e].double().t()).float()
            total[first:end] = s * (1 / sa[first:end, None]) * (1 / one[1][e])
        first = max(first, end)
    for out in (torch.float32, BF16):
        y = Guarded((M, N), out)
        feedforward.mgs_mm_i8(a, sa, *one, off, out, y=y.view)
        torch.cuda.synchronize()
        y.check()
        assert torch.equal(y.view, total.to(out)), out
    two = [t[:, :F].contiguous() for t in (b, sb)]
    g, u = (fb.products(a, sa, *two, ends, 2, j, True)[0] for j in (0, 1))
    for act in (fb.SILU, fb.GELU):
        h = Guarded((M, F), BF16)
        feedforward.mgs_mm_gated_i8(a, sa, *two, off, act, h=h.view)
        torch.cuda.synchronize()
        h.check()
        want, tol = fb.gated(act, g, g.abs() * 6 * fb.U, u, u.abs() * 6 * fb.U)
        assert fb.differ(h.view, want, tol) == (0, None), act
