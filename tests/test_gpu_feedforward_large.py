"""Outputs of the gated and the integer calls past 2^31 and 2^32 bytes: rows
that repeat give rows that repeat, wherever in memory they lie."""
import pytest
import torch

import feedforward_bounds as fb
import group_scaling_fp8_amd as mgs
from group_scaling_fp8_amd import feedforward
from test_gpu_long_products import codes, generator, scales

pytestmark = pytest.mark.gpu

M, PERIOD, F, K = 140001, 4111, 8192, 144          # gu and dgu 4.6 GB, h 2.3 GB
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _memory():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mgs.lib()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GiB")
    yield
    torch.cuda.empty_cache()


def repeated(t):
    return t[torch.arange(M, device="cuda") % PERIOD].contiguous()


def check_repeats(y):
    first = y[:PERIOD]
    for at in range(PERIOD, M, PERIOD):
        part = y[at:at + PERIOD]
        assert torch.equal(part, first[:part.shape[0]]), at


def operands(gen, W):
    kb = -(-K // 128)
    a, b = codes(gen, "codes", (PERIOD, K)), codes(gen, "codes", (W, F, K))
    return (a, scales(gen, "codes", (PERIOD, kb), K), b, scales(gen, "codes", (W, F // 128, kb), K))


@pytest.mark.parametrize("fast", [True, False])
def test_gated_and_gradient(fast):
    gen = generator(1)
    a, sa, b, sb = operands(gen, 2)
    (g, mg), (u, mu) = (fb.products(a, sa, b, sb, [PERIOD], 2, j, False) for j in (0, 1))
    eg, eu = fb.sum_error(g, mg, K, fast), fb.sum_error(u, mu, K, fast)
    h, gu = feedforward.mgs_mm_gated_block128(repeated(a), repeated(sa), b, sb, None, fb.SILU, fast, keep=True)
    assert fb.differ(h[:PERIOD], *fb.gated(fb.SILU, g, eg, u, eu)) == (0, None)
    both = torch.cat([g, u], 1)
    assert fb.differ(gu[:PERIOD], both, fb.half(both, torch.cat([eg, eu], 1))) == (0, None)
    check_repeats(h)
    check_repeats(gu)
    del h, g, u, mg, mu, eg, eu, both
    a, sa, b, sb = operands(gen, 1)
    dh, mag = fb.products(a, sa, b, sb, [PERIOD], 1, 0, False)
    kept = gu[:PERIOD].double()
    (dg, tg), (du, tu), (want, tol) = fb.gated_grad(fb.SILU, dh, fb.sum_error(dh, mag, K, fast), kept[:, :F], kept[:, F:])
    a, sa = repeated(a), repeated(sa)
    dgu, h = feedforward.mgs_mm_gated_grad_block128(a, sa, b, sb, gu, None, fb.SILU, fast, hidden=True)
    assert fb.differ(dgu[:PERIOD], torch.cat([dg, du], 1), torch.cat([tg, tu], 1)) == (0, None)
    assert fb.differ(h[:PERIOD], want, tol) == (0, None)
    check_repeats(dgu)
    check_repeats(h)
    again = feedforward.mgs_mm_gated_grad_block128(a, sa, b, sb, gu, None, fb.SILU, fast, dgu=gu)       # in place
    assert again is gu and torch.equal(gu.view(torch.int16), dgu.view(torch.int16))


def test_integers():
    gen = generator(2)
    a = torch.randint(-128, 128, (PERIOD, K), generator=gen, device="cuda", dtype=torch.int8)
    b = torch.randint(-128, 128, (2, F, K), generator=gen, device="cuda", dtype=torch.int8)
    sa = torch.exp2(torch.rand((PERIOD,), generator=gen, device="cuda") * 2 + 7)
    sb = torch.exp2(torch.rand((2, F), generator=gen, device="cuda") * 2 + 7)
    rows, srows = repeated(a), repeated(sa)
    y = feedforward.mgs_mm_i8(rows, srows, b[:1], sb[:1], None, torch.float32)
    want = (a.double() @ b[0].double().t()).float() * (1 / sa[:, None]) * (1 / sb[0])
    assert torch.equal(y[:PERIOD], want)
    check_repeats(y)
    del y
    h = feedforward.mgs_mm_gated_i8(rows, srows, b, sb, None, fb.GELU)
    g, u = (fb.products(a, sa, b, sb, [PERIOD], 2, j, True)[0] for j in (0, 1))
    assert fb.differ(h[:PERIOD], *fb.gated(fb.GELU, g, g.abs() * 6 * fb.U, u, u.abs() * 6 * fb.U)) == (0, None)
    check_repeats(h)
