"""The 8-bit integer calls: the cast byte for byte, products whose sums are
exact against whole numbers, and the gated pair within its roundings."""
import numpy as np
import pytest
import torch

import experts_ref as ref
import feedforward_ref as ff
import group_scaling_fp8_amd as mgs
from feedforward_cases import GATED, ROWS
from group_scaling_fp8_amd import feedforward, workloads as wl
from gpu_util import Guarded, assert_same_bytes, to_dev
from test_gpu_gated import groups
from test_gpu_mm import OUT, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mgs.lib()


# every width class of the cast and its edges; rows that do not fill a workgroup
@pytest.mark.parametrize("M,K", [(1, 8), (5, 16), (17, 120), (33, 512), (7, 520), (1, 2048), (9, 2056), (3, 5120), (2, 8192),
                                 (5, 8200), (2, 16384), (3, 16392), (2, 32768), (2, 40000), (1, 131056), (1, 131072), (2, 131080),
                                 (1, 300000), (1000, 136), (6, 4096), (5, 4104)])
def test_cast(M, K):
    rng = np.random.default_rng(M + K)
    x = wl.randn_bf16(rng, (M, K), 0.5, 0.01, 20.0)
    x[M // 2] = 0                                                # a row of zeros
    x[0, K // 2] = 0x8000                                        # -0
    x[-1, :8] = wl.f32_to_bf16_bits(np.float32([1e-38, -1e-38, 3e38, -3e38, 1e30, 0, 1, -1]))[:8]
    q, s = Guarded((M, K), torch.int8), Guarded((M,), torch.float32)
    feedforward.mgs_quant_rows_i8(to_dev(x), q=q.view, scales=s.view)
    torch.cuda.synchronize()
    q.check()
    s.check()
    want_q, want_s = ff.quant_rows_i8(x)
    assert_same_bytes(q.numpy(), want_q, "q")
    assert_same_bytes(s.numpy(), want_s, "scales")


def test_cast_of_every_value_beside_a_maximum():
    """All finite bf16 below each of many maxima, ties among them."""
    mags = np.arange(0, 0x7F80, dtype=np.uint16)
    rng = np.random.default_rng(0)
    for top in [0x0001, 0x0080, 0x2B8D, 0x3F80, 0x3FFF, 0x42FE, 0x437F, 0x7F7F, *rng.integers(0x3000, 0x5000, 24).tolist()]:
        v = mags[mags <= top]
        row = np.zeros(-(-2 * len(v) // 8) * 8 + 8, np.uint16)
        row[0], row[8:8 + len(v)], row[8 + len(v):8 + 2 * len(v)] = top, v, v | 0x8000
        q, s = feedforward.mgs_quant_rows_i8(to_dev(row[None]))
        want_q, want_s = ff.quant_rows_i8(row[None])
        assert_same_bytes(q.cpu().numpy(), want_q, hex(top))
        assert_same_bytes(s.cpu().numpy(), want_s, hex(top))


def test_cast_of_more_rows_than_a_launch_has_workgroups():
    """2^24 rows and a few: workgroups walk on. Every row against the first ones, whose values it repeats."""
    M, period = (1 << 24) + 37, 4099
    x = torch.from_numpy(wl.randn_bf16(np.random.default_rng(5), (period, 8), 0.5, 0.01, 20.0).view(np.int16)).cuda()
    rows = torch.arange(M, device="cuda") % period
    q, s = feedforward.mgs_quant_rows_i8(x[rows])
    want_q, want_s = ff.quant_rows_i8(x.cpu().numpy().view(np.uint16))
    assert_same_bytes(q[:period].cpu().numpy(), want_q, "q")
    assert_same_bytes(s[:period].cpu().numpy(), want_s, "scales")
    assert torch.equal(q, q[:period][rows]) and torch.equal(s, s[:period][rows])


def test_cast_of_weights():
    rng = np.random.default_rng(1)
    w = wl.randn_bf16(rng, (3, 48, 272), 0.02, 0.001, 0.5)
    q, s = feedforward.mgs_quant_rows_i8(to_dev(w).view(torch.bfloat16))
    want_q, want_s = ff.quant_rows_i8(w)
    assert q.shape == (3, 48, 272) and s.shape == (3, 48)
    assert_same_bytes(q.cpu().numpy(), want_q, "q")
    assert_same_bytes(s.cpu().numpy(), want_s, "scales")


def whole(rng, shape):
    return rng.integers(-128, 128, size=shape).astype(np.int8)


def operands(rng, M, K, W, N, ends, least=-3, most=12):
    a, b = whole(rng, (M, K)), whole(rng, (W, N, K))
    sa, sb = (np.exp2(rng.uniform(least, most, size=s)).astype(np.float32) for s in ((M,), (W, N)))
    last = max([0, *ends])
    clean = [v.copy() for v in (a, sa)]
    sa[last:] = np.nan                       # of no group
    clean[0][last:], clean[1][last:] = 0, 1
    return (a, sa, b, sb), (*clean, b, sb)


@pytest.mark.parametrize("case", ROWS, ids=str)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_product(case, out):
    M, N, K, G, kind, *_ = case
    rng = np.random.default_rng(M * 3 + N + K)
    off, ends = groups(rng, kind, M, G)
    held, clean = operands(rng, M, K, G, N, ends)
    y = Guarded((M, N), OUT[out])
    feedforward.mgs_mm_i8(*[to_dev(v) for v in held], None if off is None else to_dev(off), OUT[out], y=y.view)
    torch.cuda.synchronize()
    y.check()
    want, tol = ff.product(*clean, ends, "i8")
    check(y.view.float().cpu().numpy(), want, tol if out == "f32" else ff.half(want, tol), case)


@pytest.mark.parametrize("M,N,K,G", [(3, 64, 131056, 1), (130, 144, 131056, 1), (700, 528, 4096, 1), (2100, 4112, 1024, 1)])
def test_sums_are_exact(M, N, K, G):
    """Scales of 1: sums below 2^24 come back as they are, larger ones rounded
    once, up to the largest that any bytes give."""
    rng = np.random.default_rng(N)
    a, b = whole(rng, (M, K)), whole(rng, (G, N, K))
    a[0], b[0, 5] = -128, -128               # 2^14 K: one less than 2^31 would hold no more
    a[1], b[0, 6] = 127, -128
    one = lambda *s: torch.ones(s, dtype=torch.float32, device="cuda")  # noqa: E731
    y = feedforward.mgs_mm_i8(to_dev(a), one(M), to_dev(b), one(G, N), None, torch.float32).cpu().numpy()
    _, want = ff.mm_i8(a, np.ones(M, np.float32), b, np.ones((G, N), np.float32), [M])
    assert want[0, 5] == 16384.0 * K and np.array_equal(y, want.astype(np.float32))


@pytest.mark.parametrize("case", GATED, ids=str)
@pytest.mark.parametrize("act", [ff.SILU, ff.GELU])
def test_gated(case, act):
    M, F, K, G, kind, *_ = case
    rng = np.random.default_rng(M * 5 + F + K)
    off, ends = groups(rng, kind, M, G)
    near = 0.5 * np.log2(K) / 2 + 6          # sums near 1
    held, clean = operands(rng, M, K, 2 * G, F, ends, near - 1, near + 1)
    h = Guarded((M, F), torch.bfloat16)
    feedforward.mgs_mm_gated_i8(*[to_dev(v) for v in held], None if off is None else to_dev(off), act, h=h.view)
    torch.cuda.synchronize()
    h.check()
    (want, tol), _ = ff.gated(*clean, ends, act, "i8")
    check(h.view.float().cpu().numpy(), want, tol, case)


def test_forms_agree():
    """A row's result is the same whatever batch it comes in: the sums are exact and scaled alike."""
    rng = np.random.default_rng(8)
    M, N, K = 4100, 2064, 272
    held, _ = operands(rng, M, K, 2, N, [M])
    a, sa, b, sb = (to_dev(v) for v in held)
    y = feedforward.mgs_mm_i8(a, sa, b[:1], sb[:1], None, torch.float32)
    h = feedforward.mgs_mm_gated_i8(a, sa, b, sb)
    for rows in (1, 30, 200, 1000):
        assert torch.equal(feedforward.mgs_mm_i8(a[:rows], sa[:rows], b[:1], sb[:1], None, torch.float32), y[:rows])
        assert torch.equal(feedforward.mgs_mm_gated_i8(a[:rows], sa[:rows], b, sb), h[:rows])


def test_empty_sizes():
    i8 = lambda *s: torch.ones(s, dtype=torch.int8, device="cuda")  # noqa: E731
    f32 = lambda *s: torch.ones(s, dtype=torch.float32, device="cuda")  # noqa: E731
    assert feedforward.mgs_mm_i8(i8(0, 64), f32(0), i8(1, 32, 64), f32(1, 32)).shape == (0, 32)
    assert not feedforward.mgs_mm_i8(i8(5, 0), f32(5), i8(1, 32, 0), f32(1, 32)).any()
    assert not feedforward.mgs_mm_gated_i8(i8(5, 0), f32(5), i8(2, 32, 0), f32(2, 32)).any()
    with pytest.raises(mgs.MgsError):
        feedforward.mgs_mm_i8(i8(1, 131072), f32(1), i8(1, 16, 131072), f32(1, 16))
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    q, s = feedforward.mgs_quant_rows_i8(x)
    assert q.shape == (0, 64) and s.shape == (0,)
