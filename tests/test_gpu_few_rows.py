"""The form for few rows: a row's bits are the same whether its workgroup has
one tile or walks through many, and where rows end inside a block nothing of
what lies behind them is taken."""
import numpy as np
import pytest
import torch

import experts_ref as ref
import group_scaling_fp8_amd as mgs
from group_scaling_fp8_amd import feedforward, workloads as wl
from gpu_util import to_dev
from test_gpu_gated import operands
from test_gpu_mm import OUT, check

pytestmark = pytest.mark.gpu

G, ROWS, N = 70, 9, 4128        # 70 groups of nine rows, 129 tiles of 32 columns each: more tiles than workgroups


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mgs.lib()


def calls(K):
    """Each call on rows r of group e (and on all of them), as f(rows, weights, offsets)."""
    rng = np.random.default_rng(K)
    M = G * ROWS
    (a, sa, b, sb), _ = operands(rng, M, K, 2 * G, N, [M])
    a, sa, b, sb = (to_dev(v) for v in (a, sa, b, sb))
    gu = to_dev(wl.randn_bf16(rng, (M, 2 * N), 1.0)).view(torch.bfloat16)
    q, qs = feedforward.mgs_quant_rows_i8(to_dev(wl.randn_bf16(rng, (M, K), 1.0)).view(torch.bfloat16))
    w, ws = feedforward.mgs_quant_rows_i8(to_dev(wl.randn_bf16(rng, (2 * G, N, K), 0.1)).view(torch.bfloat16))

    def one(e):
        return slice(e, e + 1)

    def two(e):
        return slice(2 * e, 2 * e + 2)
    return {
        "block128": lambda r, e, off: [mgs.mgs_mm_block128(a[r], sa[r], b[e], sb[e], off, torch.float32)],
        "gated": lambda r, e, off: feedforward.mgs_mm_gated_block128(a[r], sa[r], b[e], sb[e], off, keep=True),
        "gated fast": lambda r, e, off: feedforward.mgs_mm_gated_block128(a[r], sa[r], b[e], sb[e], off, fast_accum=True,
                                                                          keep=True),
        "grad": lambda r, e, off: feedforward.mgs_mm_gated_grad_block128(a[r], sa[r], b[e], sb[e], gu[r], off, hidden=True),
        "grad fast": lambda r, e, off: feedforward.mgs_mm_gated_grad_block128(a[r], sa[r], b[e], sb[e], gu[r], off,
                                                                              fast_accum=True, hidden=True),
        "i8": lambda r, e, off: [feedforward.mgs_mm_i8(q[r], qs[r], w[e], ws[e], off, torch.float32)],
        "gated i8": lambda r, e, off: [feedforward.mgs_mm_gated_i8(q[r], qs[r], w[e], ws[e], off)],
    }, {n: two if n.startswith("gated") else one for n in ("block128", "gated", "gated fast", "grad", "grad fast", "i8", "gated i8")}


@pytest.mark.parametrize("K", [16, 400, 1040, 1296])
def test_one_tile_and_many(K):
    offsets = torch.arange(ROWS, G * ROWS + 1, ROWS, dtype=torch.int32, device="cuda")
    fs, weights = calls(K)
    for name, f in fs.items():
        print(name, flush=True)
        whole = f(slice(None), slice(0, (2 if name.startswith("gated") else 1) * G), offsets)
        for e in (0, 1, 33, 64, G - 1):
            rows = slice(e * ROWS, (e + 1) * ROWS)
            alone = f(rows, weights[name](e), None)
            for x, y in zip(whole, alone):
                assert torch.equal(x[rows].contiguous().view(torch.uint8), y.view(torch.uint8)), (name, e)


@pytest.mark.parametrize("K", [16, 48, 112, 144, 1040, 1168])
@pytest.mark.parametrize("M", [1, 16, 30])
def test_rows_that_end_inside_a_block(K, M):
    """What follows the last row and the last weight in memory is not a number, and the
    rows' first bytes are the largest: neither may reach the sums."""
    rng = np.random.default_rng(K + M)
    cols = 48
    a, b = (np.full((n + 1, K), 0x7F, np.uint8) for n in (M, cols))
    a[:M], b[:cols] = rng.integers(0, 64, (M, K)), rng.integers(0, 64, (cols, K))
    a[:M, :16], b[:cols, :16] = 0x7E, 0x7E
    kb = -(-K // 128)
    sa, sb = np.ones((M, kb), np.float32), np.ones((1, 1, kb), np.float32)
    x, w = to_dev(a), to_dev(b)
    y = mgs.mgs_mm_block128(x[:M], to_dev(sa), w[None, :cols], to_dev(sb), None, torch.float32)
    want, mag = ref.mm_block128(a[:M], sa, b[None, :cols], sb, [M])
    check(y.cpu().numpy(), want, ref.mm_tolerance(want, mag, K, "f32", False), (M, K))
    q, p = a.view(np.int8).copy(), b.view(np.int8).copy()
    y = feedforward.mgs_mm_i8(to_dev(q)[:M], torch.ones(M, device="cuda"), to_dev(p)[None, :cols],
                              torch.ones((1, cols), device="cuda"), None, OUT["f32"])
    assert np.array_equal(y.cpu().numpy(), (q[:M].astype(np.int64) @ p[:cols].astype(np.int64).T).astype(np.float32))
