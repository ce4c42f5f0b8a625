"""Integer products bit for bit as include/mgs.h says they are rounded: the
exact sum to fp32, times fl32(1 / a_scales), times fl32(1 / b_scales)."""
import numpy as np
import pytest
import torch

import group_scaling_fp8_amd as mgs
from feedforward_cases import FEW16_32, FEW32_32, FEW16_64, FEW32_64, FEW64_64, ROWS, TILE128, TILE256, TWO128
from group_scaling_fp8_amd import feedforward
from gpu_util import to_dev
from test_gpu_gated import groups
from test_gpu_i8 import operands

pytestmark = pytest.mark.gpu

FORMS = (FEW16_32, FEW32_32, FEW16_64, FEW32_64, FEW64_64, TWO128, TILE128, TILE256)
CASES = [next(c for c in ROWS if c[5] == f and c[2] > 128) for f in FORMS]        # one of each form


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mgs.lib()


@pytest.mark.parametrize("case", CASES, ids=str)
def test_roundings(case):
    M, N, K, G, kind, *_ = case
    rng = np.random.default_rng(N)
    off, ends = groups(rng, kind, M, G)
    (a, sa, b, sb), _ = operands(rng, M, K, G, N, ends)
    y = feedforward.mgs_mm_i8(*[to_dev(v) for v in (a, sa, b, sb)], None if off is None else to_dev(off), torch.float32)
    one, first = np.float32(1), 0
    want = np.zeros((M, N), np.float32)
    for e, end in enumerate(ends):
        if end > first:
            total = a[first:end].astype(np.float64) @ b[e].astype(np.float64).T          # exact below 2^53
            want[first:end] = total.astype(np.float32) * (one / sa[first:end, None]) * (one / sb[e])
        first = max(first, end)
    assert np.array_equal(y.cpu().numpy().view(np.uint32), want.view(np.uint32))
