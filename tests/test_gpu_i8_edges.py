"""The 8-bit integer cast where there is nothing to cast, and rows that are not
finite through the cast and the products."""
import numpy as np
import pytest
import torch

import feedforward_ref as ff
import group_scaling_fp8_amd as mgs
from group_scaling_fp8_amd import feedforward, workloads as wl
from gpu_util import Guarded, to_dev

pytestmark = pytest.mark.gpu

OF_ZEROS = np.float32(127) / np.float32(1e-12)


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mgs.lib()


def test_a_row_of_zeros():
    _, s = feedforward.mgs_quant_rows_i8(torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda"))
    assert (s.cpu().numpy() == OF_ZEROS).all()


@pytest.mark.parametrize("shape", [(5, 0), (3, 16, 0), (0, 0)])
@pytest.mark.parametrize("where", ["current", "stream", "handle"])
def test_rows_of_no_columns_have_the_scale_of_zeros(shape, where):
    x = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    stream = {"current": None, "stream": side, "handle": side.cuda_stream}[where]
    s = Guarded(shape[:-1], torch.float32)
    s.view.fill_(-1)
    torch.cuda.synchronize()
    q, got = feedforward.mgs_quant_rows_i8(x, scales=s.view, stream=stream)
    torch.cuda.synchronize()
    s.check()
    assert got is s.view and q.shape == shape and (s.numpy() == OF_ZEROS).all()
    held = [torch.full((64,), -1.0, device="cuda") for _ in range(64)]       # so that memory of this size is not zeros
    del held
    _, own = feedforward.mgs_quant_rows_i8(x, stream=stream)
    torch.cuda.synchronize()
    assert own.shape == shape[:-1] and (own.cpu().numpy() == OF_ZEROS).all()


def test_product_of_rows_of_no_columns():
    x, w = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((5, 0), (1, 32, 0)))
    y = feedforward.mgs_mm_i8(*feedforward.mgs_quant_rows_i8(x), *feedforward.mgs_quant_rows_i8(w))
    assert y.shape == (5, 32) and not y.any()


NOT_FINITE = {"nan": 0x7FC0, "-nan": 0xFFC1, "inf": 0x7F80, "-inf": 0xFF80}


@pytest.mark.parametrize("kind", NOT_FINITE)
@pytest.mark.parametrize("K", [8, 512, 2048, 4096, 8192, 16384, 32768, 131072, 131080])     # every width class of the cast
def test_cast_of_rows_that_are_not_finite(kind, K):
    """Such a row is zeros with the scale NaN or 0, wherever in the row the value stands; the others are as they were."""
    M = 9
    rng = np.random.default_rng(K)
    x = wl.randn_bf16(rng, (M, K), 0.5, 0.01, 20.0)
    clean_q, clean_s = ff.quant_rows_i8(x)
    bad = [1, 4, 8]
    for r, at in zip(bad, (0, K // 2, K - 1)):
        x[r, at] = NOT_FINITE[kind]
    q, s = (t.cpu().numpy() for t in feedforward.mgs_quant_rows_i8(to_dev(x)))
    others = np.setdiff1d(np.arange(M), bad)
    assert np.array_equal(q[others], clean_q[others]) and np.array_equal(s[others], clean_s[others])
    assert not q[bad].any()
    assert np.isnan(s[bad]).all() if "nan" in kind else (s[bad] == 0).all()


@pytest.mark.parametrize("kind", NOT_FINITE)
@pytest.mark.parametrize("M,N", [(3, 48), (40, 8224), (700, 1200), (2000, 4128), (8200, 4128)])     # few rows and every tile
def test_products_of_rows_that_are_not_finite(kind, M, N):
    """NaN in the rows of such tokens and the columns of such weights, nowhere else."""
    K = 272
    rng = np.random.default_rng(M)
    x, w = wl.randn_bf16(rng, (M, K), 0.5), wl.randn_bf16(rng, (2, N, K), 0.1)
    clean = feedforward.mgs_mm_i8(*feedforward.mgs_quant_rows_i8(to_dev(x)), *feedforward.mgs_quant_rows_i8(to_dev(w[:1])),
                                  None, torch.float32)
    x[1, 7], w[0, N - 2, 9], w[1, 5, 11] = [NOT_FINITE[kind]] * 3
    (a, sa), (b, sb) = feedforward.mgs_quant_rows_i8(to_dev(x)), feedforward.mgs_quant_rows_i8(to_dev(w))
    y = feedforward.mgs_mm_i8(a, sa, b[:1], sb[:1], None, torch.float32)
    bad = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    bad[1], bad[:, N - 2] = True, True
    assert torch.equal(torch.isnan(y), bad) and torch.equal(y[~bad], clean[~bad])
    bad[:, 5] = True
    h = feedforward.mgs_mm_gated_i8(a, sa, b, sb)
    assert torch.equal(torch.isnan(h), bad) and torch.isfinite(h[~bad]).all()
