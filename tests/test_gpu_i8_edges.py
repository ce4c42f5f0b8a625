"""The 8-bit integer cast where there is nothing to cast."""
import numpy as np
import pytest
import torch

import group_scaling_fp8_amd as mgs
from group_scaling_fp8_amd import feedforward
from gpu_util import Guarded

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
