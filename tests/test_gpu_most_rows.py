"""Products of as many rows as a call accepts."""
import pytest
import torch

import group_scaling_fp8_amd as mgs

pytestmark = pytest.mark.gpu

ONE, TWO, THREE = 0x38, 0x40, 0x44        # E4M3


@pytest.fixture(autouse=True)
def _memory():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mgs.lib()
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def test_block128_of_2_to_the_31_rows_but_one():
    """Rows of ones and a few of twos: every row of y is 16 or 32 times its group's weight."""
    if torch.cuda.mem_get_info()[0] < 125 << 30:
        pytest.skip("needs 125 GiB")
    M = 2 ** 31 - 1
    at = [0, 4, 5, 255, 256, 1 << 30, M - 300, M - 257, M - 256, M - 255, M - 129, M - 128, M - 17, M - 16, M - 2, M - 1]
    a = torch.empty((M, 16), dtype=torch.uint8, device="cuda").fill_(ONE)
    a[at] = TWO
    sa = torch.ones((M, 1), device="cuda")
    b = torch.empty((2, 16, 16), dtype=torch.uint8, device="cuda").fill_(ONE)
    b[1] = THREE
    sb = torch.ones((2, 1, 1), device="cuda")
    y = torch.empty((M, 16), dtype=torch.bfloat16, device="cuda")
    for offsets, fast in ((None, True), (None, False), ([5, M], True), ([5, M], False), ([5, 5], True)):
        print(offsets, fast, flush=True)
        y.fill_(-1)
        off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
        mgs.mgs_mm_block128(a, sa, b[:1] if off is None else b, sb[:1] if off is None else sb, off, fast_accum=fast, y=y)
        weight = [lambda r: 1 if offsets is None or r < 5 else 3 if offsets[1] == M else 0][0]
        for r in at:
            assert bool((y[r] == 32 * weight(r)).all()), r
            y[r] = 16 * weight(r)
        assert bool((y[:5] == 16).all()) and all(bool((part == 16 * weight(9)).all()) for part in y[5:].split(1 << 27))
