"""CPU check of the lines of weights that a tile of few rows takes in 8-bit
integers: by the blocks a wave has, the tiles a workgroup walks and rows that
begin on the same channels of memory."""
import pytest

from test_feedforward_host import form  # noqa: F401  (a fixture)
from test_mm_form import CUS


@pytest.mark.parametrize("M,N,G,least", [
    (128, 16384, 16, 28),        # 4 tokens to 2 of 16 experts, both projections of 8192 columns: many tiles a workgroup
    (1024, 4096, 64, 28),        # 16 tokens to 4 of 64 experts
    (272, 4096, 16, 40),         # 16 tokens to 2 of 16 experts of few columns
    (16, 32768, 1, 40), (1, 65536, 1, 40),
])
def test_lines_by_blocks(form, M, N, G, least):  # noqa: F811
    for K in (*range(128, 9000, 128), *range(144, 9000, 272)):
        want = 64 if K // 128 >= least and K % 4096 else 32
        assert form(1, 1, G > 1, M, N, K, G, CUS) == (16, want, 0), K
        assert form(0, 1, G > 1, M, N, K, G, CUS) == (16, 64, 0), K
