"""CPU check of the sizes of tests/test_gpu_long_products.py: the forms they take, and that every
form of tiles runs steps whose loads and scales were started by earlier steps of the same tile."""
import pytest

from feedforward_cases import TILE128, TILE256, TWO128
from feedforward_long_cases import LONG, half_columns
from test_feedforward_host import form  # noqa: F401  (a fixture)
from test_mm_form import CUS

MIN_STEPS = 3        # that a tile's loads run ahead by, scales included


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("case", LONG, ids=str)
def test_forms(form, case, gated):  # noqa: F811
    M, N, K, G, kind, ints, fast, exact = case
    N = 2 * half_columns(N) if gated else N
    for args, want in (((1, 1), ints), ((0, 1), fast), ((0, 0), exact)):
        assert form(*args, kind != "none", M, N, K, G, CUS) == want


def test_every_form_of_tiles_runs_long():
    for tile in (TWO128, TILE128, TILE256):
        assert max(-(-c[2] // (128 * tile[2])) for c in LONG if tile in c[5:]) > MIN_STEPS + 4, tile
    # and the two sets of waves of a tile run unlike numbers of steps
    assert any(-(-c[2] // 128) % 2 for c in LONG if TWO128 in c[5:])
