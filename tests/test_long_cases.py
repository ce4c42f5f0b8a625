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


def test_forms_of_the_range_tests(form):  # noqa: F811
    """tests/test_gpu_activation_range.py: few rows, then each form of tiles, in a pair and in its gradient of twice the rows."""
    import test_gpu_activation_range as rt
    for rows, columns in ((rt.ROWS, 2 * rt.F), ([2 * m for m in rt.ROWS], rt.F)):
        fast = [form(0, 1, 0, m, columns, 128, 1, CUS) for m in rows]
        exact = [form(0, 0, 0, m, columns, 128, 1, CUS) for m in rows]
        assert fast[0][0] and exact[0][0] and fast[1:] == [TWO128, TILE128, TILE256], (fast, exact)
        assert exact[1:] == [TWO128, TILE128, TILE128], exact


def test_every_form_of_tiles_runs_long():
    for tile in (TWO128, TILE128, TILE256):
        assert max(-(-c[2] // (128 * tile[2])) for c in LONG if tile in c[5:]) > MIN_STEPS + 4, tile
    # and the two sets of waves of a tile run unlike numbers of steps
    assert any(-(-c[2] // 128) % 2 for c in LONG if TWO128 in c[5:])
