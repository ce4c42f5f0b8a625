"""Sizes of the gated and the 8-bit integer products whose tiles run many steps,
with the form that each takes on 256 compute units (as in feedforward_cases;
tests/test_long_cases.py checks both)."""
from feedforward_cases import TILE128, TILE256, TWO128

# M, columns of one product, K, groups, ends; form of integers, of E4M3 with 8-bit sums, with binary32 sums
LONG = [
    (1500, 1200, 2064, 1, "none", TWO128, TWO128, TWO128),
    (2000, 1200, 5136, 5, "tail", TWO128, TWO128, TWO128),
    (1003, 4192, 2064, 1, "none", TILE128, TILE128, TILE128),
    (2000, 2336, 2192, 5, "bad", TILE128, TILE128, TILE128),
    (8200, 4000, 2064, 6, "even", TILE256, TILE256, TILE128),
    (8200, 4128, 1296, 1, "none", TILE256, TILE256, TILE128),
]


def half_columns(N):
    """F of a gated pair: half of N where that is a multiple of 16, else the next one."""
    return N // 32 * 16 + (16 if N % 32 else 0)
