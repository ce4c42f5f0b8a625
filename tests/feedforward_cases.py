"""Sizes of the gated and the 8-bit integer products for the tests, with the
form that each takes on 256 compute units (tests/test_feedforward_host.py checks
it against the library's rule; a gated pair counts as one product of twice the
columns)."""

# rows a tile of the few-row form (or 0), tile of the form through LDS, sets of waves
FEW16, FEW32, FEW64 = (16, 0, 0), (32, 0, 0), (64, 0, 0)
TILE128, TWO128, TILE256 = (0, 128, 1), (0, 128, 2), (0, 256, 1)

# M, N, K, groups, ends; form with 8-bit sums; with binary32 sums
ROWS = [
    (1, 16, 16, 1, "none", FEW16, FEW16),
    (1, 144, 272, 1, "none", FEW16, FEW16),
    (17, 272, 1040, 1, "none", FEW16, FEW16),
    (64, 272, 528, 4, "tail", FEW16, FEW16),
    (80, 80, 160, 70, "even", FEW16, FEW16),
    (96, 272, 400, 12, "bad", FEW16, FEW16),
    (300, 400, 272, 1, "none", FEW16, FEW16),
    (48, 144, 144, 2, "empty", FEW16, FEW16),
    (20, 16448, 144, 1, "none", FEW16, FEW16),
    (33, 4064, 144, 1, "none", FEW32, FEW32),
    (40, 8224, 400, 1, "even", FEW32, FEW32),
    (900, 144, 144, 6, "bad", FEW32, FEW32),
    (600, 272, 528, 5, "tail", FEW32, FEW32),
    (700, 528, 1040, 1, "none", FEW64, FEW64),
    (700, 528, 16, 5, "one", FEW64, FEW64),
    (1000, 272, 272, 9, "even", FEW64, FEW64),
    (1300, 272, 144, 3, "empty", FEW64, FEW64),
    (1300, 272, 400, 8, "bad", FEW64, FEW64),
    (700, 1200, 656, 1, "none", TWO128, TILE128),
    (2000, 1200, 528, 5, "tail", TWO128, TILE128),
    (1500, 1200, 16, 4, "one", TWO128, TILE128),
    (1500, 1200, 272, 4, "empty", TWO128, TILE128),
    (2000, 1200, 144, 5, "bad", TWO128, TILE128),
    (1003, 4192, 272, 1, "none", TILE128, TILE128),
    (2000, 2336, 528, 5, "even", TILE128, TILE128),
    (2000, 2336, 400, 5, "bad", TILE128, TILE128),
    (4100, 4128, 528, 1, "none", TILE128, TILE128),
    (3000, 4128, 144, 12, "tail", TILE128, TILE128),
    (640, 4128, 144, 40, "bad", TILE128, FEW16),
    (8200, 4000, 144, 6, "even", TILE256, TILE128),
    (8200, 4000, 400, 5, "tail", TILE256, TILE128),
    (9000, 4256, 16, 3, "bad", TILE256, TILE128),
    (8200, 4000, 272, 5, "one", TILE256, TILE128),
    (9000, 4256, 144, 4, "empty", TILE256, TILE128),
    (8200, 4128, 528, 1, "none", TILE256, TILE128),
]

# F of a gated pair is half of N where that is a multiple of 16, else the next one
GATED = [(M, N // 32 * 16 + (16 if N % 32 else 0), *rest) for M, N, *rest in ROWS]
