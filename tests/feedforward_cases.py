"""Sizes of the gated and the 8-bit integer products for the tests, with the
form that each takes on 256 compute units (tests/test_feedforward_host.py checks
it against the library's rule; a gated pair counts as one product of twice the
columns)."""

# rows and lines of weights of a tile of the few-row form, or 0 and the tile of the form through LDS, sets of waves
FEW16_32, FEW32_32, FEW16_64, FEW32_64, FEW64_64 = (16, 32, 0), (32, 32, 0), (16, 64, 0), (32, 64, 0), (64, 64, 0)
TILE128, TWO128, TILE256 = (0, 128, 1), (0, 128, 2), (0, 256, 1)

# M, N, K, groups, ends; form of integers, of E4M3 with 8-bit sums, with binary32 sums
ROWS = [
    (1, 16, 16, 1, "none", FEW16_32, FEW16_32, FEW16_32),
    (1, 144, 272, 1, "none", FEW16_32, FEW16_32, FEW16_32),
    (17, 272, 1040, 1, "none", FEW16_32, FEW16_32, FEW16_32),
    (64, 272, 528, 4, "tail", FEW16_32, FEW16_32, FEW16_32),
    (80, 80, 160, 70, "even", FEW16_32, FEW16_32, FEW16_32),
    (96, 272, 400, 12, "bad", FEW16_32, FEW16_32, FEW16_32),
    (300, 400, 272, 1, "none", FEW16_32, FEW16_32, FEW16_32),
    (48, 144, 144, 2, "empty", FEW16_32, FEW16_32, FEW16_32),
    (20, 16448, 144, 1, "none", FEW16_32, FEW16_64, FEW16_64),
    (19, 8256, 1296, 1, "even", FEW32_64, FEW32_64, FEW32_64),
    (18, 16448, 5136, 1, "none", FEW16_64, FEW16_64, FEW16_64),
    (40, 32912, 5136, 2, "even", FEW16_64, FEW16_64, FEW16_64),
    (33, 4064, 144, 1, "none", FEW32_32, FEW32_32, FEW32_32),
    (600, 272, 528, 5, "tail", FEW32_32, FEW32_32, FEW32_32),
    (900, 144, 144, 6, "bad", FEW32_32, FEW32_32, FEW32_32),
    (30, 4064, 1040, 1, "even", FEW16_32, FEW16_32, FEW16_32),
    (250, 960, 272, 1, "none", FEW32_32, FEW32_32, FEW32_32),
    (1500, 1200, 144, 1, "none", TWO128, TWO128, TWO128),
    (1000, 160, 400, 9, "bad", FEW32_32, FEW32_32, FEW32_32),
    (30, 8192, 144, 1, "none", FEW32_32, FEW32_32, FEW32_32),
    (250, 960, 272, 4, "tail", FEW32_64, FEW32_64, FEW32_64),
    (300, 1184, 400, 4, "bad", FEW32_64, FEW32_64, FEW32_64),
    (40, 8224, 400, 1, "even", FEW64_64, FEW32_64, FEW32_64),
    (600, 400, 528, 5, "one", FEW32_64, FEW32_64, FEW32_64),
    (1300, 272, 144, 3, "empty", FEW32_64, FEW32_64, FEW32_64),
    (16, 16384, 144, 1, "none", FEW16_64, FEW16_64, FEW16_64),
    (640, 4128, 272, 40, "tail", FEW16_32, FEW16_64, FEW16_64),
    (700, 528, 1040, 1, "none", FEW32_64, FEW32_64, FEW32_64),
    (700, 528, 16, 5, "one", FEW32_64, FEW32_64, FEW32_64),
    (1000, 272, 272, 9, "even", FEW32_64, FEW32_64, FEW32_64),
    (1300, 272, 400, 8, "bad", FEW32_64, FEW32_64, FEW32_64),
    (40, 16384, 144, 1, "none", FEW64_64, FEW32_64, FEW32_64),
    (1000, 800, 272, 1, "none", FEW64_64, TWO128, FEW32_64),
    (1200, 544, 144, 9, "tail", FEW64_64, TWO128, FEW32_64),
    (700, 1200, 656, 1, "none", FEW64_64, TWO128, FEW32_64),
    (2000, 1200, 528, 5, "tail", TWO128, TWO128, TWO128),
    (1500, 1200, 16, 4, "one", TWO128, TWO128, TWO128),
    (1500, 1200, 272, 4, "empty", TWO128, TWO128, TWO128),
    (2000, 1200, 144, 5, "bad", TWO128, TWO128, TWO128),
    (1003, 4192, 272, 1, "none", TILE128, TILE128, TILE128),
    (2000, 2336, 528, 5, "even", TILE128, TILE128, TILE128),
    (2000, 2336, 400, 5, "bad", TILE128, TILE128, TILE128),
    (4100, 4128, 528, 1, "none", TILE128, TILE128, TILE128),
    (3000, 4128, 144, 12, "tail", TILE128, TILE128, TILE128),
    (640, 4128, 144, 40, "bad", FEW16_32, FEW16_64, FEW16_64),
    (900, 4128, 144, 30, "tail", TILE128, FEW32_64, FEW32_64),
    (8200, 4000, 144, 6, "even", TILE256, TILE256, TILE128),
    (8200, 4000, 400, 5, "tail", TILE256, TILE256, TILE128),
    (9000, 4256, 16, 3, "bad", TILE256, TILE256, TILE128),
    (8200, 4000, 272, 5, "one", TILE256, TILE256, TILE128),
    (9000, 4256, 144, 4, "empty", TILE256, TILE256, TILE128),
    (8200, 4128, 528, 1, "none", TILE256, TILE256, TILE128),
]

# F of a gated pair is half of N where that is a multiple of 16, else the next one
GATED = [(M, N // 32 * 16 + (16 if N % 32 else 0), *rest) for M, N, *rest in ROWS]
