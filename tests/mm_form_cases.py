"""Products of every form that large and mid sizes take, for the tests: the
form each size takes on 256 compute units (tests/test_mm_form.py checks it
against the library's rule) and whether its workgroups walk several tiles."""

# rows a tile of the few-row form (or 0), tile of the form through LDS, sets of waves
FEW32, TILE128, TILE256 = (32, 0, 0), (0, 128, 1), (0, 256, 1)

# M, N, K, groups, ends; form with fast sums, with binary32 sums; whether there are
# more tiles than workgroups in both
BLOCK128 = [
    (21, 48, 144, 1, "even", FEW32, FEW32, False),
    (33, 272, 1040, 1, "none", FEW32, FEW32, False),
    (40, 8208, 400, 1, "none", FEW32, FEW32, False),
    (2000, 1040, 656, 5, "even", TILE128, TILE128, False),
    (1003, 4176, 400, 1, "none", TILE128, TILE128, False),
    (4000, 2320, 528, 6, "tail", TILE128, TILE128, True),
    (8200, 4000, 400, 6, "even", TILE256, TILE128, True),
    (8200, 4000, 1168, 6, "tail", TILE256, TILE128, True),
    (6000, 4112, 272, 70, "tail", TILE256, TILE128, True),
    (9000, 4240, 144, 3, "bad", TILE256, TILE128, True),
    (8200, 4000, 656, 5, "one", TILE256, TILE128, True),
    (9000, 4240, 272, 4, "empty", TILE256, TILE128, True),
    (4100, 4112, 1296, 1, "none", TILE256, TILE128, True),
    (4100, 4112, 16, 1, "none", TILE256, TILE128, True),
]

# the same for weight gradients; the forms of both sums agree
WGRAD = [
    (2064, 4112, 4000, 1, "even", TILE256, TILE256, True),
    (10400, 2064, 1936, 5, "even", TILE256, TILE256, True),
    (1040, 2064, 2064, 16, "tail", TILE256, TILE256, True),
    (1040, 2064, 2064, 16, "bad", TILE256, TILE256, True),
    (16400, 1296, 1296, 8, "one", TILE256, TILE256, True),
    (4096, 2064, 3600, 2, "tail", TILE256, TILE256, True),
    (0, 2064, 2064, 16, "empty", TILE256, TILE256, True),
    (8000, 1168, 1040, 8, "even", TILE128, TILE128, True),
    (5008, 1040, 1040, 3, "even", TILE128, TILE128, False),
]
