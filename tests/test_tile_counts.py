"""CPU check of how many tiles rows take (mgs_mm_form.hpp), up to the most
rows that a call accepts, where the sum of both passes 31 bits."""
import subprocess

import pytest

from test_mm_form import CSRC

PROGRAM = r"""
#include <stdio.h>
#include "mgs_mm_form.hpp"
static_assert(mgs::tiles_down(0, 16) == 0, "a constant");
int main() {
    int rows, high;
    while (scanf("%d %d", &rows, &high) == 2) printf("%d\n", mgs::tiles_down(rows, high));
    return 0;
}
"""


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    d = tmp_path_factory.mktemp("tiles")
    (d / "tiles.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC, "-o",
                    str(d / "tiles"), str(d / "tiles.cpp")], check=True)

    def run(args):
        r = subprocess.run([str(d / "tiles")], input="\n".join("%d %d" % a for a in args), capture_output=True, text=True,
                           check=True)
        return [int(v) for v in r.stdout.split()]
    return run


def test_tiles_of_rows(tiles):
    most = 2 ** 31 - 1
    args = [(rows, high) for high in (16, 32, 64, 128, 256)
            for rows in (0, 1, high - 1, high, high + 1, 4099, most - 256, most - high, most - high + 1, most - 15, most - 1, most)]
    assert tiles(args) == [-(-rows // high) for rows, high in args]
