"""CPU check of the rule that chooses a product's form (mgs_mm_form.hpp),
compiled with g++ from the header that the library uses: the sizes of
tests/mm_form_cases.py take the forms they are there for, so that a changed
threshold cannot take a form out of the GPU tests unseen."""
import os
import subprocess

import pytest

from mm_form_cases import BLOCK128, WGRAD

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "group_scaling_fp8_amd", "csrc")
CUS = 256

PROGRAM = r"""
#include <stdio.h>
#include "mgs_mm_form.hpp"
int main() {
    long long wgrad, fast, grouped, M, N, K, G, cus;
    while (scanf("%lld %lld %lld %lld %lld %lld %lld %lld", &wgrad, &fast, &grouped, &M, &N, &K, &G, &cus) == 8) {
        const mgs::MmForm f = mgs::mm_form(wgrad, fast, grouped, M, N, K, G, (int)cus);
        printf("%d %d %d\n", f.few, f.tile, f.sets);
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def form(tmp_path_factory):
    d = tmp_path_factory.mktemp("form")
    (d / "form.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", CSRC, "-o", str(d / "form"), str(d / "form.cpp")], check=True)

    def run(*args):
        r = subprocess.run([str(d / "form")], input=" ".join(str(int(a)) for a in args), capture_output=True, text=True,
                           check=True)
        return tuple(int(v) for v in r.stdout.split())
    return run


@pytest.mark.parametrize("wgrad,case", [(False, c) for c in BLOCK128] + [(True, c) for c in WGRAD])
def test_sizes_take_their_forms(form, wgrad, case):
    M, N, K, G, kind, fast, exact, walks = case
    assert form(wgrad, True, kind != "none", M, N, K, G, CUS) == fast
    assert form(wgrad, False, kind != "none", M, N, K, G, CUS) == exact
    if walks:
        for _, tile, _ in (fast, exact):
            down = G * -(-N // tile) if wgrad else -(-M // tile)      # at least
            assert down * -(-(K if wgrad else N) // tile) > CUS * (1 if tile == 256 else 2)


def test_every_form_is_taken(form):
    """Sizes of the other tests, and the limits between the forms."""
    few16, few64, two = (16, 0, 0), (64, 0, 0), (0, 128, 2)
    for args, want in (
            ((0, 1, 0, 1, 8192, 8192, 1), few16), ((0, 0, 0, 20, 8192, 8192, 1), few16), ((0, 1, 0, 21, 16, 16, 1), (32, 0, 0)),
            ((0, 1, 0, 64, 8192, 8192, 1), few64), ((0, 1, 0, 65, 8192, 8192, 1), two), ((0, 0, 0, 65, 8192, 8192, 1), (0, 128, 1)),
            ((0, 1, 1, 21, 16, 16, 1), (32, 0, 0)), ((0, 1, 1, 42, 16, 16, 2), two), ((0, 1, 1, 40, 16, 16, 2), few16),
            ((0, 1, 0, 4096, 4096, 4096, 1), (0, 256, 1)), ((0, 1, 0, 4096, 3840, 4096, 1), (0, 128, 1)),
            ((0, 1, 1, 16640, 5120, 8192, 16), (0, 256, 1)), ((0, 1, 1, 4096, 4096, 4096, 16), (0, 128, 1)),
            ((1, 1, 1, 16640, 256, 272, 1), few16), ((1, 0, 1, 16384, 1024, 512, 1), few64),
            ((1, 1, 1, 16384, 1024, 1024, 1), two), ((1, 0, 1, 16384, 1024, 1024, 1), few64),
            ((1, 1, 1, 16640, 8192, 5120, 16), (0, 256, 1)), ((1, 1, 1, 256, 1040, 4096, 4), (0, 128, 1))):
        assert form(*args, CUS) == want, args
