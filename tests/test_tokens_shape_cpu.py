"""Which form of its kernels the layer for a few tokens takes, compiled from the library's own rule: every form that the
library holds is reached by sizes that a GPU test runs."""
import os
import subprocess

import pytest

from test_gpu_24_moe_tokens import CASES
from test_gpu_28_tokens_shapes import CHOICES, SHAPES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "ep_tokens_shape.h"
using namespace epk;
int main(int, char** v) {
    const TokensShape f = tokens_shape({atoi(v[1]), atoi(v[2]), atoi(v[3]), atoi(v[4]), atoi(v[5]), atoi(v[6]), atoi(v[7])});
    printf("%d %d %d %d %d %lld %lld\n", f.route_here, f.many, f.up_tiles, f.up_groups, f.down_tiles, (long long)f.up_items,
           (long long)f.down_items);
}
"""


@pytest.fixture(scope="module")
def shape(tmp_path_factory):
    d = tmp_path_factory.mktemp("shape")
    (d / "shape.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-I", os.path.join(ROOT, "combine_ep_layout_amd", "csrc"), "-o",
                    str(d / "shape"), str(d / "shape.cpp")], check=True)

    def f(T, E, K, H, I, four, cu=256):
        out = subprocess.run([str(d / "shape"), *map(str, (T, K, E, H, I, 2 if four else 1, cu))], check=True,
                             capture_output=True, text=True).stdout
        return tuple(map(int, out.split()))
    return f


def up_and_down(f):
    route_here, many, tiles, groups, down = f[:5]
    return (bool(many), tiles, groups), (bool(many), down)


def test_the_gpu_tests_reach_every_form(shape):
    """With a choice given: the gate and up products' forms for up to 16 tokens and for more, and the down product's."""
    for four in (False, True):
        ups, downs = set(), set()
        for T, E, K, H, I, _ in [*CASES, *SHAPES]:
            if not four or (H % 32 == 0 and I % 32 == 0):
                up, down = up_and_down(shape(T, E, K, H, I, four))
                ups.add(up)
                downs.add(down)
        forms = [(1, 1), (2, 1), (2, 2)] if four else [(1, 1)]
        assert ups == {(many, *form) for many in (False, True) for form in forms}, four
        assert downs == {(many, tiles) for many in (False, True) for tiles in (1, 2)}, four
        # and the gate and up products' forms that make the choice themselves
        made = {f[2:4] for f in (shape(T, E, K, H, I, four) for T, E, K, H, I, _ in CHOICES) if f[0]}
        assert made == set(forms), four


def test_the_cases_that_name_a_form(shape):
    for T, E, K, H, I, (up, down) in SHAPES:
        if H % 32 == 0 and I % 32 == 0:
            assert shape(T, E, K, H, I, True)[2:5] == (*up, down), (T, E, K, H, I)
        assert shape(T, E, K, H, I, False)[4] == down, (T, E, K, H, I)


@pytest.mark.parametrize("sizes,four,want", [
    # one token and batches of a large layer
    ((1, 64, 8, 7168, 2048), False, (1, 0, 1, 1, 2, 1024, 224)),
    ((1, 64, 8, 7168, 2048), True, (1, 0, 2, 2, 2, 256, 224)),
    ((32, 64, 8, 7168, 2048), False, (0, 1, 1, 1, 2, 8192, 224)),
    ((64, 64, 8, 7168, 2048), True, (0, 1, 2, 2, 2, 2048, 224)),
    # small and odd layers
    ((4, 8, 2, 256, 512), False, (1, 0, 1, 1, 1, 256, 16)),
    ((13, 24, 3, 2056, 1000), False, (0, 0, 1, 1, 1, 1512, 129)),
    ((7, 24, 3, 2080, 992), True, (1, 0, 2, 1, 1, 651, 130)),
    # past eight tokens or 256 experts the choice has its own launch
    ((8, 256, 8, 64, 64), True, (1, 0, 1, 1, 1, 256, 4)),
    ((8, 257, 8, 64, 64), False, (0, 0, 1, 1, 1, 256, 4)),
    ((9, 256, 8, 64, 64), False, (0, 0, 1, 1, 1, 288, 4)),
])
def test_shapes(shape, sizes, four, want):
    assert shape(*sizes, four) == want


def test_limits(shape):
    """Counts of the largest sizes, and of one compute unit."""
    assert shape(64, 1024, 32, 65536, 8192, False)[5:] == (1024 * 512, 2048)
    assert shape(64, 1024, 32, 8192, 65536, True)[5:] == (1024 * 1024, 256)
    assert shape(1, 1, 1, 32, 32, True, 1)[5] >= 1
