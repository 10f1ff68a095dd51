"""Which tile shape each product of the feed-forward takes, compiled from the library's own rule: the sizes that the GPU
tests name for a shape must reach it."""
import os
import subprocess

import pytest

from test_gpu_21_ffn_edges import WIDE

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "ep_ffn_shape.h"
using namespace epk;
int main(int, char** v) {
    const int T = atoi(v[1]), K = atoi(v[2]), E = atoi(v[3]), H = atoi(v[4]), I = atoi(v[5]), cu = atoi(v[6]);
    const long long slots = (long long)T * K;
    const char* name[] = {"wide", "middle", "low", "small", "few"};
    const FfnSizes up{E, slots, 0, I, cu}, down{E, slots, 0, H, cu}, gate_up{E, slots, 2 * I, H, cu}, wd{E, slots, H, I, cu};
    printf("%s %s %s ", name[ffn_rows_shape(kUp, up)], name[ffn_rows_shape(kDown, down)], name[ffn_rows_shape(kActGrad, up)]);
    if (ffn_after_in_one(down, gate_up, wd)) puts("one");
    else printf("%s %s %s\n", name[ffn_rows_shape(kRowGrad, down)], name[ffn_weight_grad_shape(gate_up)], name[ffn_weight_grad_shape(wd)]);
}
"""


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    d = tmp_path_factory.mktemp("shape")
    (d / "shape.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-I", os.path.join(ROOT, "combine_ep_layout_amd", "csrc"), "-o",
                    str(d / "shape"), str(d / "shape.cpp")], check=True)

    def f(T, K, E, H, I, cu=256):
        return subprocess.run([str(d / "shape"), *map(str, (T, K, E, H, I, cu))], check=True, capture_output=True,
                              text=True).stdout.split()
    return f


def test_the_widest_shape_in_every_product(shapes):
    for T, K, E, _, H, I, _ in WIDE:
        assert shapes(T, K, E, H, I) == ["wide"] * 6, (T, K, E, H, I)


@pytest.mark.parametrize("sizes,want", [
    # one token; a decoding batch; prompts and training batches
    ((1, 8, 64, 7168, 2048), ["few"] * 4 + ["wide"] * 2),
    ((256, 8, 64, 7168, 2048), ["low"] * 4 + ["wide"] * 2),
    ((16384, 8, 256, 7168, 2048), ["wide"] * 6),
    ((8192, 8, 32, 7168, 2048), ["wide"] * 6),
    # a gradient of the activation of three column tiles: 303 wide tiles are less than two rounds
    ((2400, 4, 64, 1288, 648), ["wide", "wide", "middle", "wide", "wide", "wide"]),
    ((300, 1, 1, 520, 264), ["middle"] * 6),
    # less than a round of tiles: the last three products in one launch, from 17 rows an expert to 48
    ((128, 2, 8, 256, 512), ["small"] * 3 + ["one"]),
    ((136, 1, 8, 256, 512), ["small"] * 3 + ["one"]),
    ((128, 1, 8, 256, 512), ["few"] * 4 + ["middle"] * 2),
    ((385, 1, 8, 256, 512), ["middle"] * 6),
])
def test_shapes(shapes, sizes, want):
    assert shapes(*sizes) == want


def test_one_compute_unit_and_no_rows(shapes):
    assert shapes(0, 1, 4, 64, 32)[:4] == ["few"] * 4
    assert shapes(1, 1, 1, 8, 8, 1)
    assert shapes(1 << 19, 32, 1, 65536, 8192) == ["wide"] * 6          # 64-bit counts
