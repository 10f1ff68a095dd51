"""Which tiles each product of the orthogonalisation takes, compiled from the library's own rule: the sizes that the GPU
tests name for the widest tiles must reach them, with tiles that the matrices fill only in part."""
import os
import subprocess

import pytest

from test_gpu_30_muon_shapes import WIDE

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "ep_muon_shape.h"
using namespace epk;
// v: compute units, then batch, rows and columns of each tensor.  A line for each product: its name and the matrices
// of each tensor that go to small, middle and wide tiles.
int main(int n, char** v) {
    const char* name[] = {"gram", "poly", "next", "last", "last tall"};
    for (int op = kGram; op <= kLastTall; ++op) {
        MuonSizes s[kMuonProblems];
        int count = 0;
        for (int i = 2; i + 2 < n; i += 3) {
            const int batch = atoi(v[i]), rows = atoi(v[i + 1]), cols = atoi(v[i + 2]);
            if (op >= kLast && (rows > cols) != (op == kLastTall)) continue;
            s[count++] = {rows < cols ? rows : cols, ((rows < cols ? cols : rows) + 7) / 8 * 8, batch};
        }
        if (!count) continue;
        const MuonShape f = muon_shape(op, count, s, atoi(v[1]));
        printf("%s:", name[op]);
        for (int i = 0; i < count; ++i)
            printf(" %d/%d/%d", f.small ? s[i].mats : 0, f.small ? 0 : s[i].mats - f.wide_mats[i], f.wide_mats[i]);
        printf("\n");
    }
}
"""


# v: bytes of the workspace, of a matrix, m, ld_n, partial sums of a matrix.  Matrices that a launch takes, filled by tensors
# of at most 2^20.
FIT = r"""
#include <cstdio>
#include <cstdlib>
#include "ep_muon_shape.h"
using namespace epk;
int main(int, char** v) {
    const long long bytes = atoll(v[1]), each = atoll(v[2]), blocks_each = muon_blocks_of(atoi(v[3]), atoi(v[4]), atoi(v[5]));
    long long all = 0;
    for (int i = 0; i < kMuonProblems; ++i) {
        const long long fit = muon_fit(bytes - all * each, each, all * blocks_each, blocks_each);
        all += fit < 1 << 20 ? fit : 1 << 20;
    }
    printf("%lld\n", all);
}
"""


def compiled(tmp_path_factory, text):
    d = tmp_path_factory.mktemp("shape")
    (d / "shape.cpp").write_text(text)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-I", os.path.join(ROOT, "combine_ep_layout_amd", "csrc"), "-o",
                    str(d / "shape"), str(d / "shape.cpp")], check=True)
    return str(d / "shape")


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    """{product: [(small, middle, wide) matrices of each tensor]}."""
    program = compiled(tmp_path_factory, PROGRAM)

    def f(*tensors, cu=256):
        out = subprocess.run([program, str(cu), *(str(n) for t in tensors for n in t)], check=True, capture_output=True,
                             text=True).stdout
        return {line.split(":")[0]: [tuple(map(int, t.split("/"))) for t in line.split(":")[1].split()]
                for line in out.splitlines()}
    return f


def test_the_widest_tiles_in_every_product(tiles):
    """Of matrices that end inside a tile of 256, inside a step of 64 and off the multiples of 8."""
    last = set()
    for shape in WIDE:
        m, n = sorted(shape[1:])
        assert m % 256 and n % 256 and m % 64 and n % 64 and m % 8 and n % 8
        got = tiles(shape)
        assert len(got) == 4
        for product, ((small, middle, wide),) in got.items():
            assert small == 0 and wide > 0 and middle + wide == shape[0], (shape, product)
        last |= set(got) & {"last", "last tall"}
    assert last == {"last", "last tall"}


def test_some_matrices_of_a_batch_in_middle_tiles(tiles):
    """Whole rounds of wide tiles and a rest, both in one product, are among the same sizes."""
    assert any(middle > 0 and wide > 0 for shape in WIDE for ((_, middle, wide),) in tiles(shape).values())


@pytest.mark.parametrize("tensors,want", [
    # the matrices of eight experts: gate and up, down
    ([(16, 2048, 7168)], {"gram": [(0, 2, 14)], "poly": [(0, 2, 14)], "next": [(0, 0, 16)], "last": [(0, 0, 16)]}),
    ([(8, 7168, 2048)], {"gram": [(0, 1, 7)], "poly": [(0, 1, 7)], "next": [(0, 0, 8)], "last tall": [(0, 0, 8)]}),
    # small and middle matrices
    ([(16, 512, 256)], {"gram": [(16, 0, 0)], "poly": [(16, 0, 0)], "next": [(16, 0, 0)], "last tall": [(16, 0, 0)]}),
    ([(6, 777, 1001)], {"gram": [(0, 6, 0)], "poly": [(0, 6, 0)], "next": [(0, 6, 0)], "last": [(0, 6, 0)]}),
    # the rest takes one tensor whole and a part of another
    ([(86, 768, 800), (2, 530, 520)], {"gram": [(0, 1, 85), (0, 2, 0)], "poly": [(0, 1, 85), (0, 2, 0)]}),
])
def test_tiles(tiles, tensors, want):
    got = tiles(*tensors)
    assert {k: got[k] for k in want} == want, got


def test_one_compute_unit_and_no_matrices(tiles):
    assert tiles((1, 1, 1), cu=1)["gram"]
    assert tiles((0, 64, 64))["gram"] == [(0, 0, 0)]


@pytest.fixture(scope="module")
def fit(tmp_path_factory):
    program = compiled(tmp_path_factory, FIT)
    return lambda *v: int(subprocess.run([program, *map(str, v)], check=True, capture_output=True, text=True).stdout)


@pytest.mark.parametrize("bytes_", [4 << 30, 250 << 30])
@pytest.mark.parametrize("rows,cols", [(1, 1), (2, 4), (6, 8), (1, 9000), (64, 64), (128, 128), (300, 500), (65536, 8192)])
def test_threads_of_a_launch(fit, rows, cols, bytes_):
    """However many tiny matrices go through at once, a launch's threads, 256 a workgroup, are counted in 32 bits."""
    m, n = sorted((rows, cols))
    up8 = lambda v: (v + 7) // 8 * 8
    chunks = (m * n + 8191) // 8192
    partials = (chunks + 1) // 2 * 2 if chunks < 256 else 256
    each = 6 * m * up8(n) + 4 * m * up8(m) + 8 * partials
    many = fit(bytes_, each, m, up8(n), partials)
    assert many >= 1
    # the partial sums' launch has a workgroup each, the split at most one for 512 pieces of 8 values
    assert many * partials * 256 < 2 ** 32
    assert many * ((m * up8(n) // 8 + 511) // 512) * 256 < 2 ** 32
