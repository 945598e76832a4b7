"""The tiles that the orthogonalised updates' products take, on the host: every
side that the GPU tests mean to reach is reached."""
import os
import shutil
import subprocess

import pytest

from tests.orthogonal_tiles import TILES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "orthogonal_tiles.hpp"
using namespace sparcml;
int main(int, char** v) {
  const uint32_t rows = atoi(v[1]), cols = atoi(v[2]), count = atoi(v[3]);
  const uint32_t m = up(rows < cols ? rows : cols, kPad), n = up(rows < cols ? cols : rows, kPad);
  for (int sym = 1; sym >= 0; --sym) {
    const auto tiles = [&](uint32_t side) { return (uint64_t)count * tiles_by(m, n, sym, side); };
    printf("%u\n", tile_side(tiles(64), tiles(128), tiles(256)));
  }
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("tiles")
    (d / "tiles.cpp").write_text(PROGRAM)
    subprocess.check_call([cxx, "-std=c++17", "-Wall", "-Werror", "-I",
                           os.path.join(ROOT, "sparse_gradient_reduction_amd", "csrc"), str(d / "tiles.cpp"), "-o",
                           str(d / "tiles")])
    return str(d / "tiles")


@pytest.mark.parametrize("shape,count,square,move", TILES)
def test_sides(program, shape, count, square, move):
    for rows, cols in (shape, shape[::-1]):
        got = subprocess.check_output([program, str(rows), str(cols), str(count)], text=True).split()
        assert [int(v) for v in got] == [square, move]


def test_every_side_is_covered():
    assert {t[2] for t in TILES} == {t[3] for t in TILES} == {64, 128, 256}
