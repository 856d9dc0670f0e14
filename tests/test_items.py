"""Work items of the large tiles: the arithmetic of csrc/items.h, built for the host."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_mixture_experts_04_amd", "csrc")

# The items of one group of `rows` rows behind `before` row tiles of other groups,
# in row tiles of up to mt rows and n_tiles column tiles: 0 where they cover every
# row of every column tile once, otherwise what is wrong.
WALK = r"""
#include <cstddef>
#include <vector>
#include "items.h"
extern "C" int walk(int rows, int mt, int n_tiles, int before, bool balanced) {
  const int tiles = static_cast<int>((static_cast<long long>(rows) + mt - 1) / mt);
  const int ts[3] = {0, before, before + tiles};
  const int high = balanced ? moe::balanced_rows(rows, tiles) : mt;
  if (high <= 0 || high > mt || (balanced && high % 32 != 0)) return 1;
  std::vector<bool> seen(static_cast<size_t>(tiles) * n_tiles);
  std::vector<long long> covered(n_tiles);
  const long long first = static_cast<long long>(before) * n_tiles;
  for (long long it = 0; it < static_cast<long long>(tiles) * n_tiles; ++it) {
    const moe::Item item = moe::place_item(first + it, ts, 1, n_tiles, mt, rows, balanced);
    if (item.g != 1 || item.grows != rows) return 2;
    if (item.rows <= 0 || item.rows > high) return 3;
    if (item.m0 < 0 || item.m0 % high != 0 || item.m0 > rows - item.rows) return 4;
    if (item.n < 0 || item.n >= n_tiles) return 5;
    const size_t at = static_cast<size_t>(item.m0 / high) * n_tiles + item.n;
    if (seen[at]) return 6;
    seen[at] = true;
    covered[item.n] += item.rows;
  }
  for (long long c : covered)
    if (c != rows) return 7;
  return 0;
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("items")
    src, so = tmp / "walk.cpp", tmp / "walk.so"
    src.write_text(WALK)
    subprocess.run(["g++", "-std=c++17", "-O2", "-fwrapv", "-shared", "-fPIC", f"-I{CSRC}",
                    str(src), "-o", str(so)], check=True)
    fn = ctypes.CDLL(str(so)).walk
    fn.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_bool]
    return fn


@pytest.mark.parametrize("balanced", [True, False])
@pytest.mark.parametrize("mt", [128, 256])
def test_items_cover_every_row_once(walk, mt, balanced):
    for rows in (*range(1, 4 * mt + 2), 9 * mt - 1, 9 * mt + 33, 100 * mt + 1):
        for n_tiles, before in ((1, 0), (3, 7)):
            assert walk(rows, mt, n_tiles, before, balanced) == 0, (rows, n_tiles)


@pytest.mark.parametrize("mt", [128, 256])
@pytest.mark.parametrize("rows", [1717986900, 1718000000, 1908874300, 1910000000, 1920000000,
                                  2 ** 31 - 1024])
def test_items_up_to_the_row_limit(walk, rows, mt):
    """As many rows as moe_gemm_int8 takes (their operands fit the memory at one
    column): the sum of the rows and of a tile for each passes 32 bits."""
    assert walk(rows, mt, 1, 0, True) == 0
