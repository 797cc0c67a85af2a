"""How the block-scaled products count tiles and work items (csrc/fp8.cuh,
csrc/fp8_dev.cuh), on the CPU: the header's own arithmetic, compiled here, for
segment tables whose segments overlap and hold more tiles than an int counts."""
import subprocess

import pytest

from mxfp8_mxfp4_moe_gb300 import build as B

PROGRAM = r"""
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "fp8_dev.cuh"
using namespace kmoe;

#define CHECK(x) if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; }

// segment_prefix's order of additions, by chunks of 32 experts
static std::vector<int> units(const std::vector<long long>& tiles) {
  const int E = static_cast<int>(tiles.size());
  std::vector<int> unit(E + 1, 0);
  int before = 0;
  for (int c = 0; c * 32 < E; ++c) {
    int own = 0;
    for (int e = c * 32; e < E && e < c * 32 + 32; ++e) {
      own += static_cast<int>(tiles[e]);
      unit[e + 1] = add_units(own, before);
    }
    before = add_units(before, own);
  }
  return unit;
}

int main() {
  // every second segment holds all M rows
  for (long long M : {1LL, 1000LL, 1LL << 20, 1LL << 29, 1LL << 30})
    for (int E : {1, 2, 31, 64, 1000, 1024})
      for (int F : {16, 7168, 1 << 20}) {
        const int ft = (F + 255) / 256;
        std::vector<long long> tiles(E);
        long long all = 0;
        for (int e = 0; e < E; ++e) all += tiles[e] = e % 2 == 0 ? (M + 127) / 128 : 0;
        const std::vector<int> unit = units(tiles);
        CHECK(unit[0] == 0);
        for (int e = 0; e < E; ++e) CHECK(unit[e + 1] >= unit[e] && unit[e + 1] <= kMaxUnits);
        CHECK(unit[E] == (all < kMaxUnits ? all : kMaxUnits));
        const int items = static_cast<int>(std::min<long long>(fp8_most_tiles(M, E, 128) * ft, 1 << 30));
        const int total = product_items(ft, unit[E], items);
        CHECK(total <= items && total == std::min<long long>(all * ft, items));
        CHECK(total + 152 > 0);  // the step behind the last item
        for (int w : {0, 1, total / 3, total / 2, total - 2, total - 1}) {
          if (w < 0 || w >= total) continue;
          const int e = segment_of_unit(unit.data(), E, w / ft);
          CHECK(e >= 0 && e < E && unit[e] <= w / ft && w / ft < unit[e + 1]);
          const int nt = unit[e + 1] - unit[e], r = w - unit[e] * ft;  // (no more than w)
          CHECK(nt > 0 && r >= 0 && r / nt < ft && r % nt < tiles[e]);
        }
      }
  // an ascending table keeps all of its items
  for (int M : {1, 127, 1000, 32768})
    for (int E : {1, 3, 64, 1024}) {
      int first = 0, tiles = 0;
      for (int e = 0; e < E; ++e) {  // one row each, and the last the rest
        const int n = e == E - 1 ? M - first : (first < M ? 1 : 0);
        tiles += (n + 127) / 128;
        first += n;
      }
      const int items = static_cast<int>(fp8_most_tiles(M, E, 128) * 5);
      CHECK(product_items(5, tiles, items) == 5 * tiles);
    }
  std::puts("ok");
}
"""


def test_items_of_any_table_are_counted(tmp_path):
    try:
        cc = B.nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")
    src, exe = tmp_path / "items.cu", tmp_path / "items"
    src.write_text(PROGRAM)
    subprocess.run([cc, *B.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", B.CSRC, str(src), "-o", str(exe)],
                   check=True, capture_output=True, text=True, timeout=300)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr
