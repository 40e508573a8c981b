// The order of tiles of csrc/fp8tile_order.h, for tests/test_tile_order.py.  Reads lines "row_tiles col_tiles", prints
// whether they go in blocks, the workgroups, the tiles taken once and the tiles taken more often.
#include <algorithm>
#include <cstdio>
#include <vector>

#include "../blockwise_fp8_linear_amd/csrc/fp8tile_order.h"

using namespace fp8blk;

int main() {
  long long rows, cols;
  while (std::scanf("%lld %lld", &rows, &cols) == 2) {
    const TileGrid g = tile_grid(128 * rows, 128 * cols);
    std::vector<int> taken(rows * cols);
    for (uint32_t w = 0; w < g.workgroups; ++w) {
      uint32_t rt, ct;
      tile_of(w, g.col_tiles, g.blocked, rt, ct);
      if (rt >= g.row_tiles || ct >= g.col_tiles) continue;
      ++taken[(size_t)rt * g.col_tiles + ct];
    }
    std::printf("%d %u %lld %lld\n", (int)g.blocked, g.workgroups, (long long)std::count(taken.begin(), taken.end(), 1),
                (long long)std::count_if(taken.begin(), taken.end(), [](int n) { return n > 1; }));
  }
  return 0;
}
