// The rules of csrc/fp8moe_plan.h, for tests/test_moe_paths.py.  Reads lines
//   0 M N K scale_mode   -> raw, and the tile of the kernel that multiplies codes
//   1 T H I E k scale_mode -> narrow, its workgroups across an expert's columns
//                           and those that there are, the two wide kernels' plans
#include <cstdio>

#include "../blockwise_fp8_linear_amd/csrc/fp8moe_plan.h"

using namespace fp8blk;

int main() {
  int what;
  while (std::scanf("%d", &what) == 1) {
    long long v[6] = {};
    for (int i = 0; i < (what ? 6 : 4); ++i)
      if (std::scanf("%lld", &v[i]) != 1) return 1;
    if (what == 0) {
      const RowsTile t = codes_tile(v[0], v[1]);
      std::printf("%d %d %d %d %d\n", rows_raw(v[0], v[1], v[2], v[3] != 0), t.waves, t.columns, t.tokens, t.slots);
    } else {
      const int T = (int)v[0], H = (int)v[1], I = (int)v[2], E = (int)v[3], k = (int)v[4];
      const WidePlan g = gate_up_plan(T, I, E, k), d = down_plan(T, H, E, k);
      std::printf("%d %d %d %d %d %d %d %d %d\n", few_plan(T, I, E, k, v[5] != 0), few_columns(T, I, E, k), I / 16,
                  g.tiles, g.parts, g.slots, d.tiles, d.parts, d.slots);
    }
  }
  return 0;
}
