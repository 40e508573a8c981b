// The rules of csrc/fp8train_launch.h, for tests/test_train_paths.py.  Reads lines
//   0|1|2 (Fprop, Dgrad, Wgrad) R N K E scale_mode misaligned -> the tiles (0 large, 1 small, 2 few), tiles a workgroup
//   3 T H R k both -> whether the gather goes in the order of tokens
#include <cstdio>

#include "../blockwise_fp8_linear_amd/csrc/fp8train_launch.h"

using namespace fp8blk;

int main() {
  int what;
  alignas(16) static float scales[8];
  while (std::scanf("%d", &what) == 1) {
    long long v[6] = {};
    for (int i = 0; i < (what == 3 ? 5 : 6); ++i)
      if (std::scanf("%lld", &v[i]) != 1) return 1;
    if (what == 3) {
      std::printf("%d\n", (int)gather_ordered(v[0], v[1], v[2], (int)v[3], v[4] != 0));
      continue;
    }
    GroupedArgs a{};
    a.E = v[3];
    a.g.sa = a.g.sb = scales + (v[5] ? 1 : 0);
    const GemmAlgo algo = v[4] ? GemmAlgo::Promote : GemmAlgo::ScaledMfma;
    if (what == 2) {
      a.g.I = v[1];
      a.g.J = v[2];
      a.g.R = v[0];
      a.g.bmode = BScale::Row;
      std::printf("%d %lld\n", (int)grouped_wgrad_tiles(a, algo), (long long)wgrad_plan(a).each);
    } else {
      a.g.I = v[0];
      a.g.J = what ? v[2] : v[1];
      a.g.R = what ? v[1] : v[2];
      a.g.bmode = BScale::Block;
      a.g.bt = what == 1;
      std::printf("%d 1\n", (int)grouped_rows_tiles(a, algo));
    }
  }
  return 0;
}
