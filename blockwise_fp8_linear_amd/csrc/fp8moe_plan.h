// Host-side rules of the operators declared in include/fp8moe.h: which kernel,
// tiles and launch a size gets.  Plain C++, so that a test can ask which kernels
// its sizes reach.
#pragma once

#include <stdint.h>

namespace fp8blk {

constexpr int kCus = 256;

// ---------------------------------------------------------- one linear's rows

// Up to so many rows the sums are fp32-faithful (FP8_LINEAR_FP32_ROWS).
constexpr int64_t kExactRows = 127;
// Whether one launch quantizes as it multiplies, in tiles of 16 x 16 outputs
// that each quantize their rows again, or a launch of its own does before, into
// the workspace: codes, and from rows_scales_at on their scales.  One launch is
// 2 us less of the GPU and 4 of the host, which a few rows and small products
// do not win back.  us of the GPU, one launch and two: power-of-two scales 48 x
// 12288 x 2048 11.8 and 11.6, 64 rows 13.7 and 12.4; 333 x 512 x 2048 8.1 and
// 9.7, x 1024 10.9 and 10.9; 700 x 1024 x 512 7.3 and 10.5; 64 x 4096 x 4096
// 11.3 and 11.8; 700 x 2048 x 128 7.7 and 9.0, 1500 rows 12.1 and 9.9.  amax /
// 448, whose quotients cost more: 8 x 2048 x 6144 10.8 and 10.2; 200 x 1024 x
// 2048 9.8 and 9.6, 24 x 4096 x 2048 9.1 and 8.5, 333 x 1024 x 2048 17.1 and
// 11.0; 24 x 512 x 4096 11.0 and 8.4; 700 x 1024 x 512 10.1 and 10.6, 100 x 8192
// 11.1 and 10.2; 333 x 2048 x 128 7.4 and 9.4, x 4096 9.9 and 8.9.
inline bool rows_raw(int64_t M, int64_t N, int64_t K, bool fp32_scale) {
  const int64_t tiles = N / 16 * ((M + 15) / 16);
  return fp32_scale ? M <= 8 || (K <= 2048 && tiles <= 4096 && tiles * K <= int64_t(3) << 19)
                    : M <= 48 || (tiles <= 6144 && tiles * K <= int64_t(3) << 20);
}

// A kernel that multiplies codes: waves of a workgroup, its tiles of 16 columns
// and of 16 tokens, and of the wide kernel the slots of its ring (others 0).
struct RowsTile {
  int waves, columns, tokens, slots;
};
constexpr int kWideTiles = 4;  // the wide kernel's tiles of tokens

// Tiles are chosen so that a launch has about one workgroup of eight waves per
// CU: a smaller tile loads the tokens more often, a larger one leaves CUs idle.
// us as a graph node at K 2048 (an empty node takes 2.1), power-of-two scales.
// The smallest of (tiles of columns, of tokens) (1, 1), (2, 1), (2, 2), (4, 2),
// (4, 4) that has at most 256 workgroups: 24 x 4096 (2, 1) 4.1; 64 x 4096 (2, 2)
// 4.9 and (4, 1) 5.1; 128 x 4096 (4, 2) 6.0 and (2, 2) 6.6; 256 x 4096 (4, 4)
// 8.2 and (4, 2) 9.9.  Where all have more, smaller workgroups of (3, 2): 64 x
// 12288 10.4 and (4, 4) 11.4; 96 x 12288 12.0 and (4, 2) 13.3.  Above kExactRows
// rows, and with 200 workgroups of it, the wide kernel: 512 x 4096 12.8 and
// 16.6, 1467 x 2560 (K 6400) 44 and 73; with fewer, 333 x 2048 11.4 and 8.3.
// Its slots: four while each CU has one workgroup, 1000 x 2048 (K 6400) 34.0 and
// with two 37.4; beyond, two, so that two fit (1467 x 2560: 45.0, three 48.6).
inline RowsTile codes_tile(int64_t M, int64_t N) {
  const int64_t tiles = N / 16, m1 = (M + 15) / 16, m2 = (M + 31) / 32, m4 = (M + 63) / 64;
  const int64_t wide = tiles / 8 * m4;
  if (M > kExactRows && wide >= 200) return {8, 8, kWideTiles, wide <= kCus ? 4 : 2};
  if (tiles * m1 <= kCus) return {16, 1, 1, 0};
  if (tiles / 2 * m1 <= kCus) return {8, 2, 1, 0};
  if (tiles / 2 * m2 <= kCus) return {8, 2, 2, 0};
  if (tiles / 4 * m2 <= kCus) return {8, 4, 2, 0};
  if (tiles / 4 * m4 <= kCus && M > 64) return {8, 4, 4, 0};
  return tiles % 3 == 0 ? RowsTile{4, 3, 2, 0} : RowsTile{4, 4, 2, 0};
}

// ------------------------------------------------------------- the mixture --

constexpr int kFew = 16;  // tokens of the narrow kernels, at most

// How many experts the tokens reach, if each is as likely as the next.
inline double experts_reached(int T, int E, int k) {
  double missed = 1.0;
  for (int t = 0; t < T; ++t) missed *= 1.0 - (double)k / E;
  return E * (1.0 - missed);
}

// Whether the narrow gate/up kernel takes a call.  With fewer than 64 workgroups
// the wide one leaves too many CUs idle (14 tokens, 9 experts of 1664 x 256, 88
// workgroups: narrow 43 us, wide 24).  Up to 8 tokens the narrow one is as fast
// at any number (8 tokens, 128 experts of 768: 60 us, wide 67; 16 tokens, 64
// experts of 1024: 112 and 93), but it quantizes x again for each 16 columns,
// which amax / 448 scales make dearer (8 tokens 73 us, wide 64).
inline bool few_plan(int T, int I, int E, int k, bool fp32_scale) {
  return T <= (fp32_scale ? 4 : 8) || (T <= kFew && experts_reached(T, E, k) * (I / 128) < 64);
}

// Workgroups of the narrow gate/up that share an expert's columns, 16 each: about
// 2304 of them in all at most; beyond, each takes several columns, so that its
// start counts less (4 tokens, 18 experts of 1408 x 256: 44 us without, 35 with;
// at 768 as well, but 8 tokens, 51 experts of 768 x 2048 60 and 62).
inline int few_columns(int T, int I, int E, int k) {
  constexpr int grid = 2304;
  const int most = T * k < E ? T * k : E, across = I / 16;  // experts reached, at most
  return across * most > grid ? (grid + most - 1) / most : across;
}

// How a wide kernel's workgroups take the rows of an expert: `tiles` of 16 at a
// time, `parts` workgroups in turn.
struct RowSplit {
  int tiles, parts;
};
// `columns`: workgroups of an expert's columns.  Tiles for about twice as many
// rows as an expert has on average, since some have more (64 experts, k 8; one,
// two, four tiles at most: 64 tokens 90, 97, - us; 100 tokens 119, 107, 107; 200
// tokens -, 115, 104).  Where the columns leave CUs idle, fewer tiles in more
// workgroups, which read the weights again, from a cache (256 tokens, 4 experts
// of 512 x 1024: 80 us without, 26 with; 512 tokens, 64 of 256 x 2048 89 and 75).
inline RowSplit row_split(int T, int E, int k, int columns) {
  const int mean = T * k / E, rows = 2 * mean < T ? 2 * mean : T;
  const int most = mean <= 8 ? 1 : mean <= 20 ? 2 : 4, fit = kCus / (columns * E);
  for (int tiles = 1;; tiles *= 2) {
    const int parts = (rows + 16 * tiles - 1) / (16 * tiles);
    if (parts <= fit) return RowSplit{tiles, parts < 1 ? 1 : parts};
    if (tiles == most) return RowSplit{tiles, fit < 1 ? 1 : fit};
  }
}

// A wide kernel: its row split and the slots of its ring, as many as fit while
// each CU has one workgroup (17 tokens, 8 experts of 6144: 86 us, with two slots
// 106); beyond, two (256 tokens, 64 experts of 1024, three slots of four tiles:
// 127 us, two 120).
struct WidePlan {
  int tiles, parts, slots;
};
constexpr int gate_up_slots(int tiles) { return tiles == 1 ? 4 : 3; }
constexpr int down_slots(int tiles) { return tiles == 1 ? 3 : 4; }
// Tiles of 16 columns that a wave of the down projection owns.
constexpr int down_columns(int tiles) { return tiles == 1 ? 2 : 1; }

inline WidePlan gate_up_plan(int T, int I, int E, int k) {
  const RowSplit s = T <= kFew ? RowSplit{1, 1} : row_split(T, E, k, I / 128);
  return {s.tiles, s.parts, (int64_t)(I / 128) * E * s.parts > kCus ? 2 : gate_up_slots(s.tiles)};
}
inline WidePlan down_plan(int T, int H, int E, int k) {
  const RowSplit s = row_split(T, E, k, H / 128);
  const int across = 128 * down_columns(s.tiles);
  return {s.tiles, s.parts, (int64_t)((H + across - 1) / across) * E * s.parts > kCus ? 2 : down_slots(s.tiles)};
}

}  // namespace fp8blk
