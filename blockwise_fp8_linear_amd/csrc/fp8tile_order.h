// Which 128 x 128 tile is which workgroup's: fp8tile_device.h's kernels, their launchers
// and the test of both.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8blk {

// Tile order of the one-pass quantizers.  A tile's scales are 128 four-byte
// values strided through s (one per row) and 128 through sT (one per
// column); the 8 tiles side by side along a row band fill one 32-byte
// sector of s, the 8 above one another one of sT.  Where the shape allows
// (tile_blocked: a multiple of 16 row tiles and of 8 column tiles, whole
// multiples of 8 blocks), the tiles go in blocks of 8 column tiles x 16 row
// tiles, block k to the workgroups k, k + 8, ... mod 8, i.e. to one XCD
// (workgroups are dealt to the 8 XCDs in turn), walked down each column of
// the block: every sector of s and sT is then written by one XCD, whose L2
// merges the pieces before writing the sector back.  Measured on the
// activation shapes: written bytes at the algorithmic count (+11% in row-band
// order, from partial sectors written back from several L2s), and 0-8%
// faster.  Other shapes walk row band by row band.  The codes leave with
// plain stores: non-temporal ones were faster for the quantizer timed alone
// (launch after launch) but slower in a training step, where the GEMMs read
// the codes right after (they no longer found them in the caches) and the
// quantizer itself ran slower too.
constexpr uint32_t kTileBlockCols = 8, kTileBlockRows = 16;

__host__ __device__ inline bool tile_blocked(uint32_t row_tiles, uint32_t col_tiles) {
  return row_tiles % kTileBlockRows == 0 && col_tiles % kTileBlockCols == 0 &&
         (row_tiles / kTileBlockRows) * (col_tiles / kTileBlockCols) % 8 == 0;
}

// Workgroup bid's tile.
__host__ __device__ inline void tile_of(uint32_t bid, uint32_t col_tiles, bool blocked, uint32_t& rt, uint32_t& ct) {
  if (blocked) {
    constexpr uint32_t kPerBlock = kTileBlockCols * kTileBlockRows;
    const uint32_t xcd = bid % 8, j = bid / 8;
    const uint32_t blk = xcd + 8 * (j / kPerBlock), w = j % kPerBlock;
    const uint32_t col_blocks = (col_tiles + kTileBlockCols - 1) / kTileBlockCols;
    rt = (blk / col_blocks) * kTileBlockRows + w % kTileBlockRows;
    ct = (blk % col_blocks) * kTileBlockCols + w / kTileBlockRows;
  } else {
    // consecutive workgroups walk along the rows, so that the ones in flight
    // together read whole rows
    rt = bid / col_tiles;
    ct = bid - rt * col_tiles;
  }
}

// The same order for any shape, with workgroups that find no tile (rt or ct past
// the end): blocks that the shape fills in part, and up to 7 whole ones.  Taken where
// there are kTileSomeBlocks, no more than an eighth of them is empty, so that the XCDs
// have about the same work (20608 rows of 2048 in 22 of 24 blocks: a turn 24.5 us, row
// band by row band 22.1; 16384 of 1536, half of the blocks half as wide: gated backward
// 70 and 61), and a launch of all of them stays below 2^32 threads.  Gated
// backward of 8192 rows of 6144 113 us row band by row band and 103.5, of 65536 of 2048
// 272 and 238; a turn of 69632 rows of 2048 66 and 63.
constexpr uint32_t kTileSomeBlocks = 8, kTileMostBlocks = 1 << 16;
struct TileGrid {
  uint32_t row_tiles, col_tiles;
  bool blocked;
  uint32_t workgroups;
};
inline TileGrid tile_grid(int64_t rows, int64_t cols) {
  TileGrid g{(uint32_t)(rows / 128), (uint32_t)(cols / 128), false, 0};
  const uint32_t col_blocks = (g.col_tiles + kTileBlockCols - 1) / kTileBlockCols;
  const uint32_t blocks = (g.row_tiles + kTileBlockRows - 1) / kTileBlockRows * col_blocks, all = (blocks + 7) / 8 * 8;
  const uint32_t width = col_blocks == 1 ? g.col_tiles : kTileBlockCols;  // all blocks are as narrow, or the last ones
  g.blocked = blocks >= kTileSomeBlocks && blocks <= kTileMostBlocks && g.col_tiles >= kTileBlockCols / 2 &&
              uint64_t(8) * all * kTileBlockRows * width <= uint64_t(9) * g.row_tiles * g.col_tiles;
  g.workgroups = g.blocked ? all * kTileBlockCols * kTileBlockRows : g.row_tiles * g.col_tiles;
  return g;
}

}  // namespace fp8blk
