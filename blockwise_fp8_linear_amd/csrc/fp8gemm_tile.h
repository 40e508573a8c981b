// The tiles of the general GEMM (gemm.hip): their shapes, what each keeps in LDS and
// where the scales are in it.
#pragma once

#include <stdint.h>

#include <type_traits>

namespace fp8blk {

// BT_: B stored [R][J] (Dgrad from the weight codes as quantized): the B
// tile is staged as 128 reduction rows of BN bytes and its fragments come
// from LDS transpose reads.
// CHUNK_: reduction blocks whose scales sit in LDS at once.
template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, bool PROMOTE_, bool BROW_, bool BT_ = false,
          int CHUNK_ = 32>
struct Cfg {
  static constexpr int BM = BM_, BN = BN_, CHUNK = CHUNK_;
  static constexpr bool BT = BT_;
  static_assert(!BT_ || (!BROW_ && BN_ == 128), "transposed B: Dgrad's weight-block layout, 128-byte rows");
  static constexpr int WAVES_M = WAVES_M_, WAVES_N = WAVES_N_;
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
  static constexpr int TM = WM / 16, TN = WN / 16;
  static constexpr int THREADS = 64 * WAVES_M * WAVES_N;
  static constexpr bool PROMOTE = PROMOTE_, BROW = BROW_;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  // one staged scale: fp32 for PROMOTE, its E8M0 byte for the scaled MFMA
  using SType = typename std::conditional<PROMOTE_, float, uint8_t>::type;
  static constexpr int SA_BYTES = CHUNK * BM * (int)sizeof(SType);
  static constexpr int SB_BYTES = (BROW ? CHUNK * BN : CHUNK * (BN / 128 > 0 ? BN / 128 : 1)) * (int)sizeof(SType);
  static constexpr int LDS = 2 * STAGE + SA_BYTES + ((SB_BYTES + 15) / 16) * 16;
  static_assert(A_BYTES % (1024 * (THREADS / 64)) == 0 && B_BYTES % (1024 * (THREADS / 64)) == 0,
                "whole KiB of direct loads per wave");
  static_assert(WN <= 128 && 128 % WN == 0, "a wave's columns must sit inside one 128-block");
  // The scales of block kbl of a lane's rows l16, l16 + 16, ... of wave row wm: TM in a
  // row, in [kbl][row % 16][row / 16].  As bytes they are read in words of as many as
  // there are (up to four), each on a multiple of its size, since everything in front of
  // it is a multiple of TM.
  static constexpr uint32_t sa_at(uint32_t kbl, uint32_t l16, uint32_t wm) {
    return kbl * BM + l16 * (BM / 16) + wm * TM;
  }
  static_assert(TM % 4 == 0 || TM == 2, "a lane's scale bytes are whole words or half words");
  using SAWord = typename std::conditional<TM % 4 == 0, uint32_t, uint16_t>::type;
  static constexpr int SA_WORDS = TM / (int)sizeof(SAWord);
};

using PromoteBlock = Cfg<256, 128, 2, 2, true, false>;
using PromoteRow = Cfg<256, 128, 2, 2, true, true>;
using ScaledBlock = Cfg<256, 128, 2, 2, false, false>;
using ScaledRow = Cfg<256, 128, 2, 2, false, true>;
using PromoteBlockBT = Cfg<256, 128, 2, 2, true, false, true>;
using ScaledBlockBT = Cfg<256, 128, 2, 2, false, false, true>;

// Experts' products are many short ones: what a tile takes besides its blocks -- the
// first loads, the scales, the store -- has to be hidden behind another tile.  So the
// tiles are 128 x 128, two workgroups a CU (72 KiB of LDS each), against the dense
// kernel's one of 256 x 128 (both before their store went through LDS: 414 rows of 52
// experts of 896 x 3328, amax / 448, Fprop 80 us and 43, Wgrad 209 and 149; 65536 rows
// of 64 of 2048 x 2048 Dgrad 508 and 444, now 413).
// Where no more than a CU's worth of them are left, 64 x 128, so that more CUs work:
// 512 rows of 2 experts, Dgrad of 4736 x 256, 35 us and 27.
template <bool PROMOTE, bool BROW, bool BT, int BM>
using Expert = Cfg<BM, 128, 2, 2, PROMOTE, BROW, BT, 8>;

}  // namespace fp8blk
