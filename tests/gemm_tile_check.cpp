// Where the tiles of csrc/fp8gemm_tile.h keep their scale bytes, for tests/test_gemm_tile.py: prints, for each
// configuration of the scaled MFMA, the lanes' reads that are off their alignment, that pass the end of the scales, and
// that find another row's byte.
#include <cstdio>

#include "../blockwise_fp8_linear_amd/csrc/fp8gemm_tile.h"

using namespace fp8blk;

template <class C>
void check(const char* name) {
  using Word = typename C::SAWord;
  const int word = (int)sizeof(Word), bytes = word * C::SA_WORDS;
  int off = 0, past = 0, other = 0;
  for (uint32_t kbl = 0; kbl < (uint32_t)C::CHUNK; ++kbl)
    for (uint32_t wm = 0; wm < (uint32_t)C::WAVES_M; ++wm)
      for (uint32_t l16 = 0; l16 < 16; ++l16) {
        const uint32_t at = C::sa_at(kbl, l16, wm);
        off += (2 * C::STAGE + at) % word != 0;
        past += (int)at + bytes > C::SA_BYTES;
        for (uint32_t ms = 0; ms < (uint32_t)C::TM; ++ms) {
          const uint32_t i = wm * C::WM + ms * 16 + l16;  // the row, and where its scale was staged
          other += at + ms != kbl * C::BM + (i & 15) * (C::BM / 16) + (i >> 4);
        }
      }
  std::printf("%s %d %d %d\n", name, off, past, other + (bytes != C::TM));
}

int main() {
  check<ScaledBlock>("block");
  check<ScaledRow>("row");
  check<ScaledBlockBT>("block_bt");
  check<Expert<false, false, false, 128>>("expert_128");
  check<Expert<false, false, true, 128>>("expert_128_bt");
  check<Expert<false, true, false, 128>>("expert_128_row");
  check<Expert<false, false, false, 64>>("expert_64");
  check<Expert<false, false, true, 64>>("expert_64_bt");
  return 0;
}
