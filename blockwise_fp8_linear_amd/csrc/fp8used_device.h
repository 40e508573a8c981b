// How many rows of a buffer are in use, read on the device (include/fp8train.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8blk {

// *used within [0, rows], or all rows where it is null.
__device__ __forceinline__ int64_t used_rows(const int32_t* __restrict__ used, int64_t rows) {
  if (!used) return rows;
  const int64_t n = *used;
  return n < 0 ? 0 : n < rows ? n : rows;
}

// The same in tiles of 128 rows, a partial one counted whole.
__device__ __forceinline__ uint32_t used_tiles(const int32_t* __restrict__ used, int64_t rows) {
  return (uint32_t)((used_rows(used, rows) + 127) / 128);
}

}  // namespace fp8blk
