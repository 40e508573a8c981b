// Internal launch entry points of the operators declared in include/fp8moe.h.
// Arguments are validated by the C ABI layer (api_moe.cpp) before any of these
// is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "fp8moe_plan.h"

namespace fp8blk {

// What an output element is stored as (include/fp8blk.h's fp8blk_out_dtype).
struct RowsOut {
  void* y;          // dense rows
  bool f32;         // fp32 instead of bf16
  bool accumulate;  // fp32 only: y += result
};

inline size_t rows_scales_at(int64_t M, int64_t K) { return ((size_t)(M * K) + 255) & ~size_t(255); }
inline size_t rows_workspace_bytes(int64_t M, int64_t N, int64_t K, bool fp32_scale) {
  return M == 0 || rows_raw(M, N, K, fp32_scale)
             ? 0
             : rows_scales_at(M, K) + (((size_t)(M * (K / 128)) * sizeof(float) + 255) & ~size_t(255));
}
// y = x W^T for M rows; x is quantized on the way (fp32_scale: amax / 448).
hipError_t launch_linear_rows(int64_t M, int64_t N, int64_t K, const uint16_t* x, int64_t ld_x, const uint8_t* qw,
                              const float* sw, RowsOut out, bool fp32_scale, void* ws, hipStream_t stream);

// f32: the logits' (and dlogits') type is fp32 instead of bf16.
hipError_t launch_moe_route(int64_t T, int E, int k, const void* logits, bool f32, int64_t ld, bool renorm,
                            int32_t* ids, float* weights, hipStream_t stream);
hipError_t launch_moe_route_backward(int64_t T, int E, int k, const void* logits, bool f32, int64_t ld,
                                     const int32_t* ids, const float* dweights, bool renorm, void* dlogits,
                                     int64_t ld_d, hipStream_t stream);

// One call of the experts, or of the whole layer where wr is not null.
struct MoeArgs {
  int T, H, I, E, k;
  const uint16_t* x;
  int64_t ld_x;
  const uint16_t* wr;  // [E][H], or null: ids and weights are given
  bool renorm;
  int32_t* ids;        // [T][k]; read, or written first where wr is not null
  float* weights;
  const uint8_t *qw1, *qw2;
  const float *sw1, *sw2;
  RowsOut out;
  bool fp32_scale;
  void* ws;
};

// Where the pieces of a call's workspace start; ids and weights are used only
// where the caller of the layer does not take them.
struct MoeWorkspace {
  size_t logits, ids, weights, qx, sx, h, sh, partial, bytes;
};
MoeWorkspace moe_workspace(int64_t T, int64_t H, int64_t I, int64_t E, int k);

hipError_t launch_moe(const MoeArgs& a, hipStream_t stream);

}  // namespace fp8blk
