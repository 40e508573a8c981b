// Internal launch entry points of the operators declared in include/fp8moe.h.
// Arguments are validated by the C ABI layer (api_moe.cpp) before any of these
// is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fp8blk {

// What an output element is stored as (include/fp8blk.h's fp8blk_out_dtype).
struct RowsOut {
  void* y;          // dense rows
  bool f32;         // fp32 instead of bf16
  bool accumulate;  // fp32 only: y += result
};

// y = x W^T for M rows; x is quantized on the way (fp32_scale: amax / 448).
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
inline size_t rows_scales_at(int64_t M, int64_t K) { return ((size_t)(M * K) + 255) & ~size_t(255); }
inline size_t rows_workspace_bytes(int64_t M, int64_t N, int64_t K, bool fp32_scale) {
  return M == 0 || rows_raw(M, N, K, fp32_scale)
             ? 0
             : rows_scales_at(M, K) + (((size_t)(M * (K / 128)) * sizeof(float) + 255) & ~size_t(255));
}
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
