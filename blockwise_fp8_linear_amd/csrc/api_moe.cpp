// C ABI of libfp8blk, include/fp8moe.h: argument validation and dispatch.
#include "../../include/fp8moe.h"

#include <hip/hip_runtime.h>

#include "fp8blk_host.h"
#include "fp8blk_launch.h"
#include "fp8blk_plan.h"
#include "fp8moe_launch.h"

using namespace fp8blk;

namespace {

// The kernels hold byte offsets from a wave's base in 31 bits: of a row among 16
// of x, among 64 of its codes, among all T k rows of h.
constexpr int64_t kMaxStride = int64_t(1) << 26;

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

static_assert(kExactRows == FP8_LINEAR_FP32_ROWS, "the header's promise");

// The rows that the GEMMs of fp8blk.h take: none where the kernels for any
// number of rows are faster, else the multiples of 128.  us of the GPU, with the
// GEMM and without:
//   the block-scaled GEMM, whose 256x256 tiles leave many CUs idle below.  K
//   2048, 1536 x 4096 33.3 and 31.9, 2048 x 4096 32.9 and 35.5; where rows
//   beyond a multiple of 128 need launches of their own, 2000 x 4096 41.4 and
//   36.7, 2500 x 4096 41.4 and 42.9;
//   the general one (amax / 448 scales, and reductions that the other does not
//   take), from memory rather than a cache: four sets of operands in turn.
//   amax / 448, K 2048, 768 x 12288 61 and 42, 3000 x 9216 130 and 99, 4096 x
//   7680 129 and 124, 4000 x 10240 161 and 142, (two sets) 8192 x 8192 235 and
//   325.  Power-of-two scales, K 640, 3000 x 9216 71 and 47, 4000 x 10240 85 and
//   64; K 4224, 3000 x 9216 250 and 193, 4000 x 7680 251 and 242, 4000 x 9216
//   307 and 257, 4000 x 10240 316 and 282, but 4096 x 7680 240 and 252.  Long
//   reductions turn earlier: amax / 448, K 8192, 3000 x 9216 413 and 367, 4096 x
//   6144 313 and 316, 4000 x 7680 414 and 455, 4096 x 8192 405 and 419, 4096 x
//   7680 399 and 474.
int64_t gemm_rows(int64_t M, int64_t N, int64_t K, bool fp32_scale) {
  const bool block_scaled = !fp32_scale && K / kGroup % 4 == 0 && K / kGroup <= kMxMaxKb;
  const int64_t most = (block_scaled ? 7500000 : K <= 6144 ? 40000000 : 28000000) + (M % kGroup ? 2000000 : 0);
  return M <= FP8_LINEAR_FP32_ROWS || M * N <= most ? 0 : M / kGroup * kGroup;
}
// Their codes and scales in the workspace, in front of the other rows'.
size_t codes_bytes(int64_t rows, int64_t K) { return up256((size_t)(rows * K)); }
size_t gemm_bytes(int64_t rows, int64_t K) {
  return rows ? codes_bytes(rows, K) + up256((size_t)(rows * (K / kGroup)) * sizeof(float)) : 0;
}
size_t linear_bytes(int64_t M, int64_t N, int64_t K, bool fp32_scale) {
  const int64_t main = gemm_rows(M, N, K, fp32_scale);
  return gemm_bytes(main, K) + rows_workspace_bytes(M - main, N, K, fp32_scale);
}

bool linear_limits(int64_t M, int64_t N, int64_t K) {
  return N / kGroup < (1 << 20) && K / kGroup < (1 << 18) && M < (int64_t(1) << 27) && prod_le(M, N, kMaxElems) &&
         prod_le(M, K, kMaxElems) && prod_le(N, K, kMaxElems) && prod_lt(M, K / kGroup, int64_t(1) << 31);
}

// Checks shared by the router's two directions.
int check_route(int64_t T, int64_t E, int k, const void* logits, int dtype, int64_t ld, int renormalize) {
  if ((dtype != FP8MOE_BF16 && dtype != FP8MOE_FP32) || (renormalize != 0 && renormalize != 1)) return FP8BLK_ERR_ARG;
  if (!logits) return FP8BLK_ERR_NULL;
  if (T <= 0 || E <= 0 || k <= 0) return FP8BLK_ERR_DIM;
  if (E > FP8MOE_MAX_EXPERTS || k > FP8MOE_MAX_TOPK || k > E || ld < E || T >= (int64_t(1) << 31) ||
      !prod_le(T, ld, kMaxElems))
    return FP8BLK_ERR_ARG;
  const uintptr_t size = dtype == FP8MOE_FP32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % size) return FP8BLK_ERR_ALIGN;
  return FP8BLK_OK;
}

int check_moe_shape(int64_t T, int64_t H, int64_t I, int64_t E, int k) {
  if (T <= 0 || E <= 0 || k <= 0 || !mult128(H) || !mult128(I)) return FP8BLK_ERR_DIM;
  if (T > FP8MOE_MAX_TOKENS || E > FP8MOE_MAX_EXPERTS || k > FP8MOE_MAX_TOPK || k > E || H > (1 << 20) ||
      I > (1 << 20) || !prod_le(H, I, kMaxElems / (2 * FP8MOE_MAX_EXPERTS)) || !prod_lt(T * k, I, int64_t(1) << 31))
    return FP8BLK_ERR_ARG;
  return FP8BLK_OK;
}

int moe(int64_t T, int64_t H, int64_t I, int64_t E, int k, const uint16_t* x, int64_t ld_x, const uint16_t* wr,
        int renormalize, int32_t* ids, float* weights, const uint8_t* qw1, const float* sw1, const uint8_t* qw2,
        const float* sw2, void* y, int out_dtype, int scale_mode, void* workspace, size_t ws_bytes,
        hipStream_t stream) {
  if (!valid_scale_mode(scale_mode) || (out_dtype != FP8BLK_OUT_BF16 && out_dtype != FP8BLK_OUT_FP32) ||
      (renormalize != 0 && renormalize != 1))
    return FP8BLK_ERR_ARG;
  if (!x || !qw1 || !sw1 || !qw2 || !sw2 || !y) return FP8BLK_ERR_NULL;
  if (int rc = check_moe_shape(T, H, I, E, k)) return rc;
  if (ld_x < H || ld_x > kMaxStride) return FP8BLK_ERR_ARG;
  if (!aligned16(x) || ld_x % 8 || !aligned16(qw1) || !aligned16(qw2) || !aligned16(y) || !aligned4(sw1) ||
      !aligned4(sw2) || !aligned4(ids) || !aligned4(weights) || !aligned16(wr))
    return FP8BLK_ERR_ALIGN;
  const MoeWorkspace w = moe_workspace(T, H, I, E, k);
  if (!workspace || ws_bytes < w.bytes) return FP8BLK_ERR_WORKSPACE;
  if (!aligned16(workspace)) return FP8BLK_ERR_ALIGN;
  if (int rc = check_device()) return rc;
  char* ws = static_cast<char*>(workspace);
  MoeArgs a{};
  a.T = (int)T; a.H = (int)H; a.I = (int)I; a.E = (int)E; a.k = k;
  a.x = x; a.ld_x = ld_x; a.wr = wr; a.renorm = renormalize != 0;
  a.ids = ids ? ids : reinterpret_cast<int32_t*>(ws + w.ids);
  a.weights = weights ? weights : reinterpret_cast<float*>(ws + w.weights);
  a.qw1 = qw1; a.sw1 = sw1; a.qw2 = qw2; a.sw2 = sw2;
  a.out = RowsOut{y, out_dtype == FP8BLK_OUT_FP32, false};
  a.fp32_scale = scale_mode == FP8BLK_SCALE_FP32;
  a.ws = workspace;
  return finish(launch_moe(a, stream));
}

}  // namespace

namespace fp8blk {

MoeWorkspace moe_workspace(int64_t T, int64_t H, int64_t I, int64_t E, int k) {
  MoeWorkspace w{};
  size_t at = 0;
  const auto take = [&](int64_t elems, size_t size) {
    const size_t start = at;
    at += up256((size_t)elems * size);
    return start;
  };
  w.logits = take(T * E, sizeof(float));
  w.ids = take(T * k, sizeof(int32_t));
  w.weights = take(T * k, sizeof(float));
  w.qx = take(T * H, sizeof(uint8_t));
  w.sx = take(T * (H / kGroup), sizeof(float));
  w.h = take(T * k * I, sizeof(uint16_t));
  w.sh = take(T * k * (I / kGroup), sizeof(float));
  // by row of h, or (few tokens) by workgroup that shares a column
  w.partial = take((T <= 16 && k < 16 ? 16 : k) * T * H, sizeof(float));
  w.bytes = at;
  return w;
}

}  // namespace fp8blk

extern "C" {

size_t fp8_linear_workspace_size(int64_t M, int64_t N, int64_t K, int scale_mode) {
  if (!valid_scale_mode(scale_mode) || M <= 0 || !mult128(N) || !mult128(K) || !linear_limits(M, N, K)) return (size_t)-1;
  return linear_bytes(M, N, K, scale_mode == FP8BLK_SCALE_FP32);
}

int fp8_linear(int64_t M, int64_t N, int64_t K, const uint16_t* x, int64_t ld_x, const uint8_t* qw, const float* sw,
               void* y, int out_dtype, int scale_mode, void* workspace, size_t ws_bytes, hipStream_t stream) {
  if (!valid_scale_mode(scale_mode) || (out_dtype != FP8BLK_OUT_BF16 && out_dtype != FP8BLK_OUT_FP32 &&
                                        out_dtype != FP8BLK_OUT_FP32_ACCUM))
    return FP8BLK_ERR_ARG;
  if (!x || !qw || !sw || !y) return FP8BLK_ERR_NULL;
  if (M <= 0 || !mult128(N) || !mult128(K)) return FP8BLK_ERR_DIM;
  if (ld_x < K || ld_x > kMaxStride || !linear_limits(M, N, K) || !prod_le(M, ld_x, kMaxElems)) return FP8BLK_ERR_ARG;
  if (!aligned16(x) || ld_x % 8 || !aligned16(qw) || !aligned4(sw) || !aligned16(y)) return FP8BLK_ERR_ALIGN;
  const bool f32 = out_dtype != FP8BLK_OUT_BF16, fp32_scale = scale_mode == FP8BLK_SCALE_FP32;
  const size_t need = linear_bytes(M, N, K, fp32_scale);
  if (need > 0 && (workspace == nullptr || ws_bytes < need)) return FP8BLK_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return FP8BLK_ERR_ALIGN;
  if (int rc = check_device()) return rc;
  const int64_t main = gemm_rows(M, N, K, fp32_scale);
  if (main > 0) {
    uint8_t* q = static_cast<uint8_t*>(workspace);
    float* s = reinterpret_cast<float*>(q + codes_bytes(main, K));
    if (hipError_t e = launch_quant_rowgroup(x, main, K, ld_x, q, K, s, fp32_scale, stream)) return finish(e);
    if (int rc = fp8_block_gemm(FP8BLK_OP_FPROP, main, N, K, q, s, qw, sw, y, out_dtype, FP8BLK_ALGO_DEFAULT,
                                scale_mode, nullptr, 0, stream))
      return rc;
  }
  if (main == M) return FP8BLK_OK;
  const RowsOut out{static_cast<char*>(y) + main * N * (f32 ? 4 : 2), f32, out_dtype == FP8BLK_OUT_FP32_ACCUM};
  return finish(launch_linear_rows(M - main, N, K, x + main * ld_x, ld_x, qw, sw, out, fp32_scale,
                                   static_cast<char*>(workspace) + gemm_bytes(main, K), stream));
}

int fp8_moe_route(int64_t T, int64_t E, int k, const void* logits, int dtype, int64_t ld, int renormalize,
                  int32_t* ids, float* weights, hipStream_t stream) {
  if (int rc = check_route(T, E, k, logits, dtype, ld, renormalize)) return rc;
  if (!ids || !weights) return FP8BLK_ERR_NULL;
  if (!aligned4(ids) || !aligned4(weights)) return FP8BLK_ERR_ALIGN;
  if (int rc = check_device()) return rc;
  return finish(launch_moe_route(T, (int)E, k, logits, dtype == FP8MOE_FP32, ld, renormalize != 0, ids, weights,
                                 stream));
}

int fp8_moe_route_backward(int64_t T, int64_t E, int k, const void* logits, int dtype, int64_t ld, const int32_t* ids,
                           const float* dweights, int renormalize, void* dlogits, int64_t ld_d, hipStream_t stream) {
  if (int rc = check_route(T, E, k, logits, dtype, ld, renormalize)) return rc;
  if (!ids || !dweights || !dlogits) return FP8BLK_ERR_NULL;
  if (ld_d < E || !prod_le(T, ld_d, kMaxElems)) return FP8BLK_ERR_ARG;
  const uintptr_t size = dtype == FP8MOE_FP32 ? 4 : 2;
  if (!aligned4(ids) || !aligned4(dweights) || reinterpret_cast<uintptr_t>(dlogits) % size) return FP8BLK_ERR_ALIGN;
  if (int rc = check_device()) return rc;
  return finish(launch_moe_route_backward(T, (int)E, k, logits, dtype == FP8MOE_FP32, ld, ids, dweights,
                                          renormalize != 0, dlogits, ld_d, stream));
}

size_t fp8_moe_workspace_size(int64_t T, int64_t H, int64_t I, int64_t E, int k) {
  if (check_moe_shape(T, H, I, E, k) != FP8BLK_OK) return (size_t)-1;
  return moe_workspace(T, H, I, E, k).bytes;
}

int fp8_moe_experts(int64_t T, int64_t H, int64_t I, int64_t E, int k, const uint16_t* x, int64_t ld_x,
                    const int32_t* ids, const float* weights, const uint8_t* qw1, const float* sw1,
                    const uint8_t* qw2, const float* sw2, void* y, int out_dtype, int scale_mode, void* workspace,
                    size_t ws_bytes, hipStream_t stream) {
  if (!ids || !weights) return FP8BLK_ERR_NULL;
  return moe(T, H, I, E, k, x, ld_x, nullptr, 0, const_cast<int32_t*>(ids), const_cast<float*>(weights), qw1, sw1,
             qw2, sw2, y, out_dtype, scale_mode, workspace, ws_bytes, stream);
}

int fp8_moe_layer(int64_t T, int64_t H, int64_t I, int64_t E, int k, int renormalize, const uint16_t* x, int64_t ld_x,
                  const uint16_t* wr, const uint8_t* qw1, const float* sw1, const uint8_t* qw2, const float* sw2,
                  void* y, int out_dtype, int scale_mode, int32_t* ids, float* weights, void* workspace,
                  size_t ws_bytes, hipStream_t stream) {
  if (!wr) return FP8BLK_ERR_NULL;
  return moe(T, H, I, E, k, x, ld_x, wr, renormalize, ids, weights, qw1, sw1, qw2, sw2, y, out_dtype, scale_mode,
             workspace, ws_bytes, stream);
}

}  // extern "C"
