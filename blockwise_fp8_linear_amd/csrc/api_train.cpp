// C ABI of libfp8blk, include/fp8train.h: argument validation and dispatch.
#include "../../include/fp8train.h"

#include <hip/hip_runtime.h>

#include "fp8blk_host.h"
#include "fp8blk_launch.h"
#include "fp8train_launch.h"

using namespace fp8blk;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 24;  // of a launch with a workgroup a token
constexpr int64_t kMaxRows = int64_t(1) << 31;    // a row's number is an int32

int check_choice(int64_t T, int64_t E, int k) {
  if (T <= 0 || E <= 0 || k <= 0) return FP8BLK_ERR_DIM;
  if (T >= kMaxTokens || E > FP8MOE_MAX_EXPERTS || k > FP8MOE_MAX_TOPK || k > E) return FP8BLK_ERR_ARG;
  return FP8BLK_OK;
}

// Every choice a row, and at most 127 rows of padding for each expert reached.
int64_t sorted_rows(int64_t T, int64_t E, int k) {
  const int64_t n = T * k;
  return (n + 127 * (n < E ? n : E) + 511) / 512 * 512;
}

size_t sort_bytes(int64_t T, int64_t E, int k) {
  const SortPlan p = sort_plan(T * k);
  return p.blocks == 1 ? 0 : (size_t)(p.blocks * E) * sizeof(int32_t);
}

// What the calls on sorted rows share.
int check_sorted(int64_t T, int64_t H, int64_t R, int k) {
  if (T <= 0 || k <= 0 || !mult128(H) || !mult128(R)) return FP8BLK_ERR_DIM;
  if (T >= kMaxTokens || k > FP8MOE_MAX_TOPK || R >= kMaxRows || !prod_lt(R, H, int64_t(1) << 37) ||
      !prod_lt(T, (H + 511) / 512, int64_t(1) << 25))
    return FP8BLK_ERR_ARG;
  return FP8BLK_OK;
}

// A matrix of bf16 or codes: its row stride in elements, `multiple` of them 16
// bytes.
int check_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t multiple) {
  if (ld < cols || !prod_le(rows, ld, kMaxElems)) return FP8BLK_ERR_ARG;
  return aligned16(p) && ld % multiple == 0 ? FP8BLK_OK : FP8BLK_ERR_ALIGN;
}
int check_codes(const uint8_t* q, const float* s, int64_t rows, int64_t cols, int64_t ld) {
  if (int rc = check_matrix(q, rows, cols, ld, 16)) return rc;
  return aligned4(s) ? FP8BLK_OK : FP8BLK_ERR_ALIGN;
}

int check_gather(int64_t T, int64_t H, int64_t R, int k, const uint16_t* x, int64_t ld_x, const int32_t* source,
                 const float* weights, const int32_t* used, const CodesOut& q, const CodesOut& qT, int scale_mode) {
  if (!valid_scale_mode(scale_mode)) return FP8BLK_ERR_ARG;
  if (!x || !source || !q.q || !q.s || !qT.q != !qT.s) return FP8BLK_ERR_NULL;
  if (int rc = check_sorted(T, H, R, k)) return rc;
  if (int rc = check_matrix(x, T, H, ld_x, 8)) return rc;
  if (int rc = check_codes(q.q, q.s, R, H, q.ld)) return rc;
  if (qT.q)
    if (int rc = check_codes(qT.q, qT.s, H, R, qT.ld)) return rc;
  return aligned4(source) && aligned4(weights) && aligned4(used) ? FP8BLK_OK : FP8BLK_ERR_ALIGN;
}

enum class Way { Fprop, Dgrad, Wgrad };

int grouped(Way way, int64_t R, int64_t N, int64_t K, int64_t E, const uint8_t* a, const float* sa, const uint8_t* b,
            const float* sb, const int32_t* offsets, void* out, int out_dtype, int scale_mode, hipStream_t stream) {
  if (!valid_scale_mode(scale_mode) || (out_dtype != FP8BLK_OUT_BF16 && out_dtype != FP8BLK_OUT_FP32 &&
                                        out_dtype != FP8BLK_OUT_FP32_ACCUM))
    return FP8BLK_ERR_ARG;
  if (!a || !sa || !b || !sb || !offsets || !out) return FP8BLK_ERR_NULL;
  if (!mult128(R) || !mult128(N) || !mult128(K) || E <= 0) return FP8BLK_ERR_DIM;
  if (R >= kGroupedMaxRows || N >= (int64_t(1) << 25) || K >= (int64_t(1) << 25) || E > FP8MOE_MAX_EXPERTS ||
      !prod_le(R, N, kMaxElems) || !prod_le(R, K, kMaxElems) || !prod_le(N, K, (kMaxElems >> 2) / E))
    return FP8BLK_ERR_ARG;
  if (!aligned16(a) || !aligned16(b) || !aligned16(out) || !aligned4(sa) || !aligned4(sb) || !aligned4(offsets))
    return FP8BLK_ERR_ALIGN;
  if (int rc = check_device()) return rc;
  GroupedArgs x{};
  x.offsets = offsets;
  x.E = E;
  GemmArgs& g = x.g;
  g.a = a; g.sa = sa; g.b = b; g.sb = sb; g.out = out;
  g.out_f32 = out_dtype != FP8BLK_OUT_BF16;
  g.accumulate = out_dtype == FP8BLK_OUT_FP32_ACCUM;
  const GemmAlgo algo = scale_mode == FP8BLK_SCALE_FP32 ? GemmAlgo::Promote : GemmAlgo::ScaledMfma;
  if (way == Way::Wgrad) {
    g.I = N; g.J = K; g.R = R;
    g.bmode = BScale::Row;
    x.out_stride = N * K;
    return finish(launch_grouped_wgrad(x, algo, stream));
  }
  // weight-block scales sw[n / 128][k / 128]: Fprop's columns are n, Dgrad's k
  g.I = R;
  g.bmode = BScale::Block;
  x.b_stride = N * K;
  x.sb_stride = (N / kGroup) * (K / kGroup);
  if (way == Way::Fprop) {
    g.J = N; g.R = K; g.sb_j = K / kGroup; g.sb_r = 1;
  } else {
    g.J = K; g.R = N; g.sb_j = 1; g.sb_r = K / kGroup; g.bt = true;
  }
  return finish(launch_grouped_rows(x, algo, stream));
}

int check_gated(int64_t M, int64_t I) {
  return prod_lt(M, I, int64_t(1) << 35) && M < kMaxRows ? FP8BLK_OK : FP8BLK_ERR_ARG;
}

}  // namespace

extern "C" {

size_t fp8_moe_sorted_rows(int64_t T, int64_t E, int k) {
  return check_choice(T, E, k) == FP8BLK_OK ? (size_t)sorted_rows(T, E, k) : (size_t)-1;
}

size_t fp8_moe_sort_workspace_size(int64_t T, int64_t E, int k) {
  return check_choice(T, E, k) == FP8BLK_OK ? sort_bytes(T, E, k) : (size_t)-1;
}

int fp8_moe_sort(int64_t T, int64_t E, int k, const int32_t* ids, int32_t* rows, int32_t* source, int32_t* offsets,
                 void* workspace, size_t ws_bytes, hipStream_t stream) {
  if (!ids || !rows || !source || !offsets) return FP8BLK_ERR_NULL;
  if (int rc = check_choice(T, E, k)) return rc;
  if (!aligned4(ids) || !aligned4(rows) || !aligned4(source) || !aligned4(offsets)) return FP8BLK_ERR_ALIGN;
  const size_t need = sort_bytes(T, E, k);
  if (need > 0 && (!workspace || ws_bytes < need)) return FP8BLK_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return FP8BLK_ERR_ALIGN;
  if (int rc = check_device()) return rc;
  return finish(launch_moe_sort(T * k, (int)E, sorted_rows(T, E, k), ids, rows, source, offsets,
                                static_cast<int32_t*>(workspace), stream));
}

size_t fp8_moe_gather_workspace_size(int64_t T, int64_t H, int64_t R, int k, int transpose) {
  return check_sorted(T, H, R, k) == FP8BLK_OK ? gather_order_bytes(T, H, R, k, transpose != 0) : (size_t)-1;
}

int fp8_moe_gather(int64_t T, int64_t H, int64_t R, int k, const uint16_t* x, int64_t ld_x, const int32_t* source,
                   const float* weights, const int32_t* used, uint8_t* q, int64_t ld_q, float* s, uint8_t* qT,
                   int64_t ld_qT, float* sT, int scale_mode, void* workspace, size_t ws_bytes, hipStream_t stream) {
  const CodesOut rows{q, ld_q, s}, cols{qT, ld_qT, sT};
  if (int rc = check_gather(T, H, R, k, x, ld_x, source, weights, used, rows, cols, scale_mode)) return rc;
  const size_t need = gather_order_bytes(T, H, R, k, qT != nullptr);
  if (need > 0 && (!workspace || ws_bytes < need)) return FP8BLK_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return FP8BLK_ERR_ALIGN;
  if (int rc = check_device()) return rc;
  return finish(launch_moe_gather(
      GatherArgs{T, H, R, k, x, ld_x, source, weights, used, rows, cols, scale_mode == FP8BLK_SCALE_FP32,
                 need > 0 ? static_cast<uint32_t*>(workspace) : nullptr},
      stream));
}

int fp8_moe_combine(int64_t T, int64_t H, int64_t R, int k, const uint16_t* z, int64_t ld_z, const int32_t* rows,
                    const float* weights, void* y, int out_dtype, hipStream_t stream) {
  if (out_dtype != FP8BLK_OUT_BF16 && out_dtype != FP8BLK_OUT_FP32 && out_dtype != FP8BLK_OUT_FP32_ACCUM)
    return FP8BLK_ERR_ARG;
  if (!z || !rows || !y) return FP8BLK_ERR_NULL;
  if (int rc = check_sorted(T, H, R, k)) return rc;
  if (int rc = check_matrix(z, R, H, ld_z, 8)) return rc;
  if (!aligned16(y) || !aligned4(rows) || !aligned4(weights)) return FP8BLK_ERR_ALIGN;
  if (int rc = check_device()) return rc;
  return finish(launch_moe_combine(
      T, H, R, k, z, ld_z, rows, weights,
      RowsOut{y, out_dtype != FP8BLK_OUT_BF16, out_dtype == FP8BLK_OUT_FP32_ACCUM}, stream));
}

int fp8_moe_combine_backward(int64_t T, int64_t H, int64_t R, int k, const uint16_t* dy, int64_t ld_dy,
                             const uint16_t* z, int64_t ld_z, const int32_t* rows, const int32_t* source,
                             const float* weights, const int32_t* used, uint8_t* q, int64_t ld_q, float* s,
                             uint8_t* qT, int64_t ld_qT, float* sT, float* dweights, int scale_mode,
                             hipStream_t stream) {
  const CodesOut r{q, ld_q, s}, c{qT, ld_qT, sT};
  if (!valid_scale_mode(scale_mode)) return FP8BLK_ERR_ARG;
  if (!z || !rows || !weights || !qT || !sT || !dweights) return FP8BLK_ERR_NULL;
  if (int rc = check_gather(T, H, R, k, dy, ld_dy, source, weights, used, r, c, scale_mode)) return rc;
  if (int rc = check_matrix(z, R, H, ld_z, 8)) return rc;
  if (!aligned4(rows) || !aligned4(dweights)) return FP8BLK_ERR_ALIGN;
  if (int rc = check_device()) return rc;
  if (hipError_t e = launch_moe_gather(
          GatherArgs{T, H, R, k, dy, ld_dy, source, weights, used, r, c, scale_mode == FP8BLK_SCALE_FP32, nullptr},
          stream))
    return finish(e);
  return finish(launch_moe_combine_dweights(T, H, R, k, dy, ld_dy, z, ld_z, rows, dweights, stream));
}

int fp8_moe_gemm_fprop(int64_t R, int64_t N, int64_t K, int64_t E, const uint8_t* qx, const float* sx,
                       const uint8_t* qw, const float* sw, const int32_t* offsets, void* y, int out_dtype,
                       int scale_mode, hipStream_t stream) {
  return grouped(Way::Fprop, R, N, K, E, qx, sx, qw, sw, offsets, y, out_dtype, scale_mode, stream);
}

int fp8_moe_gemm_dgrad(int64_t R, int64_t N, int64_t K, int64_t E, const uint8_t* qdy, const float* sdy,
                       const uint8_t* qw, const float* sw, const int32_t* offsets, void* dx, int out_dtype,
                       int scale_mode, hipStream_t stream) {
  return grouped(Way::Dgrad, R, N, K, E, qdy, sdy, qw, sw, offsets, dx, out_dtype, scale_mode, stream);
}

int fp8_moe_gemm_wgrad(int64_t R, int64_t N, int64_t K, int64_t E, const uint8_t* qdyT, const float* sdyT,
                       const uint8_t* qxT, const float* sxT, const int32_t* offsets, void* dw, int out_dtype,
                       int scale_mode, hipStream_t stream) {
  return grouped(Way::Wgrad, R, N, K, E, qdyT, sdyT, qxT, sxT, offsets, dw, out_dtype, scale_mode, stream);
}

int fp8_gated_forward(int64_t M, int64_t I, const uint16_t* gu, int64_t ld_gu, const int32_t* used, uint8_t* q,
                      int64_t ld_q, float* s, uint8_t* qc, int64_t ld_qc, float* sc, int scale_mode,
                      hipStream_t stream) {
  if (!valid_scale_mode(scale_mode)) return FP8BLK_ERR_ARG;
  if (!gu || !q || !s || !qc != !sc) return FP8BLK_ERR_NULL;
  if (M <= 0 || !mult128(I)) return FP8BLK_ERR_DIM;
  if (int rc = check_gated(M, I)) return rc;
  if (int rc = check_matrix(gu, M, 2 * I, ld_gu, 8)) return rc;
  if (int rc = check_codes(q, s, M, I, ld_q)) return rc;
  if (qc)
    if (int rc = check_codes(qc, sc, M, 2 * I, ld_qc)) return rc;
  if (!aligned4(used)) return FP8BLK_ERR_ALIGN;
  if (int rc = check_device()) return rc;
  return finish(launch_gated_forward(M, I, gu, ld_gu, used, CodesOut{q, ld_q, s}, CodesOut{qc, ld_qc, sc},
                                     scale_mode == FP8BLK_SCALE_FP32, stream));
}

int fp8_gated_backward(int64_t M, int64_t I, const uint16_t* dh, int64_t ld_dh, const uint8_t* qc, int64_t ld_qc,
                       const float* sc, const int32_t* used, uint8_t* q, int64_t ld_q, float* s, uint8_t* qT,
                       int64_t ld_qT, float* sT, uint8_t* qhT, int64_t ld_qhT, float* shT, int scale_mode,
                       hipStream_t stream) {
  if (!valid_scale_mode(scale_mode)) return FP8BLK_ERR_ARG;
  if (!dh || !qc || !sc || !q || !s || !qT || !sT || !qhT || !shT) return FP8BLK_ERR_NULL;
  if (!mult128(M) || !mult128(I)) return FP8BLK_ERR_DIM;
  if (int rc = check_gated(M, I)) return rc;
  if (int rc = check_matrix(dh, M, I, ld_dh, 8)) return rc;
  if (int rc = check_codes(qc, sc, M, 2 * I, ld_qc)) return rc;
  if (int rc = check_codes(q, s, M, 2 * I, ld_q)) return rc;
  if (int rc = check_codes(qT, sT, 2 * I, M, ld_qT)) return rc;
  if (int rc = check_codes(qhT, shT, I, M, ld_qhT)) return rc;
  if (!aligned4(used)) return FP8BLK_ERR_ALIGN;
  if (int rc = check_device()) return rc;
  return finish(launch_gated_backward(M, I, dh, ld_dh, qc, ld_qc, sc, used, CodesOut{q, ld_q, s},
                                      CodesOut{qT, ld_qT, sT}, CodesOut{qhT, ld_qhT, shT},
                                      scale_mode == FP8BLK_SCALE_FP32, stream));
}

int fp8_requantize_colgroup(const uint8_t* q, int64_t rows, int64_t cols, int64_t ld_q, const float* s,
                            const int32_t* used, uint8_t* qT, int64_t ld_qT, float* sT, int scale_mode,
                            hipStream_t stream) {
  if (!valid_scale_mode(scale_mode)) return FP8BLK_ERR_ARG;
  if (!q || !s || !qT || !sT) return FP8BLK_ERR_NULL;
  if (!mult128(rows) || !mult128(cols)) return FP8BLK_ERR_DIM;
  if (rows >= kMaxRows || !prod_lt(rows, cols, int64_t(1) << 37)) return FP8BLK_ERR_ARG;
  if (int rc = check_codes(q, s, rows, cols, ld_q)) return rc;
  if (int rc = check_codes(qT, sT, cols, rows, ld_qT)) return rc;
  if (!aligned4(used)) return FP8BLK_ERR_ALIGN;
  if (int rc = check_device()) return rc;
  return finish(launch_requantize_colgroup(q, rows, cols, ld_q, s, used, CodesOut{qT, ld_qT, sT},
                                           scale_mode == FP8BLK_SCALE_FP32, stream));
}

}  // extern "C"
