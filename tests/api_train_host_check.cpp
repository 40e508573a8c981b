// Host-only check of api_train.cpp, built with g++ under the address and
// undefined-behaviour sanitizers (tests/test_train_abi.py).  The launchers and
// the HIP device queries are stubs that record what would be launched:
//   * a sort's counts fit the workspace that was asked for, its rounds cover
//     every choice once, and sorted rows hold the worst choice;
//   * launches stay below 2^32 threads at the largest sizes that are taken;
//   * the grouped products get the strides of their experts;
//   * a launch that fails ends the call with FP8BLK_ERR_HIP.
#include <cstdio>
#include <cstring>

#include "../blockwise_fp8_linear_amd/csrc/fp8train_launch.h"
#include "../include/fp8train.h"

extern "C" hipError_t hipGetDevice(int* dev) {
  *dev = 0;
  return hipSuccess;
}
extern "C" hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600* prop, int) {
  std::memset(prop, 0, sizeof *prop);
  std::strcpy(prop->gcnArchName, "gfx950:sramecc+:xnack-");
  return hipSuccess;
}

static int g_fail = 0;
#define CHECK(cond, ...)                               \
  do {                                                 \
    if (!(cond)) {                                     \
      std::printf("FAIL %s:%d: ", __FILE__, __LINE__); \
      std::printf(__VA_ARGS__);                        \
      std::printf("\n");                               \
      ++g_fail;                                        \
    }                                                  \
  } while (0)

namespace {
using namespace fp8blk;
hipError_t g_answer = hipSuccess;
int g_launches = 0;
GatherArgs g_gather;
GroupedArgs g_grouped;
GemmAlgo g_algo;
bool g_wgrad;
int64_t g_sort_n, g_sort_R;
RowsOut g_out;
template <class T>
T* at(uintptr_t a) {
  return reinterpret_cast<T*>(a << 20);
}
}  // namespace

namespace fp8blk {
hipError_t launch_moe_sort(int64_t n, int, int64_t R, const int32_t*, int32_t*, int32_t*, int32_t*, int32_t*,
                           hipStream_t) {
  g_sort_n = n;
  g_sort_R = R;
  ++g_launches;
  return g_answer;
}
hipError_t launch_moe_gather(const GatherArgs& a, hipStream_t) {
  g_gather = a;
  ++g_launches;
  return g_answer;
}
hipError_t launch_moe_combine(int64_t, int64_t, int64_t, int, const uint16_t*, int64_t, const int32_t*, const float*,
                              RowsOut out, hipStream_t) {
  g_out = out;
  ++g_launches;
  return g_answer;
}
hipError_t launch_moe_combine_dweights(int64_t, int64_t, int64_t, int, const uint16_t*, int64_t, const uint16_t*, int64_t,
                                       const int32_t*, float*, hipStream_t) {
  ++g_launches;
  return g_answer;
}
hipError_t launch_gated_forward(int64_t, int64_t, const uint16_t*, int64_t, const int32_t*, CodesOut, CodesOut, bool,
                                hipStream_t) {
  ++g_launches;
  return g_answer;
}
hipError_t launch_gated_backward(int64_t, int64_t, const uint16_t*, int64_t, const uint8_t*, int64_t, const float*,
                                 const int32_t*, CodesOut, CodesOut, CodesOut, bool, hipStream_t) {
  ++g_launches;
  return g_answer;
}
hipError_t launch_requantize_colgroup(const uint8_t*, int64_t, int64_t, int64_t, const float*, const int32_t*, CodesOut,
                                      bool, hipStream_t) {
  ++g_launches;
  return g_answer;
}
hipError_t launch_grouped_rows(const GroupedArgs& a, GemmAlgo algo, hipStream_t) {
  g_grouped = a;
  g_algo = algo;
  g_wgrad = false;
  ++g_launches;
  return g_answer;
}
hipError_t launch_grouped_wgrad(const GroupedArgs& a, GemmAlgo algo, hipStream_t) {
  g_grouped = a;
  g_algo = algo;
  g_wgrad = true;
  ++g_launches;
  return g_answer;
}
}  // namespace fp8blk

int main() {
  const int64_t kT = (int64_t(1) << 24) - 1;
  for (int64_t T : {int64_t(1), int64_t(7), int64_t(1024), int64_t(4097), int64_t(16384), int64_t(300000), kT})
    for (int64_t E : {int64_t(1), int64_t(16), int64_t(60), int64_t(1024)})
      for (int k : {1, 2, 16}) {
        if (k > E) continue;
        const int64_t n = T * k;
        const SortPlan p = sort_plan(n);
        CHECK(p.blocks >= 1 && p.blocks <= kSortMaxBlocks, "blocks of %lld", (long long)n);
        CHECK(p.blocks * p.rounds * kSortRound >= n, "rounds leave choices out at %lld", (long long)n);
        CHECK((p.blocks - 1) * p.rounds * kSortRound < n, "a workgroup without choices at %lld", (long long)n);
        const size_t need = fp8_moe_sort_workspace_size(T, E, k);
        CHECK(need == (p.blocks == 1 ? 0 : (size_t)(p.blocks * E * 4)), "workspace at %lld", (long long)n);
        // the worst choice: one choice in each of as many experts as there are choices for, the rest in one
        const int64_t m = n < E ? n : E, worst = 128 * (m - 1) + (n - m + 1 + 127) / 128 * 128;
        CHECK((int64_t)fp8_moe_sorted_rows(T, E, k) >= worst && fp8_moe_sorted_rows(T, E, k) % 512 == 0 &&
                  (int64_t)fp8_moe_sorted_rows(T, E, k) < (int64_t(1) << 31),
              "sorted rows at %lld %lld", (long long)T, (long long)E);
        CHECK(fp8_moe_sort(T, E, k, at<int32_t>(1), at<int32_t>(2), at<int32_t>(3), at<int32_t>(4), at<char>(5), need,
                           nullptr) == FP8BLK_OK,
              "sort refused");
        CHECK(g_sort_n == n && g_sort_R == (int64_t)fp8_moe_sorted_rows(T, E, k), "the sort's sizes");
      }
  // the largest calls: threads of a launch
  CHECK(((int64_t(1) << 37) - (1 << 14)) / 128 / 64 * 256 < int64_t(1) << 32, "gather of row groups");
  CHECK((int64_t(1) << 37) / (128 * 128) * 256 < int64_t(1) << 32, "gather of tiles, requantize");
  CHECK(((int64_t(1) << 35) / 128) / 32 * 256 < int64_t(1) << 32, "gated forward");
  CHECK((int64_t(1) << 25) / 4 * 256 < int64_t(1) << 32 && kT * 256 < int64_t(1) << 32, "combine");

  // operands of the three products
  const int64_t R = 1024, N = 384, K = 640, E = 5;
  auto a = at<uint8_t>(1);
  auto sa = at<float>(2);
  auto b = at<uint8_t>(3);
  auto sb = at<float>(4);
  auto off = at<int32_t>(5);
  for (int mode : {FP8BLK_SCALE_POW2, FP8BLK_SCALE_FP32})
    for (int odt : {FP8BLK_OUT_BF16, FP8BLK_OUT_FP32, FP8BLK_OUT_FP32_ACCUM}) {
      const GemmAlgo algo = mode == FP8BLK_SCALE_FP32 ? GemmAlgo::Promote : GemmAlgo::ScaledMfma;
      CHECK(fp8_moe_gemm_fprop(R, N, K, E, a, sa, b, sb, off, at<char>(6), odt, mode, nullptr) == FP8BLK_OK, "fprop");
      GemmArgs g = g_grouped.g;
      CHECK(!g_wgrad && g_algo == algo && g.I == R && g.J == N && g.R == K && !g.bt && g.sb_j == K / 128 && g.sb_r == 1 &&
                g.bmode == BScale::Block && g_grouped.b_stride == N * K && g_grouped.sb_stride == 3 * 5 &&
                g.out_f32 == (odt != FP8BLK_OUT_BF16) && g.accumulate == (odt == FP8BLK_OUT_FP32_ACCUM),
            "fprop's operands");
      CHECK(fp8_moe_gemm_dgrad(R, N, K, E, a, sa, b, sb, off, at<char>(6), odt, mode, nullptr) == FP8BLK_OK, "dgrad");
      g = g_grouped.g;
      CHECK(!g_wgrad && g_algo == algo && g.I == R && g.J == K && g.R == N && g.bt && g.sb_j == 1 && g.sb_r == K / 128 &&
                g.bmode == BScale::Block && g_grouped.b_stride == N * K && g_grouped.sb_stride == 3 * 5,
            "dgrad's operands");
      CHECK(fp8_moe_gemm_wgrad(R, N, K, E, a, sa, b, sb, off, at<char>(6), odt, mode, nullptr) == FP8BLK_OK, "wgrad");
      g = g_grouped.g;
      CHECK(g_wgrad && g_algo == algo && g.I == N && g.J == K && g.R == R && !g.bt && g.bmode == BScale::Row &&
                g_grouped.out_stride == N * K && g_grouped.E == E && g_grouped.offsets == off,
            "wgrad's operands");
    }
  // a failing launch ends the call
  g_answer = hipErrorInvalidValue;
  g_launches = 0;
  CHECK(fp8_moe_combine_backward(3, 128, 512, 2, at<uint16_t>(1), 128, at<uint16_t>(2), 128, off, off, sa, nullptr,
                                 at<uint8_t>(6), 128, at<float>(7), at<uint8_t>(8), 512, at<float>(9), at<float>(10), 0,
                                 nullptr) == FP8BLK_ERR_HIP &&
            g_launches == 1,
        "the second launch after a failed one");
  CHECK(fp8_gated_forward(3, 128, at<uint16_t>(1), 256, nullptr, at<uint8_t>(2), 128, sa, nullptr, 0, nullptr, 0,
                          nullptr) == FP8BLK_ERR_HIP,
        "gated");
  g_answer = hipSuccess;
  g_launches = 0;
  CHECK(fp8_moe_combine_backward(3, 128, 512, 2, at<uint16_t>(1), 128, at<uint16_t>(2), 128, off, off, sa, off,
                                 at<uint8_t>(6), 128, at<float>(7), at<uint8_t>(8), 512, at<float>(9), at<float>(10), 1,
                                 nullptr) == FP8BLK_OK &&
            g_launches == 2 && g_gather.weights == sa && g_gather.used == off && g_gather.qT.ld == 512 &&
            g_gather.fp32_scale,
        "the gradient's two launches");
  if (g_fail) return 1;
  std::puts("ok");
  return 0;
}
