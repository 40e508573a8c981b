// Host-only check of api_moe.cpp, built with g++ under the address and
// undefined-behaviour sanitizers (tests/test_moe_abi.py).  The launchers and
// the HIP device queries are stubs that record what would be launched:
//   * fp8_linear covers every row exactly once, by the GEMM and the kernels
//     for few rows, and both stay inside x, y and the workspace it asked for;
//   * the pieces of the mixture's workspace do not overlap and fit;
//   * an error launches nothing.
#include <cstdio>
#include <cstring>
#include <vector>

#include "../blockwise_fp8_linear_amd/csrc/fp8blk_launch.h"
#include "../blockwise_fp8_linear_amd/csrc/fp8moe_launch.h"
#include "../include/fp8moe.h"

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
struct Quant { int64_t rows, cols; const uint16_t* x; const uint8_t* q; const float* s; bool f; };
struct Gemm { int64_t M, N, K; const uint8_t* a; const float* sa; const void* out; int odt, mode; };
struct Rows { int64_t M, N, K; const uint16_t* x; fp8blk::RowsOut out; bool f; const void* ws; };
std::vector<Quant> g_quant;
std::vector<Gemm> g_gemm;
std::vector<Rows> g_rows;
std::vector<fp8blk::MoeArgs> g_moe;
int g_route = 0;
size_t launches() { return g_quant.size() + g_gemm.size() + g_rows.size() + g_moe.size() + (size_t)g_route; }
}  // namespace

namespace fp8blk {
hipError_t launch_quant_rowgroup(const uint16_t* x, int64_t rows, int64_t cols, int64_t, uint8_t* q, int64_t, float* s,
                                 bool f, hipStream_t) {
  g_quant.push_back({rows, cols, x, q, s, f});
  return hipSuccess;
}
hipError_t launch_linear_rows(int64_t M, int64_t N, int64_t K, const uint16_t* x, int64_t, const uint8_t*, const float*,
                              RowsOut out, bool f, void* ws, hipStream_t) {
  g_rows.push_back({M, N, K, x, out, f, ws});
  return hipSuccess;
}
hipError_t launch_moe_route(int64_t, int, int, const void*, bool, int64_t, bool, int32_t*, float*, hipStream_t) {
  ++g_route;
  return hipSuccess;
}
hipError_t launch_moe_route_backward(int64_t, int, int, const void*, bool, int64_t, const int32_t*, const float*, bool,
                                     void*, int64_t, hipStream_t) {
  ++g_route;
  return hipErrorInvalidValue;
}
hipError_t launch_moe(const MoeArgs& a, hipStream_t) {
  g_moe.push_back(a);
  return hipSuccess;
}
}  // namespace fp8blk

extern "C" int fp8_block_gemm(int op, int64_t M, int64_t N, int64_t K, const uint8_t* a, const float* sa, const uint8_t*,
                              const float*, void* out, int odt, int algo, int mode, void*, size_t, hipStream_t) {
  CHECK(op == FP8BLK_OP_FPROP && algo == FP8BLK_ALGO_DEFAULT && M > 0 && M % 128 == 0, "the GEMM's arguments");
  g_gemm.push_back({M, N, K, a, sa, out, odt, mode});
  return FP8BLK_OK;
}

// addresses that are only compared, never read
static char* at(uintptr_t n) { return reinterpret_cast<char*>(n); }

static void linear_checks() {
  for (int64_t N : {128, 2048, 4096, 12288, 32768}) {
    for (int64_t M : {1, 8, 9, 16, 48, 49, 64, 65, 127, 128, 129, 255, 256, 300, 333, 1024, 1100, 4096, 4133, 40000}) {
      for (int mode : {0, 1}) {
        for (int odt : {0, 1, 2}) {
          const int64_t K = 1408, ld = 1432;
          const size_t need = fp8_linear_workspace_size(M, N, K, mode), size = odt ? 4 : 2;
          g_quant.clear();
          g_gemm.clear();
          g_rows.clear();
          char *x = at(1u << 20), *y = at(uintptr_t(1) << 40), *ws = at(uintptr_t(1) << 44);
          const int rc = fp8_linear(M, N, K, reinterpret_cast<uint16_t*>(x), ld, reinterpret_cast<uint8_t*>(at(256)),
                                    reinterpret_cast<float*>(at(512)), y, odt, mode, need ? ws : nullptr, need, nullptr);
          CHECK(rc == FP8BLK_OK, "M %lld N %lld: status %d", (long long)M, (long long)N, rc);
          int64_t done = 0;
          size_t used = 0;
          CHECK(g_quant.size() == g_gemm.size() && g_gemm.size() <= 1 && g_rows.size() <= 1, "launches");
          if (!g_gemm.empty()) {
            const Gemm& g = g_gemm[0];
            const Quant& q = g_quant[0];
            CHECK(M > FP8_LINEAR_FP32_ROWS, "the GEMM took few rows");
            CHECK(q.rows == g.M && q.cols == K && g.K == K && g.N == N && q.q == g.a && q.s == g.sa && q.f == (mode == 1) &&
                      g.mode == mode && g.odt == odt && g.out == y && (const char*)q.x == x,
                  "M %lld N %lld: the GEMM's operands", (long long)M, (long long)N);
            const size_t scales = (const char*)q.s - ws;
            CHECK((const char*)q.q == ws && scales >= (size_t)(q.rows * K), "codes and scales overlap");
            used = scales + (size_t)(q.rows * (K / 128)) * 4;
            done = g.M;
          }
          if (!g_rows.empty()) {
            const Rows& r = g_rows[0];
            CHECK(r.N == N && r.K == K && (const char*)r.x == x + done * ld * 2 &&
                      (char*)r.out.y == y + (size_t)(done * N) * size && r.out.f32 == (odt != 0) &&
                      r.out.accumulate == (odt == 2) && r.f == (mode == 1),
                  "M %lld N %lld: the few rows' operands", (long long)M, (long long)N);
            if (!fp8blk::rows_raw(r.M, N, K, mode == 1)) {
              const size_t from = (const char*)r.ws - ws;
              CHECK(from >= used && from % 16 == 0, "the few rows' workspace overlaps the GEMM's");
              used = from + fp8blk::rows_scales_at(r.M, K) + (size_t)(r.M * (K / 128)) * 4;
            }
            done += r.M;
          }
          CHECK(done == M, "M %lld N %lld: %lld rows", (long long)M, (long long)N, (long long)done);
          CHECK(used <= need, "M %lld N %lld: workspace %zu of %zu", (long long)M, (long long)N, used, need);
        }
      }
    }
  }
}

static void moe_checks() {
  for (int64_t T : {1, 16, 17, 512}) {
    for (int k : {1, 3, 16}) {
      const int64_t H = 384, I = 640, E = 33;
      const fp8blk::MoeWorkspace w = fp8blk::moe_workspace(T, H, I, E, k);
      const size_t parts = T <= 16 && k < 16 ? 16 : (size_t)k;
      const size_t piece[][2] = {{w.logits, (size_t)(T * E) * 4}, {w.ids, (size_t)(T * k) * 4},
                                 {w.weights, (size_t)(T * k) * 4}, {w.qx, (size_t)(T * H)},
                                 {w.sx, (size_t)(T * H / 128) * 4}, {w.h, (size_t)(T * k * I) * 2},
                                 {w.sh, (size_t)(T * k * I / 128) * 4}, {w.partial, parts * (size_t)(T * H) * 4}};
      size_t end = 0;
      for (const auto& p : piece) {
        CHECK(p[0] >= end && p[0] % 256 == 0, "pieces of the workspace overlap");
        end = p[0] + p[1];
      }
      CHECK(end <= w.bytes && w.bytes == fp8_moe_workspace_size(T, H, I, E, k), "the workspace's size");
      char* ws = at(uintptr_t(1) << 44);
      auto *u16 = reinterpret_cast<uint16_t*>(at(4096));
      auto *u8 = reinterpret_cast<uint8_t*>(at(4096));
      auto *f = reinterpret_cast<float*>(at(4096));
      int32_t ids;
      g_moe.clear();
      CHECK(fp8_moe_layer(T, H, I, E, k, 0, u16, H, u16, u8, f, u8, f, u16, 1, 1, nullptr, nullptr, ws, w.bytes, nullptr) ==
                FP8BLK_OK, "layer");
      CHECK(fp8_moe_layer(T, H, I, E, k, 1, u16, H, u16, u8, f, u8, f, u16, 0, 0, &ids, f, ws, w.bytes, nullptr) ==
                FP8BLK_OK, "layer with its choice");
      CHECK(fp8_moe_experts(T, H, I, E, k, u16, H, &ids, f, u8, f, u8, f, u16, 0, 0, ws, w.bytes, nullptr) == FP8BLK_OK,
            "experts");
      CHECK(g_moe.size() == 3, "three launches");
      CHECK((char*)g_moe[0].ids == ws + w.ids && (char*)g_moe[0].weights == ws + w.weights && !g_moe[0].renorm &&
                g_moe[0].out.f32 && g_moe[0].fp32_scale && g_moe[0].wr == u16, "the layer's own choice");
      CHECK(g_moe[1].ids == &ids && g_moe[1].weights == f && g_moe[1].renorm && !g_moe[1].out.f32, "the caller's buffers");
      CHECK(g_moe[2].wr == nullptr && g_moe[2].ids == &ids, "the caller's choice");
      const size_t before = launches();
      CHECK(fp8_moe_layer(T, H, I, E, k, 0, u16, H, u16, u8, f, u8, f, u16, 1, 1, nullptr, nullptr, ws, w.bytes - 1,
                          nullptr) == FP8BLK_ERR_WORKSPACE && launches() == before, "an error launched something");
    }
  }
  auto* f = reinterpret_cast<float*>(at(4096));
  int32_t ids;
  CHECK(fp8_moe_route(1, 4, 2, f, FP8MOE_FP32, 4, 1, &ids, f, nullptr) == FP8BLK_OK, "route");
  CHECK(fp8_moe_route_backward(1, 4, 2, f, FP8MOE_FP32, 4, &ids, f, 1, f, 4, nullptr) == FP8BLK_ERR_HIP,
        "a launch that fails is reported");
}

int main() {
  linear_checks();
  moe_checks();
  std::printf(g_fail ? "%d failed\n" : "ok\n", g_fail);
  return g_fail != 0;
}
