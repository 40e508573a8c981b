// Which path fp8_linear takes, for tests/test_moe_paths.py: api_moe.cpp with
// stubs that only note what would be launched.  Reads lines "M N K scale_mode"
// and answers each with the rows of the GEMM and those of the other kernels.
#include <cstdio>
#include <cstring>

#include "../blockwise_fp8_linear_amd/csrc/fp8blk_launch.h"
#include "../blockwise_fp8_linear_amd/csrc/fp8moe_launch.h"
#include "../include/fp8moe.h"

extern "C" hipError_t hipGetDevice(int* dev) {
  *dev = 0;
  return hipSuccess;
}
extern "C" hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600* prop, int) {
  std::memset(prop, 0, sizeof *prop);
  std::strcpy(prop->gcnArchName, "gfx950");
  return hipSuccess;
}

static int64_t g_gemm, g_rows;

namespace fp8blk {
hipError_t launch_quant_rowgroup(const uint16_t*, int64_t, int64_t, int64_t, uint8_t*, int64_t, float*, bool,
                                 hipStream_t) {
  return hipSuccess;
}
hipError_t launch_linear_rows(int64_t M, int64_t, int64_t, const uint16_t*, int64_t, const uint8_t*, const float*,
                              RowsOut, bool, void*, hipStream_t) {
  g_rows += M;
  return hipSuccess;
}
hipError_t launch_moe_route(int64_t, int, int, const void*, bool, int64_t, bool, int32_t*, float*, hipStream_t) {
  return hipErrorUnknown;
}
hipError_t launch_moe_route_backward(int64_t, int, int, const void*, bool, int64_t, const int32_t*, const float*, bool,
                                     void*, int64_t, hipStream_t) {
  return hipErrorUnknown;
}
hipError_t launch_moe(const MoeArgs&, hipStream_t) { return hipErrorUnknown; }
}  // namespace fp8blk

extern "C" int fp8_block_gemm(int, int64_t M, int64_t, int64_t, const uint8_t*, const float*, const uint8_t*,
                              const float*, void*, int, int, int, void*, size_t, hipStream_t) {
  g_gemm += M;
  return FP8BLK_OK;
}

int main() {
  long long M, N, K;
  int mode;
  char* const at = reinterpret_cast<char*>(4096);  // never read
  while (std::scanf("%lld %lld %lld %d", &M, &N, &K, &mode) == 4) {
    g_gemm = g_rows = 0;
    const size_t need = fp8_linear_workspace_size(M, N, K, mode);
    const int rc = fp8_linear(M, N, K, reinterpret_cast<uint16_t*>(at), K, reinterpret_cast<uint8_t*>(at),
                              reinterpret_cast<float*>(at), at, FP8BLK_OUT_BF16, mode, at, need, nullptr);
    std::printf("%d %lld %lld\n", rc, (long long)g_gemm, (long long)g_rows);
  }
  return 0;
}
