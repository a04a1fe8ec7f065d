// Which kernel fp4_gemm_grouped takes, by its host code alone: stub launchers
// name themselves, fake pointers are never dereferenced.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstring>

#include "fp4.h"
#include "fp4_launch.hpp"

namespace {
const char* g_fn = "";
hipError_t reached(const char* fn) {
    g_fn = fn;
    return hipSuccess;
}
}  // namespace

namespace fp4dev {
hipError_t launch_rmsnorm_quant(const void*, const void*, const void*, double, int64_t, int64_t, int, void*, float*,
                                void*, uint8_t*, uint8_t*, hipStream_t) { return reached("norm"); }
int64_t rmsnorm_back_parts(int64_t, int64_t) { return 1; }
hipError_t launch_rmsnorm_back(const void*, const void*, const void*, const float*, const void*, int64_t, int64_t,
                               void*, float*, float*, hipStream_t) { return reached("norm back"); }
hipError_t launch_gemm_few(const uint8_t*, const uint8_t*, int, const int*, const uint8_t*, const uint8_t*, int64_t,
                           int64_t, int64_t, int64_t, void*, int, hipStream_t) { return reached("few"); }
hipError_t launch_quant_grouped(const void*, const int*, int64_t, int64_t, int64_t, int, int, uint64_t, int, uint64_t,
                                uint64_t, uint8_t*, uint8_t*, uint8_t*, uint8_t*, hipStream_t) { return reached("quant"); }
bool row_groups_fit(int64_t, int64_t, int64_t, int64_t) { return true; }
hipError_t launch_gemm_row_groups(const uint8_t*, const uint8_t*, const int*, int64_t, int64_t, const uint8_t*,
                                  const uint8_t*, int64_t, int64_t, void*, int, hipStream_t) { return reached("tiles"); }
hipError_t launch_gemm_depth_groups(const uint8_t*, const uint8_t*, const uint8_t*, const uint8_t*, const int*, int64_t,
                                    int64_t, int64_t, int64_t, void*, int, hipStream_t) { return reached("depth"); }
hipError_t launch_gemm_depth_short(const uint8_t*, const uint8_t*, const uint8_t*, const uint8_t*, const int*, int64_t,
                                   int64_t, int64_t, int64_t, void*, int, hipStream_t) { return reached("depth short"); }
}  // namespace fp4dev

int main() {
    uint8_t* const q = reinterpret_cast<uint8_t*>(0x10000);
    const int32_t* const off = reinterpret_cast<const int32_t*>(0x20000);
    const struct { int64_t experts, rows, N, K; const char* fn; } calls[] = {
        {1, 16384, 64, 1024, "few"},    {1, 16384, 64, 1056, "tiles"},  {1, 8192, 64, 14336, "few"},
        {1, 8193, 64, 14336, "tiles"},  {16, 4096, 256, 1024, "few"},   {16, 4096, 256, 14336, "tiles"},
        {16, 2048, 256, 14336, "few"},  {1, 2048, 512, 14336, "few"},   {1, 2049, 512, 14336, "tiles"},
        {17, 17 * 33, 64, 96, "tiles"}, {17, 17 * 32, 4096, 96, "few"}, {1, 257, 4096, 4096, "tiles"},
    };
    int failed = 0;
    for (const auto& c : calls) {
        const fp4_status s = fp4_gemm_grouped(q, q, FP4_FMT_MXFP4, off, c.experts, c.rows, q, q, c.N, c.K, q,
                                              FP4_OUT_BF16, nullptr);
        if (s == FP4_OK && std::strcmp(g_fn, c.fn) == 0) continue;
        std::printf("%d experts, %d rows, N %d, K %d: status %d, %s, expected %s\n", (int)c.experts, (int)c.rows,
                    (int)c.N, (int)c.K, (int)s, g_fn, c.fn);
        ++failed;
    }
    if (!failed) std::printf("ok\n");
    return failed;
}
