// Host-only test of the C ABI's norm, few-row and grouped entry points
// (fp4_abi_ops.cpp) built with AddressSanitizer and UndefinedBehaviorSanitizer
// (tests/test_abi_ops_sanitize.py): stub launchers record what reaches them,
// valid calls must reach the right one with the right sizes, invalid ones none.
// Fake device pointers are never dereferenced.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <string>

#include "fp4.h"
#include "fp4_launch.hpp"

namespace {
std::string g_fn;
int64_t g_a, g_b, g_c, g_d;
int g_i;
const void* g_p;
int g_count = 0;
bool g_fit = true;
hipError_t g_status = hipSuccess;

hipError_t record(const char* fn, int64_t a, int64_t b, int64_t c, int64_t d, int i, const void* p) {
    g_fn = fn;
    g_a = a; g_b = b; g_c = c; g_d = d; g_i = i; g_p = p;
    ++g_count;
    return g_status;
}
}  // namespace

namespace fp4dev {
hipError_t launch_rmsnorm_quant(const void*, const void*, const void*, double, int64_t rows, int64_t cols, int e4m3,
                                void* h, float*, void*, uint8_t*, uint8_t*, hipStream_t) {
    return record("norm", rows, cols, 0, 0, e4m3, h);
}
int64_t rmsnorm_back_parts(int64_t rows, int64_t) { return rows < 256 ? rows : 256; }
hipError_t launch_rmsnorm_back(const void*, const void*, const void*, const float*, const void* dh, int64_t rows,
                               int64_t cols, void*, float*, float*, hipStream_t) {
    return record("norm back", rows, cols, 0, 0, 0, dh);
}
hipError_t launch_gemm_few(const uint8_t*, const uint8_t*, int a_e4m3, const int* offsets, const uint8_t*,
                           const uint8_t*, int64_t rows, int64_t experts, int64_t N, int64_t K, void*, int,
                           hipStream_t) {
    return record("few", rows, experts, N, K, a_e4m3, offsets);
}
hipError_t launch_quant_grouped(const void*, const int*, int64_t experts, int64_t rows, int64_t cols, int, int had,
                                uint64_t, int, uint64_t, uint64_t, uint8_t* cr, uint8_t*, uint8_t* cc, uint8_t*,
                                hipStream_t) {
    return record("quant", experts, rows, cols, had, (cr ? 2 : 0) + (cc ? 1 : 0), nullptr);
}
bool row_groups_fit(int64_t, int64_t, int64_t, int64_t) { return g_fit; }
hipError_t launch_gemm_row_groups(const uint8_t*, const uint8_t*, const int*, int64_t experts, int64_t rows,
                                  const uint8_t*, const uint8_t*, int64_t N, int64_t K, void*, int bf16, hipStream_t) {
    return record("rows", experts, rows, N, K, bf16, nullptr);
}
hipError_t launch_gemm_depth_groups(const uint8_t*, const uint8_t*, const uint8_t*, const uint8_t*, const int*,
                                    int64_t experts, int64_t rows, int64_t M, int64_t N, void*, int bf16, hipStream_t) {
    return record("depth", experts, rows, M, N, bf16, nullptr);
}
hipError_t launch_gemm_depth_short(const uint8_t*, const uint8_t*, const uint8_t*, const uint8_t*, const int*,
                                   int64_t experts, int64_t rows, int64_t M, int64_t N, void*, int bf16, hipStream_t) {
    return record("depth short", experts, rows, M, N, bf16, nullptr);
}
}  // namespace fp4dev

namespace {
int g_failed = 0;
template <typename T> T* P(uintptr_t v) { return reinterpret_cast<T*>(v); }

#define CHECK(c)                                                        \
    do {                                                                \
        if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); ++g_failed; } \
    } while (0)
#define REACHES(expr, name)                                    \
    do {                                                       \
        const int before = g_count;                            \
        CHECK((expr) == FP4_OK);                               \
        CHECK(g_count == before + 1 && g_fn == name);          \
    } while (0)
#define REFUSED(expr, st)                 \
    do {                                  \
        const int before = g_count;       \
        CHECK((expr) == (st));            \
        CHECK(g_count == before);         \
    } while (0)
}  // namespace

int main() {
    const void* x = P<void>(0x10000);
    void* h = P<void>(0x20000);
    uint8_t* q = P<uint8_t>(0x30000);
    float* f = P<float>(0x40000);
    const int32_t* off = P<int32_t>(0x50004);
    const int64_t big = INT64_C(1) << 62;

    REACHES(fp4_rmsnorm_quantize(x, x, x, 0.0, 7, 32768, FP4_FMT_MXFP8, h, f, nullptr, q, q, nullptr), "norm");
    CHECK(g_a == 7 && g_b == 32768 && g_i == 1 && g_p == h);
    REACHES(fp4_rmsnorm_quantize(x, nullptr, x, 1e-5, INT32_MAX, 32, FP4_FMT_MXFP4, nullptr, nullptr, nullptr, q, q, nullptr), "norm");
    CHECK(g_i == 0 && g_p == nullptr);
    for (int64_t rows : {INT64_C(0), INT64_C(-1), big, INT64_MIN, INT64_MAX})
        REFUSED(fp4_rmsnorm_quantize(x, x, x, 0.0, rows, 64, FP4_FMT_MXFP8, h, f, nullptr, q, q, nullptr), FP4_ERR_SHAPE);
    for (int64_t cols : {INT64_C(0), INT64_C(-32), INT64_C(33), INT64_C(32800), big, INT64_MIN})
        REFUSED(fp4_rmsnorm_quantize(x, x, x, 0.0, 4, cols, FP4_FMT_MXFP8, h, f, nullptr, q, q, nullptr), FP4_ERR_SHAPE);
    REFUSED(fp4_rmsnorm_quantize(x, x, x, 0.0, 4, 64, FP4_FMT_MXFP8, nullptr, f, nullptr, q, q, nullptr), FP4_ERR_NULL);

    CHECK(fp4_rmsnorm_workspace_bytes(1000, 64) == 256 * 64 * 4);
    CHECK(fp4_rmsnorm_workspace_bytes(big, 64) == 0 && fp4_rmsnorm_workspace_bytes(4, INT64_MIN) == 0);
    REACHES(fp4_rmsnorm_backward(x, x, x, f, nullptr, 4, 64, h, f, h, 4 * 64 * 4, nullptr), "norm back");
    REFUSED(fp4_rmsnorm_backward(x, x, x, f, nullptr, 4, 64, h, f, h, 4 * 64 * 4 - 1, nullptr), FP4_ERR_WORKSPACE);

    REACHES(fp4_gemm_decode(q, q, FP4_FMT_MXFP8, q, q, 3, 5, 96, h, FP4_OUT_F32, nullptr), "few");
    CHECK(g_a == 3 && g_b == 1 && g_c == 5 && g_d == 96 && g_i == 1 && g_p == nullptr);
    for (int64_t n : {INT64_C(0), INT64_C(-5), big, INT64_MAX, INT64_MIN}) {
        REFUSED(fp4_gemm_decode(q, q, FP4_FMT_MXFP8, q, q, n, 5, 96, h, FP4_OUT_F32, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_gemm_decode(q, q, FP4_FMT_MXFP8, q, q, 5, n, 96, h, FP4_OUT_F32, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_gemm_decode(q, q, FP4_FMT_MXFP8, q, q, 5, 5, n, h, FP4_OUT_F32, nullptr), FP4_ERR_SHAPE);
    }

    REACHES(fp4_quantize_grouped(x, off, 8, 100, 64, 32, FP4_HAD_DET, 1, FP4_SR, 2, 3, q, q, q, q, nullptr), "quant");
    CHECK(g_a == 8 && g_b == 100 && g_c == 64 && g_d == 1 && g_i == 3);
    REACHES(fp4_quantize_grouped(x, off, 1024, INT32_MAX, 32, 7, FP4_HAD_NONE, 1, FP4_SR, 2, 3, nullptr, nullptr, q, q, nullptr), "quant");
    CHECK(g_i == 1);
    REFUSED(fp4_quantize_grouped(x, off, 8, INT32_MAX, (1 << 24) - 32, 32, FP4_HAD_DET, 1, FP4_SR, 2, 3, q, q, q, q, nullptr), FP4_ERR_SHAPE);
    for (int64_t n : {INT64_C(0), INT64_C(-5), big, INT64_MAX, INT64_MIN}) {
        REFUSED(fp4_quantize_grouped(x, off, n, 100, 64, 32, FP4_HAD_DET, 1, FP4_SR, 2, 3, q, q, q, q, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_quantize_grouped(x, off, 8, n, 64, 32, FP4_HAD_DET, 1, FP4_SR, 2, 3, q, q, q, q, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_quantize_grouped(x, off, 8, 100, n, 32, FP4_HAD_DET, 1, FP4_SR, 2, 3, q, q, q, q, nullptr), FP4_ERR_SHAPE);
    }

    // few rows, many rows, many rows of MXFP8, and sizes the large tiles refuse
    REACHES(fp4_gemm_grouped(q, q, FP4_FMT_MXFP4, off, 8, 8 * 32, q, q, 64, 96, h, FP4_OUT_BF16, nullptr), "few");
    CHECK(g_p == off);
    REACHES(fp4_gemm_grouped(q, q, FP4_FMT_MXFP4, off, 17, 17 * 32 + 1, q, q, 64, 96, h, FP4_OUT_BF16, nullptr), "rows");
    CHECK(g_a == 17 && g_b == 545 && g_c == 64 && g_d == 96 && g_i == 1);
    REACHES(fp4_gemm_grouped(q, q, FP4_FMT_MXFP4, off, 17, 17 * 32, q, q, 1 << 20, 96, h, FP4_OUT_BF16, nullptr), "few");
    // up to 16 experts also 2^20 outputs
    REACHES(fp4_gemm_grouped(q, q, FP4_FMT_MXFP4, off, 16, 1 << 14, q, q, 64, 96, h, FP4_OUT_BF16, nullptr), "few");
    REACHES(fp4_gemm_grouped(q, q, FP4_FMT_MXFP4, off, 16, (1 << 14) + 1, q, q, 64, 96, h, FP4_OUT_BF16, nullptr), "rows");
    REACHES(fp4_gemm_grouped(q, q, FP4_FMT_MXFP8, off, 8, 10000, q, q, 64, 96, h, FP4_OUT_BF16, nullptr), "few");
    g_fit = false;
    REACHES(fp4_gemm_grouped(q, q, FP4_FMT_MXFP4, off, 8, 10000, q, q, 63, 96, h, FP4_OUT_BF16, nullptr), "few");
    g_fit = true;
    REFUSED(fp4_gemm_grouped(q, q, FP4_FMT_MXFP4, nullptr, 8, 100, q, q, 64, 96, h, FP4_OUT_BF16, nullptr), FP4_ERR_NULL);
    for (int64_t n : {INT64_C(0), INT64_C(-5), big, INT64_MAX, INT64_MIN}) {
        REFUSED(fp4_gemm_grouped(q, q, FP4_FMT_MXFP4, off, n, 100, q, q, 64, 96, h, FP4_OUT_BF16, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_gemm_grouped(q, q, FP4_FMT_MXFP4, off, 8, n, q, q, 64, 96, h, FP4_OUT_BF16, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_gemm_grouped(q, q, FP4_FMT_MXFP4, off, 8, 100, q, q, n, 96, h, FP4_OUT_BF16, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_gemm_grouped(q, q, FP4_FMT_MXFP4, off, 8, 100, q, q, 64, n, h, FP4_OUT_BF16, nullptr), FP4_ERR_SHAPE);
    }

    REACHES(fp4_gemm_grouped_wgrad(q, q, q, q, off, 8, 8 * 512, 64, 96, h, FP4_OUT_F32, nullptr), "depth short");
    CHECK(g_a == 8 && g_b == 4096 && g_c == 64 && g_d == 96 && g_i == 0);
    REACHES(fp4_gemm_grouped_wgrad(q, q, q, q, off, 8, 8 * 512 + 1, 64, 96, h, FP4_OUT_BF16, nullptr), "depth");
    for (int64_t n : {INT64_C(0), INT64_C(-32), big, INT64_MAX, INT64_MIN}) {
        REFUSED(fp4_gemm_grouped_wgrad(q, q, q, q, off, n, 100, 64, 96, h, FP4_OUT_F32, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_gemm_grouped_wgrad(q, q, q, q, off, 8, n, 64, 96, h, FP4_OUT_F32, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_gemm_grouped_wgrad(q, q, q, q, off, 8, 100, n, 96, h, FP4_OUT_F32, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_gemm_grouped_wgrad(q, q, q, q, off, 8, 100, 64, n, h, FP4_OUT_F32, nullptr), FP4_ERR_SHAPE);
    }

    g_status = hipErrorInvalidValue;
    CHECK(fp4_gemm_decode(q, q, FP4_FMT_MXFP4, q, q, 3, 5, 96, h, FP4_OUT_F32, nullptr) == FP4_ERR_LAUNCH);
    CHECK(fp4_gemm_grouped_wgrad(q, q, q, q, off, 8, 100, 64, 96, h, FP4_OUT_F32, nullptr) == FP4_ERR_LAUNCH);
    if (g_failed == 0) std::printf("ok\n");
    return g_failed;
}
