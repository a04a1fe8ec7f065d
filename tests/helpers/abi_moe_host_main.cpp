// Host-only test of the C ABI's entry points around the experts' products
// (fp4_abi_moe.cpp) built with AddressSanitizer and UndefinedBehaviorSanitizer
// (tests/test_abi_moe_sanitize.py): stub launchers record what reaches them, valid
// calls must reach the right one with the right sizes, invalid ones none.  Fake
// device pointers are never dereferenced.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <string>

#include "fp4.h"
#include "fp4_launch.hpp"

namespace {
std::string g_fn;
int64_t g_a, g_b, g_c, g_d;
int g_i, g_j;
const void* g_p;
int g_count = 0;
hipError_t g_status = hipSuccess;

hipError_t record(const char* fn, int64_t a, int64_t b, int64_t c, int64_t d, int i, int j, const void* p) {
    g_fn = fn;
    g_a = a; g_b = b; g_c = c; g_d = d; g_i = i; g_j = j; g_p = p;
    ++g_count;
    return g_status;
}
}  // namespace

namespace fp4dev {
hipError_t launch_moe_route(const void*, int bf16, int64_t tokens, int64_t experts, int64_t k, int sigmoid, int normalize,
                            int*, float*, hipStream_t) {
    return record("route", tokens, experts, k, bf16, sigmoid, normalize, nullptr);
}
hipError_t launch_moe_route_back(const float*, const void*, int bf16, const int* ids, int64_t tokens, int64_t experts,
                                 int64_t k, int sigmoid, int normalize, void*, hipStream_t) {
    return record("route back", tokens, experts, k, bf16, sigmoid, normalize, ids);
}
int64_t moe_sort_workgroups(int64_t slots) { return slots <= 4096 ? 1 : 10; }
hipError_t launch_moe_sort(const int*, int64_t slots, int64_t experts, int*, int*, int*, int* counts, hipStream_t) {
    return record("sort", slots, experts, 0, 0, 0, 0, counts);
}
hipError_t launch_moe_gather(const void*, int64_t row_bytes, const uint8_t* scales, int64_t scale_bytes, const int*,
                             int64_t tokens, int64_t k, int64_t rows, void*, uint8_t*, hipStream_t) {
    return record("gather", row_bytes, tokens, k, rows, (int)scale_bytes, 0, scales);
}
hipError_t launch_moe_combine(const void*, const int*, const float* weights, int64_t tokens, int64_t k, int64_t rows,
                              int64_t cols, void*, hipStream_t) {
    return record("combine", tokens, k, rows, cols, 0, 0, weights);
}
hipError_t launch_moe_combine_back(const void*, const void*, const int*, const float* weights, int64_t tokens, int64_t k,
                                   int64_t rows, int64_t cols, void*, float*, hipStream_t) {
    return record("combine back", tokens, k, rows, cols, 0, 0, weights);
}
hipError_t launch_glu(const void*, const float*, const int*, const int* offsets, int64_t experts, int gelu, int64_t rows,
                      int64_t cols, void* y, int fmt, uint8_t*, uint8_t*, uint8_t* xq, uint8_t*, hipStream_t) {
    return record("glu", experts, rows, cols, (y ? 1 : 0) + (xq ? 2 : 0), gelu, fmt, offsets);
}
hipError_t launch_glu_back(const void*, const uint8_t*, const uint8_t*, const float* weights, const int*, const int*,
                           int64_t experts, int gelu, int64_t rows, int64_t cols, void*, float*, hipStream_t) {
    return record("glu back", experts, rows, cols, 0, gelu, 0, weights);
}
hipError_t launch_quant_mx_stack(const void*, int64_t count, int64_t rows, int64_t cols, uint8_t*, uint8_t*, uint8_t*,
                                 uint8_t*, hipStream_t) {
    return record("stack", count, rows, cols, 0, 0, 0, nullptr);
}
hipError_t launch_quant_mx_dual(const void* x, int64_t rows, int64_t cols, int, int had_r, uint64_t, int rnd_r, uint64_t,
                                uint8_t* codes_r, uint8_t*, int, int, uint64_t, int, uint64_t, uint8_t*,
                                uint8_t* scales_c, hipStream_t) {
    return record("dual", rows, cols, codes_r - (uint8_t*)nullptr, scales_c - (uint8_t*)nullptr, had_r, rnd_r, x);
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
    void* x = P<void>(0x10000);
    uint8_t* q = P<uint8_t>(0x30000);
    float* f = P<float>(0x40004);
    int32_t* i = P<int32_t>(0x50004);
    const int64_t big = INT64_C(1) << 62;
    const int64_t bad[] = {INT64_C(0), INT64_C(-5), big, INT64_MAX, INT64_MIN};

    REACHES(fp4_moe_route(f, FP4_OUT_F32, 7, 1024, 64, FP4_SCORE_SIGMOID, 1, i, f, nullptr), "route");
    CHECK(g_a == 7 && g_b == 1024 && g_c == 64 && g_d == 0 && g_i == 1 && g_j == 1);
    REACHES(fp4_moe_route(P<void>(0x10002), FP4_OUT_BF16, INT32_MAX, 1, 1, FP4_SCORE_SOFTMAX, 0, i, f, nullptr), "route");
    REFUSED(fp4_moe_route(f, FP4_OUT_F32, INT32_MAX, 2, 2, FP4_SCORE_SOFTMAX, 0, i, f, nullptr), FP4_ERR_SHAPE);
    for (int64_t n : bad) {
        REFUSED(fp4_moe_route(f, FP4_OUT_F32, n, 64, 6, FP4_SCORE_SOFTMAX, 0, i, f, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_moe_route(f, FP4_OUT_F32, 4, n, 6, FP4_SCORE_SOFTMAX, 0, i, f, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_moe_route(f, FP4_OUT_F32, 4, 64, n, FP4_SCORE_SOFTMAX, 0, i, f, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_moe_route_backward(f, f, FP4_OUT_F32, i, n, 64, 6, FP4_SCORE_SOFTMAX, 0, f, nullptr), FP4_ERR_SHAPE);
    }
    REACHES(fp4_moe_route_backward(f, f, FP4_OUT_F32, i, 9, 64, 6, FP4_SCORE_SOFTMAX, 0, f, nullptr), "route back");
    CHECK(g_a == 9 && g_b == 64 && g_c == 6 && g_p == i);

    CHECK(fp4_moe_sort_workspace_bytes(4096, 8) == 0 && fp4_moe_sort_workspace_bytes(4097, 8) == 10 * 9 * 4);
    for (int64_t n : bad) {
        CHECK(fp4_moe_sort_workspace_bytes(n, 8) == 0 && fp4_moe_sort_workspace_bytes(5000, n) == 0);
        REFUSED(fp4_moe_sort(i, n, 8, i, i, i, x, 1 << 20, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_moe_sort(i, 5000, n, i, i, i, x, 1 << 20, nullptr), FP4_ERR_SHAPE);
    }
    REACHES(fp4_moe_sort(i, 4096, 1024, i, i, i, nullptr, 0, nullptr), "sort");
    REACHES(fp4_moe_sort(i, 4097, 8, i, i, i, x, 360, nullptr), "sort");
    CHECK(g_a == 4097 && g_b == 8 && g_p == x);
    REFUSED(fp4_moe_sort(i, 4097, 8, i, i, i, x, 359, nullptr), FP4_ERR_WORKSPACE);
    REFUSED(fp4_moe_sort(i, 4097, 8, i, i, i, nullptr, 360, nullptr), FP4_ERR_WORKSPACE);
    REFUSED(fp4_moe_sort(i, 4097, 8, i, i, i, P<void>(0x10008), 360, nullptr), FP4_ERR_ALIGN);

    REACHES(fp4_moe_gather(x, nullptr, i, 5, 2, 11, 96, x, nullptr, nullptr), "gather");
    CHECK(g_a == 192 && g_b == 5 && g_c == 2 && g_d == 11 && g_p == nullptr);
    REACHES(fp4_moe_gather(x, P<uint8_t>(0x30001), i, 5, 2, 11, 96, x, P<uint8_t>(0x30003), nullptr), "gather");
    CHECK(g_a == 96 && g_i == 3);
    REFUSED(fp4_moe_gather(x, q, i, 5, 2, 11, 96, x, nullptr, nullptr), FP4_ERR_NULL);
    REFUSED(fp4_moe_gather(x, nullptr, i, 5, 2, 11, 96, x, q, nullptr), FP4_ERR_NULL);
    // more workgroups than 32 bits count
    REFUSED(fp4_moe_combine(x, i, f, INT32_MAX, 1, 5, (1 << 24) - 32, x, nullptr), FP4_ERR_SHAPE);
    REACHES(fp4_moe_combine(x, i, nullptr, INT32_MAX, 1, INT32_MAX, 8192, x, nullptr), "combine");
    CHECK(g_a == INT32_MAX && g_b == 1 && g_c == INT32_MAX && g_d == 8192 && g_p == nullptr);
    REACHES(fp4_moe_combine_backward(x, x, i, f, 5, 2, 11, 96, x, f, nullptr), "combine back");
    REFUSED(fp4_moe_combine_backward(x, x, i, nullptr, 5, 2, 11, 96, x, f, nullptr), FP4_ERR_NULL);
    for (int64_t n : bad) {
        REFUSED(fp4_moe_gather(x, nullptr, i, n, 2, 11, 96, x, nullptr, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_moe_gather(x, nullptr, i, 5, n, 11, 96, x, nullptr, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_moe_gather(x, nullptr, i, 5, 2, n, 96, x, nullptr, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_moe_gather(x, nullptr, i, 5, 2, 11, n, x, nullptr, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_moe_combine(x, i, f, n, 2, 11, 96, x, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_moe_combine_backward(x, x, i, f, 5, 2, 11, n, x, f, nullptr), FP4_ERR_SHAPE);
    }

    REACHES(fp4_glu(x, f, i, i, 8, FP4_ACT_GELU, 3, 64, x, FP4_FMT_MXFP8, nullptr, nullptr, q, q, nullptr), "glu");
    CHECK(g_a == 8 && g_b == 3 && g_c == 64 && g_d == 3 && g_i == 1 && g_j == 0 && g_p == i);
    REACHES(fp4_glu(x, nullptr, nullptr, nullptr, 0, FP4_ACT_SILU, 3, 64, nullptr, FP4_FMT_MXFP8, q, q, nullptr, nullptr, nullptr), "glu");
    CHECK(g_d == 0 && g_j == 1);
    REACHES(fp4_glu(x, nullptr, nullptr, nullptr, 0, FP4_ACT_SILU, 3, 64, nullptr, FP4_FMT_MXFP4, q, q, nullptr, nullptr, nullptr), "glu");
    CHECK(g_j == 2);
    REFUSED(fp4_glu(x, f, i, i, 8, FP4_ACT_SILU, 3, 64, nullptr, FP4_FMT_MXFP8, nullptr, nullptr, nullptr, nullptr, nullptr), FP4_ERR_NULL);
    REFUSED(fp4_glu(x, f, i, i, 8, FP4_ACT_SILU, INT32_MAX, 1 << 12, x, FP4_FMT_MXFP8, nullptr, nullptr, nullptr, nullptr, nullptr), FP4_ERR_SHAPE);
    REACHES(fp4_glu_backward(x, q, q, f, i, i, 8, FP4_ACT_GELU, 3, 64, x, f, nullptr), "glu back");
    CHECK(g_a == 8 && g_b == 3 && g_c == 64 && g_i == 1 && g_p == f);
    REACHES(fp4_glu_backward(x, q, q, nullptr, i, nullptr, 0, FP4_ACT_SILU, 3, 64, x, nullptr, nullptr), "glu back");
    REFUSED(fp4_glu_backward(x, q, q, f, i, i, 8, FP4_ACT_GELU, 3, 64, x, nullptr, nullptr), FP4_ERR_NULL);
    for (int64_t n : bad) {
        REFUSED(fp4_glu(x, f, i, i, n, FP4_ACT_SILU, 3, 64, x, FP4_FMT_MXFP8, nullptr, nullptr, q, q, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_glu(x, f, i, i, 8, FP4_ACT_SILU, n, 64, x, FP4_FMT_MXFP8, nullptr, nullptr, q, q, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_glu(x, f, i, i, 8, FP4_ACT_SILU, 3, n, x, FP4_FMT_MXFP8, nullptr, nullptr, q, q, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_glu_backward(x, q, q, f, i, i, 8, FP4_ACT_SILU, n, 64, x, f, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_glu_backward(x, q, q, f, i, i, 8, FP4_ACT_SILU, 3, n, x, f, nullptr), FP4_ERR_SHAPE);
    }

    REACHES(fp4_quantize_experts(x, 64, 2816, 2048, q, q, q, q, nullptr), "stack");
    CHECK(g_a == 64 && g_b == 2816 && g_c == 2048);
    for (int64_t n : bad) {
        REFUSED(fp4_quantize_experts(x, n, 64, 64, q, q, q, q, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_quantize_experts(x, 4, n, 64, q, q, q, q, nullptr), FP4_ERR_SHAPE);
        REFUSED(fp4_quantize_experts(x, 4, 64, n, q, q, q, q, nullptr), FP4_ERR_SHAPE);
    }
    // an expert of 2 GiB: one launch each, at its own operands
    {
        const int before = g_count;
        const int64_t N = 1 << 15, K = 1 << 15;
        CHECK(fp4_quantize_experts(x, 3, N, K, q, q, q, q, nullptr) == FP4_OK);
        CHECK(g_count == before + 3 && g_fn == "dual" && g_a == N && g_b == K);
        CHECK(g_p == P<char>(0x10000) + 2 * N * K * 2);
        CHECK(g_c == 0x30000 + 2 * FP4_CODE_BYTES(K, N));
        CHECK(g_d == 0x30000 + 2 * FP4_SCALE_BYTES(N, K));
    }

    g_status = hipErrorInvalidValue;
    CHECK(fp4_quantize_experts(x, 3, 1 << 15, 1 << 15, q, q, q, q, nullptr) == FP4_ERR_LAUNCH);
    CHECK(fp4_moe_sort(i, 5, 8, i, i, i, nullptr, 0, nullptr) == FP4_ERR_LAUNCH);
    CHECK(fp4_moe_gather(x, nullptr, i, 5, 2, 11, 96, x, nullptr, nullptr) == FP4_ERR_LAUNCH);
    CHECK(fp4_glu_backward(x, q, q, f, i, i, 8, FP4_ACT_GELU, 3, 64, x, f, nullptr) == FP4_ERR_LAUNCH);
    if (g_failed == 0) std::printf("ok\n");
    return g_failed;
}
