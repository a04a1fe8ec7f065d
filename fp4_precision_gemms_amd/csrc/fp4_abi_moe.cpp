// fp4_abi_moe.cpp -- the C ABI's entry points around the experts' products
// (declared in include/fp4.h): router, sorted slots, rows gathered and combined,
// gated activation, the experts' weights.  Argument validation, then dispatch to the HIP launchers, with
// no HIP call before every argument has been checked, shapes before pointers.
#include "fp4.h"

#include <hip/hip_runtime.h>

#include "fp4_check.hpp"
#include "fp4_launch.hpp"

using namespace fp4abi;

extern "C" {

namespace {
constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxChoices = 64;            // a lane of a wave each

static bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }

static fp4_status check_route(int64_t tokens, int64_t experts, int64_t k, fp4_out_dtype dtype, fp4_score score,
                              int normalize) {
    if (dtype != FP4_OUT_F32 && dtype != FP4_OUT_BF16) return FP4_ERR_ENUM;
    if (score != FP4_SCORE_SOFTMAX && score != FP4_SCORE_SIGMOID) return FP4_ERR_ENUM;
    if (normalize != 0 && normalize != 1) return FP4_ERR_ENUM;
    if (tokens <= 0 || experts <= 0 || experts > kMaxExperts || k <= 0 || k > experts || k > kMaxChoices ||
        tokens > INT32_MAX / k)
        return FP4_ERR_SHAPE;
    return FP4_OK;
}

static bool aligned_logits(const void* p, fp4_out_dtype dtype) {
    return dtype == FP4_OUT_BF16 ? aligned2(p) : aligned4(p);
}

static fp4_status check_rows(int64_t tokens, int64_t k, int64_t rows, int64_t cols) {
    if (tokens <= 0 || k <= 0 || tokens > INT32_MAX / k || rows <= 0 || rows > INT32_MAX || cols <= 0 || cols % 32 ||
        cols >= kMaxContraction)
        return FP4_ERR_SHAPE;
    // a token's choices are counted in 32 bits, 64 at a time
    if (k > INT32_MAX - 64) return FP4_ERR_SHAPE;
    // workgroups are counted in 32 bits, of 512 pieces of 16 bytes at most
    if (tokens > UINT32_MAX / ((cols + 4095) / 4096)) return FP4_ERR_SHAPE;
    return FP4_OK;
}

static fp4_status check_glu(int64_t rows, int64_t cols, fp4_act act, const int32_t* offsets, int64_t experts) {
    if (act != FP4_ACT_SILU && act != FP4_ACT_GELU) return FP4_ERR_ENUM;
    if (rows <= 0 || rows > INT32_MAX || cols <= 0 || cols % 32 || cols >= kMaxContraction) return FP4_ERR_SHAPE;
    if (offsets && (experts <= 0 || experts > kMaxExperts)) return FP4_ERR_SHAPE;
    // waves are counted in 32 bits, of 512 columns at most
    if (rows > (UINT32_MAX - 3) / ((cols + 511) / 512)) return FP4_ERR_SHAPE;
    return FP4_OK;
}
}  // namespace

fp4_status fp4_moe_route(const void* logits, fp4_out_dtype dtype, int64_t tokens, int64_t experts, int64_t k,
                         fp4_score score, int normalize, int32_t* ids, float* weights, void* stream) {
    if (const fp4_status s = check_route(tokens, experts, k, dtype, score, normalize)) return s;
    if (!logits || !ids || !weights) return FP4_ERR_NULL;
    if (!aligned_logits(logits, dtype) || !aligned4(ids) || !aligned4(weights)) return FP4_ERR_ALIGN;
    return from_hip(fp4dev::launch_moe_route(logits, dtype == FP4_OUT_BF16, tokens, experts, k,
                                             score == FP4_SCORE_SIGMOID, normalize, ids, weights, (hipStream_t)stream));
}

fp4_status fp4_moe_route_backward(const float* dweights, const void* logits, fp4_out_dtype dtype, const int32_t* ids,
                                  int64_t tokens, int64_t experts, int64_t k, fp4_score score, int normalize,
                                  void* dlogits, void* stream) {
    if (const fp4_status s = check_route(tokens, experts, k, dtype, score, normalize)) return s;
    if (!dweights || !logits || !ids || !dlogits) return FP4_ERR_NULL;
    if (!aligned4(dweights) || !aligned_logits(logits, dtype) || !aligned4(ids) || !aligned_logits(dlogits, dtype))
        return FP4_ERR_ALIGN;
    return from_hip(fp4dev::launch_moe_route_back(dweights, logits, dtype == FP4_OUT_BF16, ids, tokens, experts, k,
                                                  score == FP4_SCORE_SIGMOID, normalize, dlogits, (hipStream_t)stream));
}

size_t fp4_moe_sort_workspace_bytes(int64_t slots, int64_t experts) {
    if (slots <= 0 || slots > INT32_MAX || experts <= 0 || experts > kMaxExperts) return 0;
    const int64_t n = fp4dev::moe_sort_workgroups(slots);
    return n > 1 ? (size_t)(n * (experts + 1)) * sizeof(int32_t) : 0;
}

fp4_status fp4_moe_sort(const int32_t* ids, int64_t slots, int64_t experts, int32_t* offsets, int32_t* order,
                        int32_t* position, void* workspace, size_t workspace_bytes, void* stream) {
    if (slots <= 0 || slots > INT32_MAX || experts <= 0 || experts > kMaxExperts) return FP4_ERR_SHAPE;
    if (!ids || !offsets || !order || !position) return FP4_ERR_NULL;
    const size_t need = fp4_moe_sort_workspace_bytes(slots, experts);
    if (need && (!workspace || workspace_bytes < need)) return FP4_ERR_WORKSPACE;
    if (!aligned4(ids) || !aligned4(offsets) || !aligned4(order) || !aligned4(position) || !aligned16(workspace))
        return FP4_ERR_ALIGN;
    return from_hip(fp4dev::launch_moe_sort(ids, slots, experts, offsets, order, position, (int*)workspace,
                                            (hipStream_t)stream));
}

fp4_status fp4_moe_gather(const void* x, const uint8_t* scales, const int32_t* position, int64_t tokens, int64_t k,
                          int64_t rows, int64_t cols, void* out, uint8_t* out_scales, void* stream) {
    if (const fp4_status s = check_rows(tokens, k, rows, cols)) return s;
    if (!x || !position || !out || !scales != !out_scales) return FP4_ERR_NULL;
    if (!aligned16(x) || !aligned4(position) || !aligned16(out)) return FP4_ERR_ALIGN;
    return from_hip(fp4dev::launch_moe_gather(x, scales ? cols : 2 * cols, scales, cols / 32, position, tokens, k, rows,
                                              out, out_scales, (hipStream_t)stream));
}

fp4_status fp4_moe_combine(const void* y_bf16, const int32_t* position, const float* weights, int64_t tokens, int64_t k,
                           int64_t rows, int64_t cols, void* out_bf16, void* stream) {
    if (const fp4_status s = check_rows(tokens, k, rows, cols)) return s;
    if (!y_bf16 || !position || !out_bf16) return FP4_ERR_NULL;
    if (!aligned16(y_bf16) || !aligned4(position) || !aligned4(weights) || !aligned16(out_bf16)) return FP4_ERR_ALIGN;
    return from_hip(fp4dev::launch_moe_combine(y_bf16, position, weights, tokens, k, rows, cols, out_bf16,
                                               (hipStream_t)stream));
}

fp4_status fp4_moe_combine_backward(const void* dout_bf16, const void* y_bf16, const int32_t* position,
                                    const float* weights, int64_t tokens, int64_t k, int64_t rows, int64_t cols,
                                    void* dy_bf16, float* dweights, void* stream) {
    if (const fp4_status s = check_rows(tokens, k, rows, cols)) return s;
    if (!dout_bf16 || !y_bf16 || !position || !weights || !dy_bf16 || !dweights) return FP4_ERR_NULL;
    if (!aligned16(dout_bf16) || !aligned16(y_bf16) || !aligned4(position) || !aligned4(weights) ||
        !aligned16(dy_bf16) || !aligned4(dweights))
        return FP4_ERR_ALIGN;
    return from_hip(fp4dev::launch_moe_combine_back(dout_bf16, y_bf16, position, weights, tokens, k, rows, cols, dy_bf16,
                                                    dweights, (hipStream_t)stream));
}

fp4_status fp4_glu(const void* x_bf16, const float* weights, const int32_t* order, const int32_t* offsets,
                   int64_t experts, fp4_act act, int64_t rows, int64_t cols, void* y_bf16, fp4_format fmt,
                   uint8_t* codes, uint8_t* scales, uint8_t* xq, uint8_t* xs, void* stream) {
    if (fmt != FP4_FMT_MXFP4 && fmt != FP4_FMT_MXFP8) return FP4_ERR_ENUM;
    if (const fp4_status s = check_glu(rows, cols, act, offsets, experts)) return s;
    if (!x_bf16 || !codes != !scales || !xq != !xs || (!y_bf16 && !codes && !xq)) return FP4_ERR_NULL;
    if (!aligned16(x_bf16) || !aligned4(weights) || !aligned4(order) || !aligned4(offsets) || !aligned16(y_bf16) ||
        !aligned16(codes) || !aligned16(scales) || !aligned16(xq) || !aligned16(xs))
        return FP4_ERR_ALIGN;
    return from_hip(fp4dev::launch_glu(x_bf16, weights, order, offsets, experts, act == FP4_ACT_GELU, rows, cols, y_bf16,
                                       !codes ? 0 : fmt == FP4_FMT_MXFP8 ? 1 : 2, codes, scales, xq, xs,
                                       (hipStream_t)stream));
}

fp4_status fp4_glu_backward(const void* dy_bf16, const uint8_t* xq, const uint8_t* xs, const float* weights,
                            const int32_t* order, const int32_t* offsets, int64_t experts, fp4_act act, int64_t rows,
                            int64_t cols, void* dx_bf16, float* dweights, void* stream) {
    if (const fp4_status s = check_glu(rows, cols, act, offsets, experts)) return s;
    if (!dy_bf16 || !xq || !xs || !dx_bf16 || (weights && !dweights)) return FP4_ERR_NULL;
    if (!aligned16(dy_bf16) || !aligned16(xq) || !aligned16(xs) || !aligned4(weights) || !aligned4(order) ||
        !aligned4(offsets) || !aligned16(dx_bf16) || !aligned4(dweights))
        return FP4_ERR_ALIGN;
    return from_hip(fp4dev::launch_glu_back(dy_bf16, xq, xs, weights, order, offsets, experts, act == FP4_ACT_GELU, rows,
                                            cols, dx_bf16, dweights, (hipStream_t)stream));
}

fp4_status fp4_quantize_experts(const void* w_bf16, int64_t experts, int64_t N, int64_t K, uint8_t* wtq, uint8_t* wts,
                                uint8_t* wq, uint8_t* ws, void* stream) {
    if (experts <= 0 || experts > kMaxExperts || N <= 0 || K <= 0 || N % 32 || K % 32 || N >= (INT64_C(1) << 22) ||
        K >= kMaxContraction || !product_ok(N, K) || !product_ok(N * K, experts))
        return FP4_ERR_SHAPE;
    if (!w_bf16 || !wtq || !wts || !wq || !ws) return FP4_ERR_NULL;
    if (!aligned16(w_bf16) || !aligned16(wtq) || !aligned16(wts) || !aligned16(wq) || !aligned16(ws))
        return FP4_ERR_ALIGN;
    if (N * K * 2 < (INT64_C(1) << 31))
        return from_hip(fp4dev::launch_quant_mx_stack(w_bf16, experts, N, K, wtq, wts, wq, ws, (hipStream_t)stream));
    // beyond the stack's 32-bit offsets within a matrix: one after another
    for (int64_t e = 0; e < experts; ++e) {
        const hipError_t s = fp4dev::launch_quant_mx_dual(
            (const char*)w_bf16 + e * N * K * 2, N, K, 32, FP4_HAD_NONE, 0, FP4_RTN, 0, wtq + e * FP4_CODE_BYTES(K, N),
            wts + e * FP4_SCALE_BYTES(K, N), 32, FP4_HAD_NONE, 0, FP4_RTN, 0, wq + e * FP4_CODE_BYTES(N, K),
            ws + e * FP4_SCALE_BYTES(N, K), (hipStream_t)stream);
        if (s != hipSuccess) return FP4_ERR_LAUNCH;
    }
    return FP4_OK;
}

}  // extern "C"
