// fp4_abi_ops.cpp -- the C ABI's norm, few-row and grouped entry points
// (declared in include/fp4.h): argument validation, then dispatch to the HIP
// launchers, with no HIP call before every argument has been checked.  Shapes
// come before pointers: an empty batch, whose pointers are NULL, is refused for
// its shape.  (Helpers inside extern "C" are static: a C function of an unnamed
// namespace would be exported.)
#include "fp4.h"

#include <hip/hip_runtime.h>

#include "fp4_check.hpp"
#include "fp4_launch.hpp"

using namespace fp4abi;

extern "C" {

namespace {
// rows and cols of a norm: whole 32-element blocks, a row held in registers
static fp4_status check_norm_shape(int64_t rows, int64_t cols) {
    if (rows <= 0 || cols <= 0 || cols % 32 || cols > 32768 || rows > INT32_MAX) return FP4_ERR_SHAPE;
    return FP4_OK;
}
}  // namespace

fp4_status fp4_rmsnorm_quantize(const void* x_bf16, const void* residual_bf16, const void* weight_bf16,
                                double eps, int64_t rows, int64_t cols, fp4_format fmt, void* h_bf16,
                                float* rstd, void* y_bf16, uint8_t* codes, uint8_t* scales, void* stream) {
    if (fmt != FP4_FMT_MXFP4 && fmt != FP4_FMT_MXFP8) return FP4_ERR_ENUM;
    if (!(eps >= 0.0)) return FP4_ERR_ENUM;
    if (const fp4_status s = check_norm_shape(rows, cols)) return s;
    if (!x_bf16 || !weight_bf16 || !codes || !scales || (residual_bf16 && !h_bf16)) return FP4_ERR_NULL;
    if (!aligned16(x_bf16) || !aligned16(residual_bf16) || !aligned16(weight_bf16) || !aligned16(h_bf16) ||
        !aligned4(rstd) || !aligned16(y_bf16) || !aligned16(codes) || !aligned16(scales))
        return FP4_ERR_ALIGN;
    return from_hip(fp4dev::launch_rmsnorm_quant(x_bf16, residual_bf16, weight_bf16, eps, rows, cols,
                                                 fmt == FP4_FMT_MXFP8, h_bf16, rstd, y_bf16, codes, scales,
                                                 (hipStream_t)stream));
}

size_t fp4_rmsnorm_workspace_bytes(int64_t rows, int64_t cols) {
    if (check_norm_shape(rows, cols) != FP4_OK) return 0;
    return (size_t)(fp4dev::rmsnorm_back_parts(rows, cols) * cols) * sizeof(float);
}

fp4_status fp4_rmsnorm_backward(const void* dy_bf16, const void* h_bf16, const void* weight_bf16,
                                const float* rstd, const void* dh_bf16, int64_t rows, int64_t cols,
                                void* dx_bf16, float* dw, void* workspace, size_t workspace_bytes,
                                void* stream) {
    if (const fp4_status s = check_norm_shape(rows, cols)) return s;
    if (!dy_bf16 || !h_bf16 || !weight_bf16 || !rstd || !dx_bf16 || !dw) return FP4_ERR_NULL;
    if (!workspace || workspace_bytes < fp4_rmsnorm_workspace_bytes(rows, cols)) return FP4_ERR_WORKSPACE;
    if (!aligned16(dy_bf16) || !aligned16(h_bf16) || !aligned16(weight_bf16) || !aligned4(rstd) ||
        !aligned16(dh_bf16) || !aligned16(dx_bf16) || !aligned16(dw) || !aligned16(workspace))
        return FP4_ERR_ALIGN;
    return from_hip(fp4dev::launch_rmsnorm_back(dy_bf16, h_bf16, weight_bf16, rstd, dh_bf16, rows, cols, dx_bf16,
                                                dw, (float*)workspace, (hipStream_t)stream));
}

namespace {
constexpr int64_t kMaxExperts = 1024;

static fp4_status check_grouped_product(const uint8_t* a, const uint8_t* as, fp4_format fmt, const uint8_t* wq,
                                        const uint8_t* ws, int64_t experts, int64_t rows, int64_t N, int64_t K,
                                        const void* c, fp4_out_dtype out) {
    if (fmt != FP4_FMT_MXFP4 && fmt != FP4_FMT_MXFP8) return FP4_ERR_ENUM;
    if (out != FP4_OUT_F32 && out != FP4_OUT_BF16) return FP4_ERR_ENUM;
    if (rows <= 0 || N <= 0 || K <= 0 || K % 32 || K >= kMaxContraction || rows > INT32_MAX || N > INT32_MAX ||
        experts <= 0 || experts > kMaxExperts)
        return FP4_ERR_SHAPE;
    if (!product_ok(rows + 32 * experts, K) || !product_ok(N * experts, K) || !product_ok(rows, N) ||
        (rows / 128 + experts) * ((N + 255) / 256) >= kMaxTiles)
        return FP4_ERR_SHAPE;
    // the few-row kernel has 4 threads a column at least, a launch 2^32 - 1
    if (N >= INT64_C(1) << 30) return FP4_ERR_SHAPE;
    // tiles are counted in 32 bits, also where offsets out of order overlap
    if (experts * (rows / 128 + 1) * ((N + 255) / 256) > INT32_MAX) return FP4_ERR_SHAPE;
    if (!a || !as || !wq || !ws || !c) return FP4_ERR_NULL;
    if (!aligned16(a) || !aligned16(as) || !aligned16(wq) || !aligned16(ws) || !aligned16(c)) return FP4_ERR_ALIGN;
    return FP4_OK;
}
}  // namespace

fp4_status fp4_gemm_decode(const uint8_t* a, const uint8_t* as, fp4_format fmt, const uint8_t* wq,
                           const uint8_t* ws, int64_t M, int64_t N, int64_t K, void* c, fp4_out_dtype out,
                           void* stream) {
    if (const fp4_status s = check_grouped_product(a, as, fmt, wq, ws, 1, M, N, K, c, out)) return s;
    return from_hip(fp4dev::launch_gemm_few(a, as, fmt == FP4_FMT_MXFP8, nullptr, wq, ws, M, 1, N, K, c,
                                            out == FP4_OUT_BF16, (hipStream_t)stream));
}

fp4_status fp4_quantize_grouped(const void* x_bf16, const int32_t* offsets, int64_t experts, int64_t rows,
                                int64_t cols, int had_n, fp4_hadamard had, uint64_t sign_seed, fp4_rounding rnd,
                                uint64_t sr_seed_rows, uint64_t sr_seed_cols, uint8_t* codes_rows,
                                uint8_t* scales_rows, uint8_t* codes_cols, uint8_t* scales_cols, void* stream) {
    if (had != FP4_HAD_NONE && had != FP4_HAD_DET && had != FP4_HAD_SIGNED) return FP4_ERR_ENUM;
    if (had != FP4_HAD_NONE && had_n != 16 && had_n != 32) return FP4_ERR_ENUM;
    if (rnd != FP4_RTN && rnd != FP4_SR) return FP4_ERR_ENUM;
    if (rows <= 0 || rows > INT32_MAX || cols <= 0 || cols % 32 || cols >= kMaxContraction || experts <= 0 ||
        experts > kMaxExperts || ((cols + 255) / 256) * (rows / 32 + 8 * experts) > INT32_MAX)
        return FP4_ERR_SHAPE;
    if (!x_bf16 || !offsets || (!codes_rows && !codes_cols) || !codes_rows != !scales_rows ||
        !codes_cols != !scales_cols)
        return FP4_ERR_NULL;
    if (!aligned16(x_bf16) || !aligned4(offsets) || !aligned16(codes_rows) || !aligned16(scales_rows) ||
        !aligned16(codes_cols) || !aligned16(scales_cols))
        return FP4_ERR_ALIGN;
    return from_hip(fp4dev::launch_quant_grouped(x_bf16, offsets, experts, rows, cols, had_n, (int)had, sign_seed,
                                                 (int)rnd, sr_seed_rows, sr_seed_cols, codes_rows, scales_rows,
                                                 codes_cols, scales_cols, (hipStream_t)stream));
}

fp4_status fp4_gemm_grouped(const uint8_t* a, const uint8_t* as, fp4_format fmt, const int32_t* offsets,
                            int64_t experts, int64_t rows, const uint8_t* wq, const uint8_t* ws, int64_t N,
                            int64_t K, void* c, fp4_out_dtype out, void* stream) {
    if (const fp4_status s = check_grouped_product(a, as, fmt, wq, ws, experts, rows, N, K, c, out)) return s;
    if (!offsets) return FP4_ERR_NULL;
    if (!aligned4(offsets)) return FP4_ERR_ALIGN;
    // Up to 32 rows an expert on average the few-row kernel, which reads the
    // weights once per 64 rows at most (64 experts of 1408 x 1408: 15.5 against
    // 19.6 us at 32 rows, 19.7 and 19.5 at 40; 128 of 2048 x 2048 54.5 and 53.3,
    // 81 and 55; 40 of 736 x 1120 5.7 and 8.4, 7.1 and 8.4).  Few experts with a
    // small output also beyond: the large tiles, too few of them for the CUs, take
    // the time of one (one expert, K = 4096: 14.5 us; the few-row kernel 12.6 for
    // 256 rows of 4096 columns, 8.2 for 512 of 1024, 9.7 for 2048 of 256, 7.4 for
    // 4096 of 64).  Its bound there is the rows, read again for every 16 or 32
    // columns: with few columns and a long contraction it falls behind at half
    // that output already (64 columns: K = 4096, 16384 rows 24.0 and 16.0, K =
    // 14336 70 and 38.6, 4096 rows 20.9 and 35.8; 16 experts of 256 columns, K =
    // 14336, 256 rows 53.4 and 36.3, 128 rows 29.2 and 36.0).
    const int64_t outputs = INT64_C(1) << (N < 512 && K > 1024 ? 19 : 20);
    const bool few = rows <= 32 * experts || (experts <= 16 && rows * N <= outputs);
    if (fmt == FP4_FMT_MXFP4 && !few && fp4dev::row_groups_fit(experts, rows, N, K))
        return from_hip(fp4dev::launch_gemm_row_groups(a, as, offsets, experts, rows, wq, ws, N, K, c,
                                                       out == FP4_OUT_BF16, (hipStream_t)stream));
    return from_hip(fp4dev::launch_gemm_few(a, as, fmt == FP4_FMT_MXFP8, offsets, wq, ws, rows, experts, N, K, c,
                                            out == FP4_OUT_BF16, (hipStream_t)stream));
}

fp4_status fp4_gemm_grouped_wgrad(const uint8_t* dytq, const uint8_t* dyts, const uint8_t* xtq,
                                  const uint8_t* xts, const int32_t* offsets, int64_t experts, int64_t rows,
                                  int64_t N, int64_t K, void* dw, fp4_out_dtype out, void* stream) {
    if (out != FP4_OUT_F32 && out != FP4_OUT_BF16) return FP4_ERR_ENUM;
    if (rows <= 0 || N <= 0 || K <= 0 || N % 32 || K % 32 || rows > INT32_MAX || N > INT32_MAX || K > INT32_MAX ||
        experts <= 0 || experts > kMaxExperts || 256 * (rows / 256 + experts) >= kMaxContraction ||
        (rows / 256 + experts) * (N > K ? N : K) >= (INT64_C(1) << 28) || K >= (INT64_C(1) << 21))
        return FP4_ERR_SHAPE;
    if (!product_ok(N, K) || !product_ok(N * K, experts) ||
        ((N + 255) / 256) * ((K + 255) / 256) >= kMaxTiles / experts)
        return FP4_ERR_SHAPE;
    if (!dytq || !dyts || !xtq || !xts || !offsets || !dw) return FP4_ERR_NULL;
    if (!aligned16(dytq) || !aligned16(dyts) || !aligned16(xtq) || !aligned16(xts) || !aligned4(offsets) ||
        !aligned16(dw))
        return FP4_ERR_ALIGN;
    // Up to 512 rows an expert on average the small tiles (32 experts of 2048 x
    // 2048, bf16: 65 against 75 us at 250 rows, 84 and 91 at 500, 108 and 103 at
    // 800; 8 experts of 14336 x 4096: 283 and 286 us at 512, 435 and 378 at 1024).
    auto* const run = rows <= 512 * experts ? &fp4dev::launch_gemm_depth_short : &fp4dev::launch_gemm_depth_groups;
    return from_hip(run(dytq, dyts, xtq, xts, offsets, experts, rows, N, K, dw, out == FP4_OUT_BF16,
                        (hipStream_t)stream));
}

}  // extern "C"
