// fp4_launch.hpp -- internal launchers behind the C ABI (validated arguments
// only; every pointer and size has been checked by the caller).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <tuple>

namespace fp4dev {

// Launches kernel k with the arguments converted to its parameter types and
// returns the status of this launch alone (hipLaunchKernel), not an error
// left over from earlier runtime calls as hipGetLastError would.
template <typename... P, typename... A>
inline hipError_t launch(void (*k)(P...), dim3 grid, dim3 block, hipStream_t st, A... a) {
    static_assert(sizeof...(P) == sizeof...(A), "argument count");
    std::tuple<P...> v(static_cast<P>(a)...);
    return std::apply(
        [&](auto&... e) {
            void* args[] = {(void*)&e..., nullptr};
            return hipLaunchKernel((const void*)k, grid, block, args, 0, st);
        },
        v);
}

// A grid of at least n workgroups of `threads` in two dimensions: HIP refuses 2^32
// threads or more in one (and the refusal stays behind as the next runtime
// call's error).  The kernel takes workgroup blockIdx.y gridDim.x + blockIdx.x
// and leaves out those past its work.
inline dim3 grid_of(int64_t n, unsigned threads) {
    const int64_t most = UINT32_MAX / threads, y = (n + most - 1) / most;
    return dim3((unsigned)((n + y - 1) / y), (unsigned)y);
}

// MXFP4 quantization of bf16 x[rows, cols] along axis 0 (cols) or 1 (rows).
hipError_t launch_quant_mx(const void* x, int64_t rows, int64_t cols, int axis, int had_n, int had,
                           uint64_t sign_seed, int rnd, uint64_t sr_seed, uint8_t* codes,
                           uint8_t* scales, hipStream_t st);

// Both MXFP4 quantizations of x from one read: along rows (codes_r/scales_r,
// as axis 1) and along cols (codes_c/scales_c, as axis 0), each with its own
// rotation and rounding.  Needs rows % 32 == 0 and cols % 32 == 0.
hipError_t launch_quant_mx_dual(const void* x, int64_t rows, int64_t cols, int had_n_r, int had_r,
                                uint64_t sign_seed_r, int rnd_r, uint64_t sr_seed_r, uint8_t* codes_r,
                                uint8_t* scales_r, int had_n_c, int had_c, uint64_t sign_seed_c,
                                int rnd_c, uint64_t sr_seed_c, uint8_t* codes_c, uint8_t* scales_c,
                                hipStream_t st);

// Both outputs, without rotation and to nearest, of each matrix of a stack [count,
// rows, cols], the operands of one matrix after those of another.  Needs rows % 32 ==
// 0, cols % 32 == 0 and rows cols 2 < 2^31.
hipError_t launch_quant_mx_stack(const void* x, int64_t count, int64_t rows, int64_t cols, uint8_t* codes_r,
                                 uint8_t* scales_r, uint8_t* codes_c, uint8_t* scales_c, hipStream_t st);

// The two Wgrad operands a [rows, n1] and b [rows, n2] quantized along rows
// with one rotation (own SR seeds), in one launch when it fits.
hipError_t launch_quant_mx_pair(const void* a, int64_t rows, int64_t n1, const void* b, int64_t n2,
                                int had_n, int had, uint64_t sign_seed, int rnd, uint64_t sr_a,
                                uint64_t sr_b, uint8_t* qa, uint8_t* sa, uint8_t* qb, uint8_t* sb,
                                hipStream_t st);

// C[M, N] (row-major; fp32, or bf16 when out_bf16) = A[M, K] B[N, K]^T
// (+ C when accumulate) over MXFP4 operands.
hipError_t launch_gemm_mx(const uint8_t* aq, const uint8_t* as, const uint8_t* bq,
                          const uint8_t* bs, int64_t M, int64_t N, int64_t K, void* c,
                          int out_bf16, int accumulate, hipStream_t st);

// NVFP4 quantization (mode: 0 RTN, 1 renormalized scales by SR, 2 element
// SR); amax_dev is either the caller's amax_in or the workspace the amax pass
// writes.
hipError_t launch_nvfp4(const void* x, int64_t rows, int64_t cols, int had, uint64_t sign_seed,
                        int mode, uint64_t sr_seed, const float* amax_in, uint8_t* codes,
                        uint8_t* scales, float* tensor_scale, void* workspace, hipStream_t st);

// Device address and size of this device's scratch array (the current
// device; looked up once per device, thread-safe).
hipError_t nvfp4_scratch(void** ptr, size_t* bytes);

// Root-mean-square norm of bf16 x (+ res) with a quantized output (e4m3: MXFP8,
// else MXFP4); h, rstd and y may be null (h not with a residual).
hipError_t launch_rmsnorm_quant(const void* x, const void* res, const void* w, double eps, int64_t rows,
                                int64_t cols, int e4m3, void* h, float* rstd, void* y, uint8_t* codes,
                                uint8_t* scales, hipStream_t st);

// Its backward pass; parts: fp32 [rmsnorm_back_parts(rows, cols), cols].
int64_t rmsnorm_back_parts(int64_t rows, int64_t cols);
hipError_t launch_rmsnorm_back(const void* dy, const void* h, const void* w, const float* rstd, const void* dh,
                               int64_t rows, int64_t cols, void* dx, float* dw, float* parts, hipStream_t st);

// C[rows, N] = A W^T for few rows (per expert): A MXFP8 (a_e4m3) or MXFP4, W
// MXFP4; offsets null and experts 1 for a product without groups.
hipError_t launch_gemm_few(const uint8_t* a, const uint8_t* as, int a_e4m3, const int* offsets, const uint8_t* w,
                           const uint8_t* ws, int64_t rows, int64_t experts, int64_t N, int64_t K, void* c,
                           int out_bf16, hipStream_t st);

// C[rows, N], each expert's MXFP4 rows times its weight on the large tiles;
// and C [experts, M, N], each expert its span of A's and B's contraction: on
// the large tiles, or on small ones where an expert's span is short.
bool row_groups_fit(int64_t experts, int64_t rows, int64_t N, int64_t K);
hipError_t launch_gemm_row_groups(const uint8_t* aq, const uint8_t* as, const int* offsets, int64_t experts,
                                  int64_t rows, const uint8_t* wq, const uint8_t* ws, int64_t N, int64_t K, void* c,
                                  int out_bf16, hipStream_t st);
hipError_t launch_gemm_depth_groups(const uint8_t* aq, const uint8_t* as, const uint8_t* bq, const uint8_t* bs,
                                    const int* offsets, int64_t experts, int64_t rows, int64_t M, int64_t N, void* c,
                                    int out_bf16, hipStream_t st);
hipError_t launch_gemm_depth_short(const uint8_t* aq, const uint8_t* as, const uint8_t* bq, const uint8_t* bs,
                                   const int* offsets, int64_t experts, int64_t rows, int64_t M, int64_t N, void* c,
                                   int out_bf16, hipStream_t st);

// MXFP4 quantization of rows grouped by expert, along rows (codes_r) and / or
// along cols (codes_c).
hipError_t launch_quant_grouped(const void* x, const int* offsets, int64_t experts, int64_t rows, int64_t cols,
                                int had_n, int had, uint64_t sign_seed, int rnd, uint64_t sr_rows, uint64_t sr_cols,
                                uint8_t* codes_r, uint8_t* scales_r, uint8_t* codes_c, uint8_t* scales_c,
                                hipStream_t st);

// The k best experts of each token and their weights; the weights' gradient.
hipError_t launch_moe_route(const void* logits, int bf16, int64_t tokens, int64_t experts, int64_t k, int sigmoid,
                            int normalize, int* ids, float* weights, hipStream_t st);
hipError_t launch_moe_route_back(const float* dweights, const void* logits, int bf16, const int* ids, int64_t tokens,
                                 int64_t experts, int64_t k, int sigmoid, int normalize, void* dlogits, hipStream_t st);

// Slots sorted by expert; counts: int32 [moe_sort_workgroups(slots), experts + 1],
// not used (may be null) where that is one workgroup.
int64_t moe_sort_workgroups(int64_t slots);
hipError_t launch_moe_sort(const int* ids, int64_t slots, int64_t experts, int* offsets, int* order, int* position,
                           int* counts, hipStream_t st);

// Tokens' rows (of row_bytes bytes, a multiple of 16, and scale_bytes bytes of
// scales, may be null) to the rows of their slots; rows combined by token; the
// gradients of that.
hipError_t launch_moe_gather(const void* x, int64_t row_bytes, const uint8_t* scales, int64_t scale_bytes,
                             const int* position, int64_t tokens, int64_t k, int64_t rows, void* out,
                             uint8_t* out_scales, hipStream_t st);
hipError_t launch_moe_combine(const void* y, const int* position, const float* weights, int64_t tokens, int64_t k,
                              int64_t rows, int64_t cols, void* out, hipStream_t st);
hipError_t launch_moe_combine_back(const void* dout, const void* y, const int* position, const float* weights,
                                   int64_t tokens, int64_t k, int64_t rows, int64_t cols, void* dy, float* dweights,
                                   hipStream_t st);

// Gated activation (fmt: 0 no codes, 1 MXFP8, 2 MXFP4; y and the checkpoint xq, xs
// may be null) and its gradient from the checkpoint; weights, order and offsets
// may be null.
hipError_t launch_glu(const void* x, const float* weights, const int* order, const int* offsets, int64_t experts,
                      int gelu, int64_t rows, int64_t cols, void* y, int fmt, uint8_t* codes, uint8_t* scales,
                      uint8_t* xq, uint8_t* xs, hipStream_t st);
hipError_t launch_glu_back(const void* dy, const uint8_t* xq, const uint8_t* xs, const float* weights, const int* order,
                           const int* offsets, int64_t experts, int gelu, int64_t rows, int64_t cols, void* dx,
                           float* dweights, hipStream_t st);

uint32_t host_sign_word(int had, uint64_t seed);

}  // namespace fp4dev
