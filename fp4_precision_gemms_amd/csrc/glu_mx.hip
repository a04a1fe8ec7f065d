// glu_mx.hip -- the gated activation between two products, its input kept in 8
// bits for the backward pass.
//
// x[rows, 2 C]: gate g (the first C columns) and up u.  Per row r, w its weight (1 if
// not given):
//     y = w act(g) u,   act(g) = g sigma(s(g))
//     SILU: s = g       GELU (the tanh form): s = 2 sqrt(2/pi) (g + 0.044715 g^3),
//                       since (1 + tanh z) / 2 = sigma(2 z)
// in binary32, rounded once: to bf16, or to 32-element blocks of MXFP8 / MXFP4.  The
// checkpoint is x itself in MXFP8 (as fp4_rmsnorm_quantize writes it): 1.03 bytes an
// element instead of 2 of what is usually the largest tensor that a layer keeps.
// Backward, from the checkpoint's values:
//     dg = dy w u (sigma + g s'(g) sigma (1 - sigma)),  du = dy w act(g),
//     dw_r = sum over C of dy act(g) u
// sigma and sigma (1 - sigma) come from e = exp(-|s|) <= 1, so that nothing
// overflows and 1 - sigma is no difference of near values.
//
// Bound by HBM: 4 bytes read an element of y and 2 written, 2.06 more for the
// checkpoint; backward 4.06 read and 4 written.  16384 x 14336: 302 us (6.3 TB/s)
// forward with the checkpoint, 300 (6.3) backward.
#include "exp_device.hpp"
#include "fp4_launch.hpp"
#include "mx_device.hpp"
#include "wave.hpp"

namespace fp4dev {
namespace {

constexpr int kThreads = 256;

// Non-temporal accesses (FAR) where the call's input is larger than the 256 MB
// last-level cache: nothing of it is there any more, or will be when the next call
// reads the outputs.  With the products before and the quantizer behind, 16384 rows
// of 14336 columns 676 to 648 us forward, 724 to 715 backward, of 4096 columns 205 to
// 186 and 213 to 200; below that size they lose: 8192 rows of 4096 columns 104 to
// 108 and 98 to 102, 4096 of 5152 71 to 72 and 70 to 75.
constexpr int64_t kFarBytes = INT64_C(1) << 28;

// Rows that belong to an expert, all of them without offsets.
struct Live {
    const int* offsets;
    int experts;
    __device__ __forceinline__ bool has(int64_t row) const {
        return !offsets || (row >= offsets[0] && row < offsets[experts]);
    }
};

// A row's weight's index: of its slot where an order is given, -1 for one out of range.
__device__ __forceinline__ int64_t weight_at(const int* order, int64_t row, int64_t rows) {
    if (!order) return row;
    const int s = wave_uniform(order[row]);
    return s >= 0 && s < rows ? s : -1;
}

template <bool GELU>
struct Act {
    float value, slope;                                // act(g) and act'(g)
    __device__ __forceinline__ Act(float g) {
        constexpr float kC = 1.59576912f, kD = 1.59576912f * 0.044715f;
        const float q = g * g;
        const float s = GELU ? g * __builtin_fmaf(q, kD, kC) : g;
        const float gds = GELU ? g * __builtin_fmaf(q, 3.0f * kD, kC) : g;      // g s'(g)
        const float e = exp_minus(fabsf(s)), r = __builtin_amdgcn_rcpf(1.0f + e);
        const float er = e * r, sigma = s < 0.0f ? er : r, both = er * r;
        value = g * sigma;
        // where sigma (1 - sigma) is zero g s'(g) may be infinite
        slope = both == 0.0f ? sigma : __builtin_fmaf(gds, both, sigma);
    }
};

// 8 elements of a row to MXFP8, this lane's quarter of a 32-element block.
template <bool FAR>
__device__ __forceinline__ void store_mxfp8(const float* a, uint8_t* codes, uint8_t* scale, bool first) {
    uint32_t m = max_abs_bits<8>(a);
    m = max(m, quad_xor1(m));
    m = max(m, quad_xor2(m));
    const uint32_t byte = e8m0_from_amax_bits_e4m3(m);
    uint2 word = make_uint2(0, 0);
    if (byte != 255u) word = encode8_e4m3(a, byte);
    store8<FAR>(codes, word);
    if (first) *scale = (uint8_t)byte;
}

// A wave takes 64 x 8 elements of a row (128 x 8: 16384 x 14336 345 against 334 us,
// 1999 x 736 5.4 and 4.9).  FMT: 0 no quantized output, 1 MXFP8, 2 MXFP4.
template <bool GELU, int FMT, bool FAR>
__global__ __launch_bounds__(kThreads) void glu_forward(const uint4* __restrict__ x, const float* __restrict__ weights,
                                                        const int* __restrict__ order, Live live, int64_t rows,
                                                        int cols, uint4* __restrict__ y, uint8_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales, uint8_t* __restrict__ xq,
                                                        uint8_t* __restrict__ xs) {
    const int nch = cols / 8, nb = cols / 32;
    const uint32_t wave = (blockIdx.y * gridDim.x + blockIdx.x) * (kThreads / 64) + wave_uniform(threadIdx.x >> 6);
    const uint32_t parts = (nch + 63) / 64, row32 = parts == 1 ? wave : wave / parts;
    const int64_t row = row32;
    const int c = (int)(wave - row32 * parts) * 64 + (threadIdx.x & 63);
    if (row >= rows || c >= nch || !live.has(row)) return;             // uniform per quad: cols % 32 == 0
    float g[8], u[8];
    unpack8(load16<FAR>(x + row * 2 * nch + c), g);
    unpack8(load16<FAR>(x + row * 2 * nch + nch + c), u);
    float w = 1.0f;
    if (weights) {
        const int64_t s = weight_at(order, row, rows);
        w = s >= 0 ? weights[s] : 0.0f;
    }
    const bool first = (c & 3) == 0;
    const int b = c >> 2;
    if (xq) {
        store_mxfp8<FAR>(g, xq + (row * 2 * nch + c) * 8, xs + row * 2 * nb + b, first);
        store_mxfp8<FAR>(u, xq + (row * 2 * nch + nch + c) * 8, xs + row * 2 * nb + nb + b, first);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = Act<GELU>(g[k]).value * u[k] * w;
    if (y) store16<FAR>(y + row * nch + c, pack8(g));
    if constexpr (FMT == 1) store_mxfp8<FAR>(g, codes + (row * nch + c) * 8, scales + row * nb + b, first);
    if constexpr (FMT == 2) {
        uint32_t m = max_abs_bits<8>(g);
        m = max(m, quad_xor1(m));
        m = max(m, quad_xor2(m));
        const uint32_t byte = e8m0_from_amax_bits(m);
        uint32_t word = 0;
        if (byte != 255u) {
            const uint4 z = make_uint4(0, 0, 0, 0);
            word = byte != 0u ? encode8_hw(g, byte) : encode8_sw<false>(g, byte, z, z);
        }
        *reinterpret_cast<uint32_t*>(codes + tiled_offset(row, b, nb) + 4 * (c & 3)) = word;
        if (first) scales[((int64_t)(b >> 3) * rows + row) * 8 + (b & 7)] = (uint8_t)byte;
    }
}

// The values of 8 E4M3 codes under scale byte `byte`; NaN under 255.
__device__ __forceinline__ void decode8_e4m3(uint2 q, uint32_t byte, float* a) {
    const float s = __uint_as_float(byte == 255u ? 0x7FC00000u : byte == 0u ? 0x00400000u : byte << 23);
    typedef float v2f __attribute__((ext_vector_type(2)));
    const v2f v[4] = {__builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, false), __builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, true),
                      __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, false), __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, true)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[2 * i] = v[i].x * s;
        a[2 * i + 1] = v[i].y * s;
    }
}

// TPR threads share a row: a wave, or the workgroup.
constexpr int back_threads(int tpr) { return tpr < 256 ? 256 : tpr; }

template <bool GELU, int TPR, bool FAR>
__global__ __launch_bounds__(back_threads(TPR)) void glu_back(const uint4* __restrict__ dy, const uint2* __restrict__ xq,
                                                     const uint8_t* __restrict__ xs, const float* __restrict__ weights,
                                                     const int* __restrict__ order, Live live, int64_t rows, int cols,
                                                     uint4* __restrict__ dx, float* __restrict__ dweights) {
    constexpr int kThreads = back_threads(TPR);
    __shared__ float part[kThreads / 64];
    const int nch = cols / 8, nb = cols / 32;
    const int64_t row =
        (int64_t)(blockIdx.y * gridDim.x + blockIdx.x) * (kThreads / TPR) + wave_uniform(threadIdx.x / TPR);
    if (row >= rows) return;                           // a wave of its own, or the whole workgroup
    const int t = threadIdx.x % TPR;
    const int64_t slot = weights ? weight_at(order, row, rows) : -1;
    if (!live.has(row)) {
        if (t == 0 && slot >= 0) dweights[slot] = 0.0f;
        return;
    }
    const float w = !weights ? 1.0f : slot >= 0 ? weights[slot] : 0.0f;
    float sum = 0.0f;
    for (int c = t; c < nch; c += TPR) {
        const uint4 d = load16<FAR>(dy + row * nch + c);
        const uint2 gq = load8<FAR>(xq + row * 2 * nch + c), uq = load8<FAR>(xq + row * 2 * nch + nch + c);
        const uint32_t gs = xs[row * 2 * nb + (c >> 2)], us = xs[row * 2 * nb + nb + (c >> 2)];
        float a[8], g[8], u[8];
        unpack8(d, a);
        decode8_e4m3(gq, gs, g);
        decode8_e4m3(uq, us, u);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const Act<GELU> act(g[k]);
            sum = __builtin_fmaf(a[k] * act.value, u[k], sum);
            const float dw = a[k] * w;
            g[k] = dw * u[k] * act.slope;
            u[k] = dw * act.value;
        }
        store16<FAR>(dx + row * 2 * nch + c, pack8(g));
        store16<FAR>(dx + row * 2 * nch + nch + c, pack8(u));
    }
    if (!weights) return;
    sum = wave_sum(sum);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
        __syncthreads();
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) sum += part[i];
    }
    if (t == 0 && slot >= 0) dweights[slot] = sum;
}

template <int FMT>
hipError_t launch_forward(bool gelu, const void* x, const float* weights, const int* order, Live live, int64_t rows,
                          int64_t cols, void* y, uint8_t* codes, uint8_t* scales, uint8_t* xq, uint8_t* xs,
                          hipStream_t st) {
    const int64_t waves = rows * ((cols / 8 + 63) / 64);
    const bool far = 4 * rows * cols >= kFarBytes;
    auto* const run = far ? (gelu ? &glu_forward<true, FMT, true> : &glu_forward<false, FMT, true>)
                          : (gelu ? &glu_forward<true, FMT, false> : &glu_forward<false, FMT, false>);
    return launch(run, grid_of((waves + 3) / 4, kThreads), dim3(kThreads), st, (const uint4*)x, weights, order, live, rows,
                  (int)cols, (uint4*)y, codes, scales, xq, xs);
}

template <int TPR>
hipError_t launch_back(bool gelu, const void* dy, const uint8_t* xq, const uint8_t* xs, const float* weights,
                       const int* order, Live live, int64_t rows, int64_t cols, void* dx, float* dweights,
                       hipStream_t st) {
    const bool far = 4 * rows * cols >= kFarBytes;
    auto* const run = far ? (gelu ? &glu_back<true, TPR, true> : &glu_back<false, TPR, true>)
                          : (gelu ? &glu_back<true, TPR, false> : &glu_back<false, TPR, false>);
    constexpr int kThreads = back_threads(TPR), kRows = kThreads / TPR;
    return launch(run, grid_of((rows + kRows - 1) / kRows, kThreads), dim3(kThreads), st, (const uint4*)dy,
                  (const uint2*)xq, xs, weights, order, live, rows, (int)cols, (uint4*)dx, dweights);
}

}  // namespace

hipError_t launch_glu(const void* x, const float* weights, const int* order, const int* offsets, int64_t experts,
                      int gelu, int64_t rows, int64_t cols, void* y, int fmt, uint8_t* codes, uint8_t* scales,
                      uint8_t* xq, uint8_t* xs, hipStream_t st) {
    auto* const run = fmt == 0 ? &launch_forward<0> : fmt == 1 ? &launch_forward<1> : &launch_forward<2>;
    return run(gelu != 0, x, weights, order, Live{offsets, (int)experts}, rows, cols, y, codes, scales, xq, xs, st);
}

hipError_t launch_glu_back(const void* dy, const uint8_t* xq, const uint8_t* xs, const float* weights, const int* order,
                           const int* offsets, int64_t experts, int gelu, int64_t rows, int64_t cols, void* dx,
                           float* dweights, hipStream_t st) {
    // 1024 threads for a row of 8192 columns or more (16384 x 14336 344 us with 256,
    // 321 with 512, 299 with 1024; 96 x 14336 8.2, 6.7 and 6.0; but 16384 x 4096 87, 86
    // and 103); a wave where it is one or two pieces of it, and where 256 threads would
    // idle for the most part, if there are rows enough (12000 x 1408 27.1 and 24.9 us).
    // A wave and 256 threads for up to 1024 columns: 12000 x 512 13.5 and 17.3 us, 12000 x
    // 1024 22.8 and 25.0; with fewer rows they are even, or the wave loses: 1999 x 512 4.0
    // and 4.1, 1999 x 736 5.9 and 5.7, 96 x 512 2.6 and 2.8, 96 x 736 3.4 and 2.8.
    auto* const run = cols >= 8192                                       ? &launch_back<1024>
                      : cols <= 1024 || (cols < 2048 && rows >= 1024) ? &launch_back<64>
                                                                         : &launch_back<256>;
    return run(gelu != 0, dy, xq, xs, weights, order, Live{offsets, (int)experts}, rows, cols, dx, dweights, st);
}

}  // namespace fp4dev
