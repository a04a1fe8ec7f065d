// norm_mx.hip -- root-mean-square norm that adds the residual and leaves its
// output quantized, and its backward pass.
//
// Forward, per row of C elements:
//     h = bf16(x + residual)                 (binary32 sum, one rounding; h = x without a residual)
//     r = fl32(1 / sqrt(sum h^2 / C + eps))  (binary64)
//     y = fl32(fl32(h r) w)
// and y goes to 32-element blocks with one E8M0 scale each, either MXFP4
// (E2M1, scale floor(log2 max|y|) - 2) or MXFP8 (E4M3, floor(log2 max|y|) - 8).
// The sum is held in binary64 so that r, and with it every code, does not
// depend on the order of the sum: an FP4 code next to a rounding border would
// otherwise change with the launch shape.  A square of a bf16 value is exact in
// binary64, so the sum is off by 2^-53 an addition at most.  y itself is not
// rounded to bf16 before the quantization: one rounding instead of two.
//
// Bound by HBM: 2 bytes read per input, 2 written for h, 1 (MXFP8) or 1/2
// (MXFP4) for the codes.  Each element is read once and kept in registers
// (bf16 pairs) across the reduction.
//
// Backward, with g = dy w, n = h r and c = sum_j g_j n_j over the row:
//     dx = r (g - n c / C) (+ dh)            (dh: the gradient that reaches h past the norm)
//     dw = sum over rows of dy n
// By way of n, of order one, and not of h and r^3, which leave binary32 when
// the row's scale does not: rows of 1e-13 or 1e13 already.
// (the quantization is passed straight through).  A workgroup walks over rows
// with its columns' part of dw in registers, so dy and h are read once; the
// parts of all workgroups are summed in a fixed order by a second kernel.
#include "fp4_launch.hpp"
#include "mx_device.hpp"

namespace fp4dev {
namespace {

// a wave's sum, in every lane
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
    return v;
}

__device__ __forceinline__ void unpack8(const uint4& w, float* a) {
    a[0] = bf16_lo(w.x); a[1] = bf16_hi(w.x); a[2] = bf16_lo(w.y); a[3] = bf16_hi(w.y);
    a[4] = bf16_lo(w.z); a[5] = bf16_hi(w.z); a[6] = bf16_lo(w.w); a[7] = bf16_hi(w.w);
}

__device__ __forceinline__ uint4 pack8(const float* a) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16_pair(a[2 * i], a[2 * i + 1]);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Codes of 8 values under scale byte `byte` (not 255) as E4M3: the hardware
// conversion rounds to nearest even but turns what lies beyond 464 into NaN,
// so the scaled value is clamped to +-448 first.
__device__ __forceinline__ uint2 encode8_e4m3(const float* y, uint32_t byte) {
    const float inv = inv_scale_from_e8m0(byte);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __builtin_amdgcn_fmed3f(y[i] * inv, -448.0f, 448.0f);
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
    return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// The row block of workgroup b of n.  Workgroups go round-robin over the 8
// XCDs, each with an L2 of its own; here B consecutive row blocks (32 rows) run
// on one XCD, so that the 16-byte code pieces and 8-byte scale groups of
// neighbouring rows meet in one L2 and leave as whole lines (8192 x 4096 to
// MXFP4 43.6 us, 52.8 with the rows in launch order; 8192 x 8192 82.9 and 98.9).
template <int B>
__device__ __forceinline__ unsigned row_block(unsigned b, unsigned n) {
    if (b >= n / (8 * B) * (8 * B)) return b;
    const unsigned xcd = b & 7, i = b >> 3;
    return (i / B) * (8 * B) + xcd * B + i % B;
}

// TPR threads share a row, RPB rows per workgroup; a lane owns V chunks of 8
// consecutive elements, so four adjacent lanes hold one 32-element block.
// (x, res and h are not __restrict__: h may be x or res itself; every lane
// writes only the chunks it has read.)
template <int TPR, int RPB, int V, bool RES, bool E4M3>
__global__ __launch_bounds__(TPR * RPB) void rmsnorm_quant(
    const uint4* x, const uint4* res, const uint4* __restrict__ weight, double eps, int64_t rows,
    int cols, uint4* h, float* __restrict__ rstd, uint4* __restrict__ y, uint8_t* __restrict__ codes,
    uint8_t* __restrict__ scales) {
    static_assert(TPR == 64 || RPB == 1, "rows that share a workgroup are a wave each");
    constexpr int kWaves = TPR / 64;
    const int t = threadIdx.x % TPR, nch = cols / 8, q = t & 3;
    const int64_t row =
        (int64_t)row_block<32 / RPB>(blockIdx.y * gridDim.x + blockIdx.x, gridDim.x * gridDim.y) * RPB + threadIdx.x / TPR;
    if (row >= rows) return;                           // a wave of its own, or the whole workgroup
    const int64_t base = row * nch;
    uint4 v[V], wv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * TPR + t;
        v[i] = c < nch ? x[base + c] : make_uint4(0, 0, 0, 0);
    }
    if constexpr (RES) {
        uint4 rv[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * TPR + t;
            rv[i] = c < nch ? res[base + c] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * TPR + t;
            wv[i] = c < nch ? weight[c] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float a[8], b[8];
            unpack8(v[i], a);
            unpack8(rv[i], b);
#pragma unroll
            for (int k = 0; k < 8; ++k) a[k] += b[k];
            v[i] = pack8(a);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * TPR + t;
            wv[i] = c < nch ? weight[c] : make_uint4(0, 0, 0, 0);
        }
    }
    if (h) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * TPR + t;
            if (c < nch) h[base + c] = v[i];
        }
    }
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float a[8];
        unpack8(v[i], a);
#pragma unroll
        for (int k = 0; k < 8; ++k) s = __builtin_fma((double)a[k], (double)a[k], s);
    }
    s = wave_sum(s);
    if constexpr (kWaves > 1) {
        __shared__ double part[kWaves];
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
        __syncthreads();
        s = 0.0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) s += part[i];
    }
    const float r = (float)(1.0 / __builtin_sqrt(s / (double)cols + eps));
    if (rstd && t == 0) rstd[row] = r;
    const int nb = cols / 32;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * TPR + t;
        if (c >= nch) continue;                        // uniform per quad: cols % 32 == 0
        float a[8], w[8];
        unpack8(v[i], a);
        unpack8(wv[i], w);
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k] = (a[k] * r) * w[k];
        if (y) y[base + c] = pack8(a);
        uint32_t m = max_abs_bits<8>(a);
        m = max(m, quad_xor1(m));
        m = max(m, quad_xor2(m));
        const int b = c >> 2;
        if constexpr (E4M3) {
            const uint32_t byte = e8m0_from_amax_bits_e4m3(m);
            uint2 word = make_uint2(0, 0);
            if (byte != 255u) word = encode8_e4m3(a, byte);
            reinterpret_cast<uint2*>(codes)[base + c] = word;
            if (q == 0) scales[row * nb + b] = (uint8_t)byte;
        } else {
            const uint32_t byte = e8m0_from_amax_bits(m);
            uint32_t word = 0;
            if (byte != 255u) {
                const uint4 z = make_uint4(0, 0, 0, 0);
                word = byte != 0u ? encode8_hw(a, byte) : encode8_sw<false>(a, byte, z, z);
            }
            *reinterpret_cast<uint32_t*>(codes + tiled_offset(row, b, nb) + 4 * q) = word;
            if (q == 0) scales[((int64_t)(b >> 3) * rows + row) * 8 + (b & 7)] = (uint8_t)byte;
        }
    }
}

template <int TPR, int RPB, int V>
hipError_t launch_norm(const void* x, const void* res, const void* w, double eps, int64_t rows, int64_t cols,
                       int e4m3, void* h, float* rstd, void* y, uint8_t* codes, uint8_t* scales, hipStream_t st) {
    const dim3 grid = grid_of((rows + RPB - 1) / RPB, TPR * RPB), block(TPR * RPB);
#define FP4_NORM(RES, E)                                                                                \
    return launch(&rmsnorm_quant<TPR, RPB, V, RES, E>, grid, block, st, (const uint4*)x, (const uint4*)res, \
                  (const uint4*)w, eps, rows, (int)cols, (uint4*)h, rstd, (uint4*)y, codes, scales)
    if (res) {
        if (e4m3) FP4_NORM(true, true);
        FP4_NORM(true, false);
    }
    if (e4m3) FP4_NORM(false, true);
    FP4_NORM(false, false);
#undef FP4_NORM
}

// ---------------------------------------------------------------- backward
// One workgroup walks over rows blockIdx.x, + gridDim.x, ...; the next row's
// loads are issued before this row's reduction (not with 1024 threads of 4
// chunks each, which have no registers for it).
template <int TPR, int V, bool DH>
__global__ __launch_bounds__(TPR) void rmsnorm_back(
    const uint4* __restrict__ dy, const uint4* __restrict__ h, const uint4* __restrict__ weight,
    const float* __restrict__ rstd, const uint4* dh, int64_t rows, int cols, uint4* dx,
    float* __restrict__ parts) {
    constexpr int kWaves = TPR / 64;
    constexpr bool kAhead = TPR * V < 4096;
    __shared__ float part[2][kWaves];
    const int t = threadIdx.x, nch = cols / 8;
    const float inv_cols = 1.0f / (float)cols;
    float acc[V][8];
    uint4 wv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * TPR + t;
        wv[i] = c < nch ? weight[c] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[i][k] = 0.0f;
    }
    uint4 gv[V], hv[V], ev[V];
    float r = 0.0f;
    auto load = [&](int64_t row) {
        const int64_t base = row * nch;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * TPR + t;
            gv[i] = c < nch ? dy[base + c] : make_uint4(0, 0, 0, 0);
            hv[i] = c < nch ? h[base + c] : make_uint4(0, 0, 0, 0);
            if constexpr (DH) ev[i] = c < nch ? dh[base + c] : make_uint4(0, 0, 0, 0);
        }
        r = rstd[row];
    };
    int64_t row = blockIdx.x;                          // gridDim.x <= rows
    if constexpr (kAhead) load(row);
    for (int turn = 0; row < rows; turn ^= 1) {
        if constexpr (!kAhead) load(row);
        uint4 g1[V], h1[V], e1[V];
        const float r1 = r;
#pragma unroll
        for (int i = 0; i < V; ++i) { g1[i] = gv[i]; h1[i] = hv[i]; if constexpr (DH) e1[i] = ev[i]; }
        const int64_t next = row + gridDim.x;
        if (kAhead && next < rows) load(next);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float a[8], b[8], w[8];
            unpack8(g1[i], a);
            unpack8(h1[i], b);
            unpack8(wv[i], w);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                b[k] *= r1;
                s += (a[k] * w[k]) * b[k];
                acc[i][k] += a[k] * b[k];
            }
        }
        s = wave_sum(s);
        if constexpr (kWaves > 1) {
            // two buffers: the next row's parts do not overwrite these before
            // the barrier that every reader of these has passed
            if ((t & 63) == 0) part[turn][t >> 6] = s;
            __syncthreads();
            s = 0.0f;
#pragma unroll
            for (int i = 0; i < kWaves; ++i) s += part[turn][i];
        }
        s *= inv_cols;
        const int64_t base = row * nch;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * TPR + t;
            if (c >= nch) continue;
            float a[8], b[8], w[8], e[8];
            unpack8(g1[i], a);
            unpack8(h1[i], b);
            unpack8(wv[i], w);
            if constexpr (DH) unpack8(e1[i], e);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                a[k] = r1 * (a[k] * w[k] - (b[k] * r1) * s);
                if constexpr (DH) a[k] += e[k];
            }
            dx[base + c] = pack8(a);
        }
        row = next;
    }
    float4* out = reinterpret_cast<float4*>(parts + (int64_t)blockIdx.x * cols);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * TPR + t;
        if (c >= nch) continue;
        out[2 * c] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        out[2 * c + 1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
    }
}

// dw[c] = sum of n rows of parts[n, cols]: 32 columns per workgroup, 32 slices
// of the rows, joined in a fixed order.
__global__ __launch_bounds__(1024) void sum_parts(const float* __restrict__ parts, int n, int cols,
                                                  float* __restrict__ dw) {
    __shared__ float part[32][32];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
    float s = 0.0f;                                    // cols % 32 == 0: c < cols
    for (int i = slice; i < n; i += 256) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = i + 32 * k < n ? parts[(int64_t)(i + 32 * k) * cols + c] : 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) s += v[k];
    }
    part[slice][threadIdx.x & 31] = s;
    __syncthreads();
    if (slice == 0) {
        s = 0.0f;
#pragma unroll
        for (int k = 0; k < 32; ++k) s += part[k][threadIdx.x];
        dw[c] = s;
    }
}

template <int TPR, int V>
hipError_t launch_back(const void* dy, const void* h, const void* w, const float* rstd, const void* dh,
                       int64_t rows, int64_t cols, void* dx, float* parts, int64_t n, hipStream_t st) {
    if (dh)
        return launch(&rmsnorm_back<TPR, V, true>, dim3((unsigned)n), dim3(TPR), st, (const uint4*)dy,
                      (const uint4*)h, (const uint4*)w, rstd, (const uint4*)dh, rows, (int)cols, (uint4*)dx, parts);
    return launch(&rmsnorm_back<TPR, V, false>, dim3((unsigned)n), dim3(TPR), st, (const uint4*)dy,
                  (const uint4*)h, (const uint4*)w, rstd, (const uint4*)dh, rows, (int)cols, (uint4*)dx, parts);
}

}  // namespace

hipError_t launch_rmsnorm_quant(const void* x, const void* res, const void* w, double eps, int64_t rows,
                                int64_t cols, int e4m3, void* h, float* rstd, void* y, uint8_t* codes,
                                uint8_t* scales, hipStream_t st) {
    const int64_t nch = cols / 8;
#define FP4_ROW(TPR, RPB, V) \
    return launch_norm<TPR, RPB, V>(x, res, w, eps, rows, cols, e4m3, h, rstd, y, codes, scales, st)
    // two 16-byte loads of each input per lane; a wave per row (four rows a
    // workgroup, no barrier) up to 1024 columns.  Measured to MXFP8 with a
    // residual, rows in launch order: 8192 x 4096 with 128, 256 and 512 threads
    // a row 45.7, 43.7 and 44.3 us (a wave a row 49), 8192 x 8192 with 256 and
    // 512 84.4 and 81.6, 8192 x 2048 with 64, 128 and 256 24.8, 23.4 and 24.1.
    if (nch <= 64) FP4_ROW(64, 4, 1);
    if (nch <= 128) FP4_ROW(64, 4, 2);
    if (nch <= 256) FP4_ROW(128, 1, 2);
    if (nch <= 512) FP4_ROW(256, 1, 2);
    if (nch <= 1024) FP4_ROW(512, 1, 2);
    if (nch <= 2048) FP4_ROW(1024, 1, 2);
    FP4_ROW(1024, 1, 4);
#undef FP4_ROW
}

// Workgroups of the backward pass: one per CU keeps the parts of dw, and the
// kernel that adds them up, small (8192 x 8192: 256 parts 97 + 5 us, 1024 parts
// 103 + 10); narrow rows, whose workgroups are a few waves, take more of them.
// Beyond 16384 columns a lane holds four chunks in 128 registers and spills 64 to
// 79 of them, which then bounds the kernel: 2048 x 32768 220 us (1.8 TB/s), with
// dh 295; 2048 x 16384 37 and 50 (5.4 TB/s).
int64_t rmsnorm_back_parts(int64_t rows, int64_t cols) {
    const int64_t most = cols <= 1024 ? 1024 : cols <= 2048 ? 512 : 256;
    return rows < most ? rows : most;
}

hipError_t launch_rmsnorm_back(const void* dy, const void* h, const void* w, const float* rstd, const void* dh,
                               int64_t rows, int64_t cols, void* dx, float* dw, float* parts, hipStream_t st) {
    const int64_t nch = cols / 8, n = rmsnorm_back_parts(rows, cols);
    hipError_t e;
    if (nch <= 128) e = launch_back<128, 1>(dy, h, w, rstd, dh, rows, cols, dx, parts, n, st);
    else if (nch <= 256) e = launch_back<256, 1>(dy, h, w, rstd, dh, rows, cols, dx, parts, n, st);
    else if (nch <= 512) e = launch_back<512, 1>(dy, h, w, rstd, dh, rows, cols, dx, parts, n, st);
    else if (nch <= 1024) e = launch_back<512, 2>(dy, h, w, rstd, dh, rows, cols, dx, parts, n, st);
    else if (nch <= 2048) e = launch_back<512, 4>(dy, h, w, rstd, dh, rows, cols, dx, parts, n, st);
    else e = launch_back<1024, 4>(dy, h, w, rstd, dh, rows, cols, dx, parts, n, st);
    if (e != hipSuccess) return e;
    return launch(&sum_parts, dim3((unsigned)(cols / 32)), dim3(1024), st, (const float*)parts, (int)n, (int)cols, dw);
}

}  // namespace fp4dev
