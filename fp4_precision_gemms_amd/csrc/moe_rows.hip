// moe_rows.hip -- tokens to their experts' rows and back.
//
// position[t, j]: the row of token t's j-th choice, anything outside [0, rows) for
// none.
//     gather            row[position[t, j]] = x[t]
//     combine           out[t] = sum_j w[t, j] y[position[t, j]]      (w = 1 if not given)
//     combine's back    dy[position[t, j]] = w[t, j] dout[t],  dw[t, j] = <dout[t], y[position[t, j]]>
// (the gather's gradient is the combination without weights, the gradient of that
// the gather).  All of them walk over the tokens, so that a token's row is read or
// written once, whatever k, and rows of no slot are not touched.  Bound by HBM:
// each row is moved in 16-byte pieces, 64 lanes 1 KB.  Sums in binary32, over j
// in their order, rounded to bf16 once.  16384 rows of 4096 columns of 8192 tokens:
// gathered in 32 us (6.3 TB/s), combined in 33 (6.1), gradients 52 (6.4).
#include "fp4_launch.hpp"
#include "mx_device.hpp"
#include "wave.hpp"

namespace fp4dev {
namespace {

constexpr int kThreads = 256;

// The rows' reads are non-temporal (FAR) where they, or with the gradient's writes
// both, are larger than the 256 MB last-level cache: combining 49152 rows of 4096
// columns 93 to 80 us, behind a product 205 to 179 with it; the gradients of 16384 rows
// of 4096 columns 68 to 55, of 49152 of 2048 88 to 69. Within that size they lose:
// gradients of 4096 rows of 2048 columns 7.9 to 9.1.  (Non-temporal writes: 49152
// gathered rows of 4096 columns 91 to 80, but 16384 32 to 38, and no gain with the
// quantizer that reads them: 209 and 209, 69 and 76.)
constexpr int64_t kFarBytes = INT64_C(1) << 28;

// A token's rows and weights, 64 choices at a time, one a lane: their loads are
// on their way together, and none of them comes behind a store, which it would wait
// for (they return in order).
struct Choices {
    int position;                                      // -1 for none
    float weight;
    __device__ __forceinline__ Choices(const int* positions, const float* weights, int64_t token, int k, int j0,
                                       int64_t rows) {
        const int j = j0 + (threadIdx.x & 63);
        position = j < k ? positions[token * k + j] : -1;
        if (position >= rows) position = -1;
        weight = weights && j < k ? weights[token * k + j] : 1.0f;
    }
    // of choice j0 + j, the same j in every lane
    __device__ __forceinline__ int64_t row(int j) const { return __builtin_amdgcn_readlane(position, j); }
    __device__ __forceinline__ float w(int j) const {
        return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(weight), j));
    }
};

struct Place {
    int64_t token;
    int c0;                                            // first 16-byte piece of this wave's lanes
};

// TPR threads share a token, V pieces each: the workgroup's tokens and the part
// of their rows of nch pieces that this wave has.
template <int TPR, int V>
__device__ __forceinline__ Place place(int nch) {
    constexpr int kTokens = kThreads / TPR;
    const uint32_t b = blockIdx.y * gridDim.x + blockIdx.x;
    const uint32_t parts = (nch + TPR * V - 1) / (TPR * V);
    const uint32_t group = parts == 1 ? b : b / parts, part = b - group * parts;
    return {(int64_t)group * kTokens + wave_uniform(threadIdx.x / TPR), (int)(part * TPR * V + threadIdx.x % TPR)};
}

template <int TPR, int V>
__global__ __launch_bounds__(kThreads) void moe_gather(const uint4* __restrict__ x, int nch,
                                                       const uint8_t* __restrict__ scales, int sb,
                                                       const int* __restrict__ position, int64_t tokens, int k,
                                                       int64_t rows, uint4* __restrict__ out,
                                                       uint8_t* __restrict__ out_scales) {
    const Place at = place<TPR, V>(nch);
    if (at.token >= tokens) return;
    // zero past the row's end: left unset there, the array went to LDS, and every
    // store waited for the one before (128 tokens to 6 rows of 4 KB 11.7 us, now 3.0)
    uint4 v[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        v[i] = at.c0 + i * TPR < nch ? x[at.token * nch + at.c0 + i * TPR] : make_uint4(0, 0, 0, 0);
    // a row's scale bytes, TPR at a time: by the lanes of its first part
    const bool scaled = scales && at.c0 < TPR;
    const uint8_t s0 = scaled && at.c0 < sb ? scales[at.token * sb + at.c0] : 0;
    for (int j0 = 0; j0 < k; j0 += 64) {
        const Choices to(position, nullptr, at.token, k, j0, rows);
        __builtin_amdgcn_s_waitcnt(0x0F70);            // the loads, here once and not after each store
        for (int j = 0; j < 64 && j0 + j < k; ++j) {
            const int64_t r = to.row(j);
            if (r < 0) continue;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (at.c0 + i * TPR < nch) out[r * nch + at.c0 + i * TPR] = v[i];
            if (scaled && at.c0 < sb) out_scales[r * sb + at.c0] = s0;
        }
        // (the same loops in every lane: each asks others for a row)
        for (int first = TPR; scales && first < sb; first += TPR) {
            const int c = at.c0 + first;
            const bool in = scaled && c < sb;
            const uint8_t s = in ? scales[at.token * sb + c] : 0;
            for (int j = 0; j < 64 && j0 + j < k; ++j) {
                const int64_t r = to.row(j);
                if (r >= 0 && in) out_scales[r * sb + c] = s;
            }
        }
    }
}

template <int TPR, int V, bool W, bool FAR>
__global__ __launch_bounds__(kThreads) void moe_combine(const uint4* __restrict__ y, int nch,
                                                        const int* __restrict__ position,
                                                        const float* __restrict__ weights, int64_t tokens, int k,
                                                        int64_t rows, uint4* __restrict__ out) {
    const Place at = place<TPR, V>(nch);
    if (at.token >= tokens) return;
    float acc[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][e] = 0.0f;
    constexpr int kAhead = 4;                          // rows on their way at a time
    Choices from(position, weights, at.token, k, 0, rows);
    for (int j0 = 0; j0 < k; j0 += kAhead) {
        if (j0 && j0 % 64 == 0) from = Choices(position, weights, at.token, k, j0, rows);
        uint4 v[kAhead][V];
        int64_t r[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            r[j] = from.row((j0 + j) % 64);            // -1 past k
            if (r[j] < 0) continue;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (at.c0 + i * TPR < nch) v[j][i] = load16<FAR>(y + r[j] * nch + at.c0 + i * TPR);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (r[j] < 0) continue;
            const float w = from.w((j0 + j) % 64);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (at.c0 + i * TPR >= nch) continue;
                float a[8];
                unpack8(v[j][i], a);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[i][e] = W ? __builtin_fmaf(w, a[e], acc[i][e]) : acc[i][e] + a[e];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (at.c0 + i * TPR < nch) out[at.token * nch + at.c0 + i * TPR] = pack8(acc[i]);
}

// A workgroup (TPR = 256) or a wave (64) takes a token.  dy may be y: a lane has
// read a piece before it writes it, and no other reads it.
template <int TPR, bool FAR>
__global__ __launch_bounds__(kThreads) void moe_combine_back(const uint4* __restrict__ dout, const uint4* y, int nch,
                                                             const int* __restrict__ position,
                                                             const float* __restrict__ weights, int64_t tokens, int k,
                                                             int64_t rows, uint4* dy, float* __restrict__ dweights) {
    constexpr int kTokens = kThreads / TPR, kAhead = 4;
    __shared__ float part[2][kAhead][kThreads / 64];
    const int64_t t = (int64_t)(blockIdx.y * gridDim.x + blockIdx.x) * kTokens + wave_uniform(threadIdx.x / TPR);
    if (t >= tokens) return;                           // a wave of its own, or the whole workgroup
    const int lane = threadIdx.x % TPR, wave = wave_uniform(threadIdx.x >> 6);
    int turn = 0;
    Choices from(position, weights, t, k, 0, rows);
    for (int j0 = 0; j0 < k; j0 += kAhead, turn ^= 1) {
        if (j0 && j0 % 64 == 0) from = Choices(position, weights, t, k, j0, rows);
        int64_t r[kAhead];
        float w[kAhead], dot[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            r[j] = from.row((j0 + j) % 64);            // -1 past k
            w[j] = from.w((j0 + j) % 64);
            dot[j] = 0.0f;
        }
        for (int c = lane; c < nch; c += TPR) {
            const uint4 d = dout[t * nch + c];
            uint4 v[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (r[j] >= 0) v[j] = load16<FAR>(y + r[j] * nch + c);
            float g[8];
            unpack8(d, g);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (r[j] < 0) continue;
                float a[8];
                unpack8(v[j], a);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dot[j] = __builtin_fmaf(g[e], a[e], dot[j]);
                    a[e] = w[j] * g[e];
                }
                dy[r[j] * nch + c] = pack8(a);
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            dot[j] = wave_sum(dot[j]);
            if (TPR > 64 && (threadIdx.x & 63) == 0) part[turn][j][wave] = dot[j];
        }
        // two buffers: the next turn's parts do not overwrite these before the
        // barrier that every reader of these has passed
        if constexpr (TPR > 64) __syncthreads();
        if (lane < kAhead && j0 + lane < k) {
            float s = 0.0f;
            if constexpr (TPR > 64) {
#pragma unroll
                for (int i = 0; i < TPR / 64; ++i) s += part[turn][lane][i];
            } else {
#pragma unroll
                for (int j = 0; j < kAhead; ++j) s = lane == j ? dot[j] : s;
            }
            dweights[t * k + j0 + lane] = s;
        }
    }
}

// Threads of a row: a wave up to 2 KB, else a workgroup.  8192 tokens to 2 rows of 1 KB
// with a wave and with a workgroup: gathered 6.0 and 9.5 us, combined 6.3 and 9.4,
// gradients 11.3 and 14.9; of 4 KB 22.4 and 22.2, 22.2 and 22.2, 38.5 and 35.6; the
// gradients of 16 tokens and 6 rows of 4 KB 6.6 and 3.9.  (Of 2 KB, 8192 tokens: 13.0
// and 12.6, 12.6 and 14.1, 19.2 and 20.3.)
constexpr int kWaveRow = 128;

dim3 grid_for(int64_t tokens, int64_t nch, int tpr, int v) {
    const int64_t per = kThreads / tpr, parts = (nch + tpr * v - 1) / (tpr * v);
    return grid_of((tokens + per - 1) / per * parts, kThreads);
}

}  // namespace

hipError_t launch_moe_gather(const void* x, int64_t row_bytes, const uint8_t* scales, int64_t scale_bytes,
                             const int* position, int64_t tokens, int64_t k, int64_t rows, void* out,
                             uint8_t* out_scales, hipStream_t st) {
    const int64_t nch = row_bytes / 16;
    const bool narrow = nch <= kWaveRow;
    return launch(narrow ? &moe_gather<64, 2> : &moe_gather<256, 2>, grid_for(tokens, nch, narrow ? 64 : 256, 2),
                  dim3(kThreads), st, (const uint4*)x, (int)nch, scales, (int)scale_bytes, position, tokens, (int)k, rows,
                  (uint4*)out, out_scales);
}

hipError_t launch_moe_combine(const void* y, const int* position, const float* weights, int64_t tokens, int64_t k,
                              int64_t rows, int64_t cols, void* out, hipStream_t st) {
    const int64_t nch = cols / 8;
    const bool narrow = nch <= kWaveRow, far = 2 * rows * cols >= kFarBytes;
    auto* run = narrow ? (weights ? &moe_combine<64, 2, true, false> : &moe_combine<64, 2, false, false>)
                       : (weights ? &moe_combine<256, 2, true, false> : &moe_combine<256, 2, false, false>);
    if (far)
        run = narrow ? (weights ? &moe_combine<64, 2, true, true> : &moe_combine<64, 2, false, true>)
                     : (weights ? &moe_combine<256, 2, true, true> : &moe_combine<256, 2, false, true>);
    return launch(run, grid_for(tokens, nch, narrow ? 64 : 256, 2), dim3(kThreads), st, (const uint4*)y, (int)nch,
                  position, weights, tokens, (int)k, rows, (uint4*)out);
}

hipError_t launch_moe_combine_back(const void* dout, const void* y, const int* position, const float* weights,
                                   int64_t tokens, int64_t k, int64_t rows, int64_t cols, void* dy, float* dweights,
                                   hipStream_t st) {
    const int64_t nch = cols / 8;
    const bool narrow = nch <= kWaveRow, far = 4 * rows * cols >= kFarBytes;
    auto* const run = narrow ? (far ? &moe_combine_back<64, true> : &moe_combine_back<64, false>)
                             : (far ? &moe_combine_back<256, true> : &moe_combine_back<256, false>);
    return launch(run, grid_of(narrow ? (tokens + 3) / 4 : tokens, kThreads), dim3(kThreads), st, (const uint4*)dout,
                  (const uint4*)y, (int)nch, position, weights, tokens, (int)k, rows, (uint4*)dy, dweights);
}

}  // namespace fp4dev
