// gemm_few.hip -- product of a few rows with MXFP4 weights on gfx950 matrix
// cores: C[m, n] = sum_k a[m, k] w[n, k], for single tokens and small batches,
// dense or with the rows grouped by expert.  The activations are MXFP8 (E4M3,
// row-major) or MXFP4 (the tiled layout of the quantizers).
//
// Bound by the weights, read once from HBM: N K (1/2 + 1/32) bytes.  So the
// split follows the weights:
//   - a workgroup owns 16 NT weight rows n (of one expert) and all of K; its
//     waves take the 256-element k-groups in turn, so that a weight matrix
//     of a few thousand rows already fills the card with loads, and the
//     partial sums meet in LDS, added in a fixed order (no atomics, no second
//     launch);
//   - the weights are the first operand of 16-row MFMAs, so a lane's
//     accumulator is four consecutive n of one row m.  16 rows is the smallest
//     tile there is; rows past the last read as zero (out-of-range buffer
//     loads fetch nothing);
//   - a lane holds block l / 16 of row l mod 16 of each 128-element k-step:
//     16 bytes of a tiled chunk (32 bytes of a row for MXFP8).  The scales of
//     a row's 8 blocks of a k-group are one 8-byte load; the next k-group's
//     loads are issued before this one's products.
//   - MXFP4 activations: one V_MFMA_SCALE_F32_16X16X128_F8F6F4 per k-step,
//     exact products, fp32 sums.  MXFP8 activations: that instruction with an
//     8-bit operand drops what lies 2^-14 below the largest product it adds up
//     (measured with one large and one small product), so both operands are
//     turned into bf16 instead -- exact: E2M1 has 2 significant bits, E4M3
//     has 4, and the block scale is a power of two that the conversion
//     applies -- and take four V_MFMA_F32_16X16X32_BF16.  A k-step's elements
//     are then in another order (the lane's 8 consecutive ones per
//     instruction), the same for both operands.  A tile
//     whose sums are not finite, since the upper end of E8M0 takes elements out
//     of bf16's range (or an input was NaN), is multiplied again, block by block
//     without the scales, which then scale each block's sum in fp32.  (A test of
//     the scales in the loop, with a branch there, took 193 registers for 128 and
//     up to 9 % of the time; this 1 to 2 %, the lift by 2^3: 96 rows over 64
//     experts of 1408 x 2048 15.1 to 15.4 us.  The second time over a tile is slow,
//     24 x 4096 x 14336 with a NaN in one row 145 us for 20.5.)
// More than 16 MT rows (of an expert) are taken one tile after another by the
// workgroups of blockIdx.z in turn; the weights then come from the caches.
#include "fp4_device.hpp"
#include "fp4_launch.hpp"
#include "grouped.hpp"
#include "mx_mfma.hpp"

namespace fp4dev {
namespace {

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// A block's 32 elements times 2^(byte - 127) as bf16, 8 consecutive ones per
// vector.  Byte 255 gives NaN and byte 0 2^-127 (the conversions take the
// exponent field of the scale as it is).
__device__ __forceinline__ void bf16_of_e2m1(const v4i& codes, uint32_t byte, v8bf* out) {
    const float s = __uint_as_float(byte << 23);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const uint32_t w = (uint32_t)codes[p];
        const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
        const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
        const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
        const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
        out[p] = v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
}
// The same for E4M3, times 2^kUp: the smallest element under the smallest scale,
// 2^-9 2^-127, is then bf16's smallest subnormal (which the MFMA does not flush;
// E2M1's, 2^-128, is above it).  What passes bf16's range at the other end (E4M3
// from byte 244 on, E2M1 from 253) becomes an infinity or a NaN.
constexpr int kUp = 3;
__device__ __forceinline__ void bf16_of_e4m3(const v4i* codes, uint32_t byte, v8bf* out) {
    const float s = __uint_as_float((min(byte, 255u - kUp) + kUp) << 23);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const uint32_t lo = (uint32_t)codes[p / 2][2 * (p & 1)], hi = (uint32_t)codes[p / 2][2 * (p & 1) + 1];
        const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false);
        const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true);
        const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false);
        const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true);
        out[p] = v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
}

// acc += w a of one k-step, whatever the scales: its four blocks one after
// another, the lanes of the other blocks giving zeros, so that a product holds
// the one block's sum alone, scaled in fp32 by 2^(ea + ew - 254).
__device__ __forceinline__ void add_unscaled(const v4i& w, int ew, const v4i* a, int ea, v4f& acc) {
    const int lane = threadIdx.x & 63, quad = lane >> 4;
#pragma unroll 1
    for (int blk = 0; blk < 4; ++blk) {
        const int keep = quad == blk ? -1 : 0;
        const v4i codes[2] = {a[0] & keep, a[1] & keep};
        v8bf fw[4], fa[4];
        bf16_of_e2m1(w & keep, 127u, fw);
        bf16_of_e4m3(codes, 127u, fa);
        v4f sum = {};
#pragma unroll
        for (int p = 0; p < 4; ++p) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw[p], fa[p], sum, 0, 0, 0);
        const int em = __shfl(ea, 16 * blk + (lane & 15));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int en = __shfl(ew, 16 * blk + 4 * quad + r);
            acc[r] += em == 255 || en == 255 ? __builtin_nanf("") : __builtin_ldexpf(sum[r], em + en - 254 - kUp);
        }
    }
}

// What one 256-element k-group needs: two 128-element k-steps of MT row tiles
// and NT weight tiles, with their scales.
template <bool A8, int MT, int NT>
struct Group {
    v4i w[NT][2];
    uint2 ws[NT];
    v4i a[MT][2][A8 ? 2 : 1];
    uint2 as[MT];       // MXFP4: the 8 blocks' bytes; MXFP8: this lane's byte of each k-step
};

template <bool A8, int MT, int NT, int W, bool OBF16>
__global__ __launch_bounds__(64 * W) void gemm_few(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ SA, const int* __restrict__ offsets,
    const uint8_t* __restrict__ B, const uint8_t* __restrict__ SB, int64_t rows, int experts, int64_t N,
    int64_t K, void* __restrict__ C) {
    __shared__ v4f part[W][MT * NT][64];
    const int lane = threadIdx.x & 63, l16 = lane & 15, quad = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int e = blockIdx.y;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * NT);
    const int nb = (int)(K / 32), groups = (nb + 7) / 8;

    // this expert's rows [lo, hi), clamped to the operand whatever the offsets say
    int64_t lo = 0, hi = rows, first = 0, arows = rows;
    if (offsets) {
        const RowRange r = expert_rows(offsets, e, rows);
        lo = r.lo;
        hi = r.hi;
        if (lo == hi) return;
        if constexpr (A8) {
            first = lo;
        } else {
            first = (lo / 32 + e) * 32;
            arows = (rows / 32 + experts) * 32;
        }
    }
    const int64_t gstride = (int64_t)nb * 512;         // bytes of a 32-row group of codes
    B += (int64_t)e * ((N + 31) / 32) * gstride;
    SB += (int64_t)e * groups * N * 8;
    const int nleft = (int)((N - n0) < 16 * NT ? (N - n0) : 16 * NT);
    const __amdgpu_buffer_rsrc_t rb =
        raw_buffer(B + (n0 / 32) * gstride, ((n0 + nleft + 31) / 32 - n0 / 32) * gstride);
    uint32_t offb[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int r = (int)(n0 & 31) + 16 * j + l16;
        offb[j] = (uint32_t)((r >> 5) * gstride) + (r & 31) * 16;
    }

    const int64_t mstart = lo + (int64_t)blockIdx.z * (16 * MT);
    for (int64_t m0 = mstart; m0 < hi; m0 += (int64_t)gridDim.z * (16 * MT)) {
        const int mleft = (int)((hi - m0) < 16 * MT ? (hi - m0) : 16 * MT);
        const int64_t p0 = first + (m0 - lo);          // the tile's first row in the A operand
        const __amdgpu_buffer_rsrc_t ra =
            A8 ? raw_buffer(A + p0 * K, (int64_t)mleft * K)
               : raw_buffer(A + (p0 / 32) * gstride, (((p0 & 31) + mleft + 31) / 32) * gstride);
        const __amdgpu_buffer_rsrc_t rsa = raw_buffer(SA + (A8 ? p0 * nb : 0), A8 ? (int64_t)mleft * nb : 0);
        auto load = [&](int g) {
            Group<A8, MT, NT> t;
            const int b0 = 8 * g + quad;
            const bool in[2] = {b0 < nb, b0 + 4 < nb};
            const __amdgpu_buffer_rsrc_t rsb = raw_buffer(SB + ((int64_t)g * N + n0) * 8, nleft * 8);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    t.w[j][s] = load16(rb, in[s] ? offb[j] + (uint32_t)(b0 + 4 * s) * 512 : kOob);
                const auto v = __builtin_amdgcn_raw_buffer_load_b64(rsb, (16 * j + l16) * 8, 0, 0);
                t.ws[j] = make_uint2(v[0], v[1]);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int m = 16 * i + l16;
                if constexpr (A8) {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const uint32_t o = in[s] ? (uint32_t)m * (uint32_t)K + (uint32_t)(b0 + 4 * s) * 32 : kOob;
                        t.a[i][s][0] = load16(ra, o);
                        t.a[i][s][1] = load16(ra, o + 16);
                    }
                    const uint32_t o = (uint32_t)m * (uint32_t)nb + (uint32_t)b0;
                    t.as[i].x = __builtin_amdgcn_raw_buffer_load_b8(rsa, in[0] ? o : kOob, 0, 0);
                    t.as[i].y = __builtin_amdgcn_raw_buffer_load_b8(rsa, in[1] ? o + 4 : kOob, 0, 0);
                } else {
                    const int r = (int)(p0 & 31) + m;
                    const uint32_t o = (uint32_t)((r >> 5) * gstride) + (r & 31) * 16;
#pragma unroll
                    for (int s = 0; s < 2; ++s)
                        t.a[i][s][0] = load16(ra, in[s] ? o + (uint32_t)(b0 + 4 * s) * 512 : kOob);
                    const auto v = __builtin_amdgcn_raw_buffer_load_b64(
                        raw_buffer(SA + ((int64_t)g * arows + p0) * 8, mleft * 8), m * 8, 0, 0);
                    t.as[i] = make_uint2(v[0], v[1]);
                }
            }
            return t;
        };
        v4f acc[MT][NT] = {};
        auto multiply = [&](Group<A8, MT, NT>& t, int g) {
            if (8 * g + 8 > nb) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    t.ws[j] = make_uint2(mask_scale_word(t.ws[j].x, 8 * g, nb),
                                         mask_scale_word(t.ws[j].y, 8 * g + 4, nb));
                if constexpr (!A8)
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        t.as[i] = make_uint2(mask_scale_word(t.as[i].x, 8 * g, nb),
                                             mask_scale_word(t.as[i].y, 8 * g + 4, nb));
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                uint32_t sw[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) sw[j] = (s ? t.ws[j].y : t.ws[j].x) >> (8 * quad);
                if constexpr (A8) {
                    v8bf a[MT][4];
#pragma unroll
                    for (int i = 0; i < MT; ++i) bf16_of_e4m3(t.a[i][s], s ? t.as[i].y : t.as[i].x, a[i]);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        v8bf w[4];
                        bf16_of_e2m1(t.w[j][s], sw[j] & 255u, w);
#pragma unroll
                        for (int p = 0; p < 4; ++p)
#pragma unroll
                            for (int i = 0; i < MT; ++i)
                                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[p], a[i][p], acc[i][j], 0, 0, 0);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const v8i w = __builtin_shufflevector(t.w[j][s], v4i{0, 0, 0, 0}, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            const v8i a = __builtin_shufflevector(t.a[i][s][0], v4i{0, 0, 0, 0}, 0, 1, 2, 3, 4, 5, 6, 7);
                            const uint32_t sa = (s ? t.as[i].y : t.as[i].x) >> (8 * quad);
                            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, acc[i][j], 4, 4, 0,
                                                                                         (int)sw[j], 0, (int)sa);
                        }
                    }
                }
            }
        };
        // tile q by add_unscaled, a k-group's sum after another
        auto tile_unscaled = [&](int q) {
            v4f total = {};
            if constexpr (A8) {
                const int m = 16 * (q / NT) + l16, n = 16 * (q % NT) + l16, r = (int)(n0 & 31) + n;
                const uint32_t offw = (uint32_t)((r >> 5) * gstride) + (r & 31) * 16;
#pragma unroll 1
                for (int g = 0; g < groups; ++g) {
                    const __amdgpu_buffer_rsrc_t rsb = raw_buffer(SB + ((int64_t)g * N + n0) * 8, nleft * 8);
                    v4f sum = {};
#pragma unroll 1
                    for (int s = 0; s < 2; ++s) {
                        const int b = 8 * g + 4 * s + quad;
                        const bool in = b < nb;
                        const uint32_t offm = in ? (uint32_t)m * (uint32_t)K + (uint32_t)b * 32 : kOob;
                        const v4i codes[2] = {load16(ra, offm), load16(ra, offm + 16)};
                        const int ea = __builtin_amdgcn_raw_buffer_load_b8(
                            rsa, in ? (uint32_t)m * (uint32_t)nb + (uint32_t)b : kOob, 0, 0);
                        const int ew = in ? __builtin_amdgcn_raw_buffer_load_b8(rsb, n * 8 + (b & 7), 0, 0) : 0;
                        add_unscaled(load16(rb, in ? offw + (uint32_t)b * 512 : kOob), ew, codes, ea, sum);
                    }
                    total += sum;
                }
            }
            return total;
        };
        int g = wave;
        if (g < groups) {
            Group<A8, MT, NT> t = load(g);
            for (; g + W < groups; g += W) {
                Group<A8, MT, NT> next = load(g + W);
                multiply(t, g);
                t = next;
            }
            multiply(t, g);
        }
        // join the waves' sums: tile (i, j) is added up by wave (i NT + j) mod W
        if (m0 != mstart) __syncthreads();             // the previous tile's sums have been read
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) part[wave][i * NT + j][lane] = acc[i][j];
        __syncthreads();
        for (int q = wave; q < MT * NT; q += W) {
            v4f s = part[0][q][lane];
#pragma unroll
            for (int w = 1; w < W; ++w) s += part[w][q][lane];
            if constexpr (A8) {
                bool finite = true;
#pragma unroll
                for (int r = 0; r < 4; ++r) finite &= __builtin_fabsf(s[r]) < __builtin_inff();
                s *= 1.0f / (1 << kUp);
                if (__builtin_expect(__any(!finite), 0)) s = tile_unscaled(q);
            }
            const int m = 16 * (q / NT) + l16, n = 16 * (q % NT) + 4 * quad;
            if (m >= mleft || n >= nleft) continue;
            const int64_t at = (m0 + m) * N + n0 + n;
            const bool whole = n + 4 <= nleft && (N & 3) == 0;
            if constexpr (OBF16) {
                uint16_t* p = reinterpret_cast<uint16_t*>(C) + at;
                if (whole) {
                    *reinterpret_cast<uint2*>(p) = make_uint2(bf16_pair(s[0], s[1]), bf16_pair(s[2], s[3]));
                } else {
                    for (int k = 0; k < 4 && n + k < nleft; ++k) p[k] = (uint16_t)bf16_rne(s[k]);
                }
            } else {
                float* p = reinterpret_cast<float*>(C) + at;
                if (whole) {
                    *reinterpret_cast<v4f*>(p) = s;
                } else {
                    for (int k = 0; k < 4 && n + k < nleft; ++k) p[k] = s[k];
                }
            }
        }
    }
}

template <bool A8, int MT, int NT, int W>
hipError_t launch_few(const uint8_t* a, const uint8_t* as, const int* offsets, const uint8_t* w, const uint8_t* ws,
                      int64_t rows, int64_t experts, int64_t N, int64_t K, void* c, int out_bf16, hipStream_t st) {
    // Row tiles go to workgroups of their own up to kFewWorkgroups in all: one
    // after another, 1 expert of 64 columns, K = 1024 and 16384 rows took 323 us,
    // so 7.4; 1024 columns, K = 4096, 1024 rows 40 and 13.3.  (Up to 256 that is
    // 12.8, but 64 columns 9.1; up to 2048 14.2 and 6.7.)
    constexpr int64_t kFewWorkgroups = 512;
    const int64_t x = (N + 16 * NT - 1) / (16 * NT), tiles = ((rows + experts - 1) / experts + 16 * MT - 1) / (16 * MT);
    const int64_t fill = kFewWorkgroups / (x * experts), z = fill < 1 ? 1 : fill < tiles ? fill : tiles;
    const dim3 grid((unsigned)x, (unsigned)experts, (unsigned)z);
    return out_bf16 ? launch(&gemm_few<A8, MT, NT, W, true>, grid, dim3(64 * W), st, a, as, offsets, w, ws, rows,
                             (int)experts, N, K, c)
                    : launch(&gemm_few<A8, MT, NT, W, false>, grid, dim3(64 * W), st, a, as, offsets, w, ws, rows,
                             (int)experts, N, K, c);
}

template <bool A8>
hipError_t choose(const uint8_t* a, const uint8_t* as, const int* offsets, const uint8_t* w, const uint8_t* ws,
                  int64_t rows, int64_t experts, int64_t N, int64_t K, void* c, int out_bf16, hipStream_t st) {
#define FP4_FEW(MT, NT, W) return launch_few<A8, MT, NT, W>(a, as, offsets, w, ws, rows, experts, N, K, c, out_bf16, st)
#define FP4_FEW_ROWS(NT, W)                      \
    do {                                         \
        if (each <= 16) FP4_FEW(1, NT, W);       \
        if (each <= 32) FP4_FEW(2, NT, W);       \
        FP4_FEW(4, A8 ? 1 : NT, W);              \
    } while (0)
    // Row tiles by the rows an expert has on average.  Weight rows and waves
    // per workgroup: 32 and 4 where that makes 256 workgroups (96 rows over 64
    // experts of 1408 x 2048: 15.8 us, against 27.4 with 16 and 8; 1 x 14336 x
    // 4096: 8.1 and 8.8), else 16 and 8 (24 x 4096 x 14336: 8.0 us, 9.4 with 32
    // rows and 10.0 with 4 waves).  Fewer waves where the contraction does not
    // have two k-groups for each (50 rows an expert, 40 experts of 1120 x 736:
    // 12.3 us with two, 14.3 with four).  MXFP8 with four row tiles has no
    // registers for a second weight tile.
    const int64_t each = (rows + experts - 1) / experts, groups = (K + 255) / 256;
    if ((N + 31) / 32 * experts >= 256) {
        if (groups >= 8) FP4_FEW_ROWS(2, 4);
        FP4_FEW_ROWS(2, 2);
    }
    if (groups >= 16) FP4_FEW_ROWS(1, 8);
    if (groups >= 8) FP4_FEW_ROWS(1, 4);
    FP4_FEW_ROWS(1, 2);
#undef FP4_FEW_ROWS
#undef FP4_FEW
}

}  // namespace

hipError_t launch_gemm_few(const uint8_t* a, const uint8_t* as, int a_e4m3, const int* offsets, const uint8_t* w,
                           const uint8_t* ws, int64_t rows, int64_t experts, int64_t N, int64_t K, void* c,
                           int out_bf16, hipStream_t st) {
    return a_e4m3 ? choose<true>(a, as, offsets, w, ws, rows, experts, N, K, c, out_bf16, st)
                  : choose<false>(a, as, offsets, w, ws, rows, experts, N, K, c, out_bf16, st);
}

}  // namespace fp4dev
