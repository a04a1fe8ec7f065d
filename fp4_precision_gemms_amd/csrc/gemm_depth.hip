// gemm_depth.hip -- the weight gradients dW_e = dY_e^T X_e of experts with up to
// a few hundred tokens each, on small tiles.
//
// The 256 x 256 tiles of gemm_mx.hip take one workgroup per CU and some 10 us
// from the first load to the last store; with a few stages of contraction most
// of that is the pipeline's start and end.  Here a tile is 128 x 128, a wave's
// share 64 x 64, and three workgroups share a CU and cover each other's
// latencies, so nothing is staged through LDS but the output:
//   - both operands' tiled codes go straight to registers, a 32-row fragment
//     of a 64-element k-step being one contiguous kilobyte per wave load; a
//     256-element stage is loaded at once;
//   - V_MFMA_SCALE_F32_32X32X64_F8F6F4 as in gemm_mx.hip, B first, so that the
//     accumulators hold C^T and leave through a wave's own LDS region as row
//     segments, stored non-temporally (32 experts of 2048 x 2048 with 50
//     tokens: 67 us, 88 with plain stores; also where the rows are no whole lines:
//     20 experts of 3200 x 2976 with 400 tokens 122 us against 187), in bf16
//     through V_CVT_PK_BF16_F32 and 16 bytes a lane (50 us; 8 bytes a lane and
//     integer rounding took 63).
// Bound by the output's bytes for few tokens (8 x 14336 x 4096 in bf16, 256
// tokens an expert: 194 us, 4.8 TB/s), by the loads through L1 for many (a wave
// loads 16 KB a stage for 16 MFMAs: 1024 cycles of a CU's L1 for four waves,
// 512 of MFMA).  64 x 128 a wave loads a quarter less but leaves two
// workgroups a CU: 75 us against 70 for 32 x 2048 x 2048 and 100 tokens; so does
// the next stage loaded ahead into registers (51 to 67 us, 400 tokens 79 to 92).
#include "fp4_device.hpp"
#include "fp4_launch.hpp"
#include "grouped.hpp"
#include "mx_mfma.hpp"

namespace fp4dev {
namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kTile = 128;
constexpr int kRow = 64 * 4 + 16;          // a staged row of 64 fp32 columns, padded

// C[e][m, n] for one expert's tile; K: elements per row of the grouped layout.
// Workgroups go round-robin over the 8 XCDs.  From 16 experts on (`per_xcd`) an
// expert's tiles all run on one XCD, whose L2 then holds its operands and joins
// the lines of C that two tiles share (40 experts of 736 x 1120: 21 us, 30 with
// the tiles spread); fewer experts would leave XCDs idle behind the longest, so
// there the column tiles, gx of them (a multiple of 8), are spread (8 experts
// of 14336 x 4096, 1024 tokens: 489 against 603 us).
constexpr int64_t kPerXcdExperts = 16;

template <bool OBF16>
__global__ __launch_bounds__(256) void gemm_mx_depth(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ SA, const uint8_t* __restrict__ B,
    const uint8_t* __restrict__ SB, int64_t M, int64_t N, int64_t K, void* __restrict__ C, int tiles_m, int gx,
    int per_xcd, const GroupArgs ga) {
    __shared__ __attribute__((aligned(16))) uint8_t stage[4][32 * kRow];
    const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    int b = blockIdx.x;
    if (per_xcd) {
        const int per = gx * tiles_m, i = b >> 3;
        b = (i / per * 8 + (b & 7)) * per + i % per;
    }
    const int y = b / gx, e = y / tiles_m;
    if (e >= ga.experts) return;
    const int64_t n0 = (int64_t)(b % gx) * kTile + 64 * (wave >> 1);
    const int64_t m0 = (int64_t)(y % tiles_m) * kTile + 64 * (wave & 1);
    if (n0 >= N || m0 >= M) return;                    // a wave of its own: no barrier below
    const RowRange r = expert_rows(ga.offsets, e, ga.rows);
    const int nk = (int)((r.hi - r.lo + 255) / 256);   // stages
    const int64_t q0 = r.lo / 256 + e;
    const int64_t gstride = K / 32 * 512;              // bytes of a 32-row group of codes
    const int rows = (int)(M - m0 < 64 ? M - m0 : 64), cols = (int)(N - n0 < 64 ? N - n0 : 64);
    // the expert's stages of this wave's two row groups; a group past the last
    // row reads as zero
    const __amdgpu_buffer_rsrc_t ra =
        raw_buffer(A + m0 / 32 * gstride + q0 * 4096, (rows > 32) * gstride + (int64_t)nk * 4096);
    const __amdgpu_buffer_rsrc_t rb =
        raw_buffer(B + n0 / 32 * gstride + q0 * 4096, (cols > 32) * gstride + (int64_t)nk * 4096);

    v16f acc[2][2] = {};
    for (int kt = 0; kt < nk; ++kt) {
        v4i fa[2][4], fb[2][4];
        uint32_t wa[2], wb[2];
        const __amdgpu_buffer_rsrc_t rsa = raw_buffer(SA + ((q0 + kt) * M + m0) * 8, rows * 8);
        const __amdgpu_buffer_rsrc_t rsb = raw_buffer(SB + ((q0 + kt) * N + n0) * 8, cols * 8);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const uint32_t o = (uint32_t)(4 * kt + s) * 1024 + (uint32_t)lane * 16;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fa[i][s] = load16(ra, o + (uint32_t)(i * gstride));
                fb[i][s] = load16(rb, o + (uint32_t)(i * gstride));
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const auto va = __builtin_amdgcn_raw_buffer_load_b64(rsa, (32 * i + l32) * 8, 0, 0);
            const auto vb = __builtin_amdgcn_raw_buffer_load_b64(rsb, (32 * i + l32) * 8, 0, 0);
            wa[i] = stage_scale_word(va[0], va[1], h);
            wb[i] = stage_scale_word(vb[0], vb[1], h);
        }
        // all of the stage's loads before its products (left alone, the
        // compiler keeps one k-step in flight to save registers)
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const v8i a = __builtin_shufflevector(fa[i][s], v4i{0, 0, 0, 0}, 0, 1, 2, 3, 4, 5, 6, 7);
                    const v8i b = __builtin_shufflevector(fb[j][s], v4i{0, 0, 0, 0}, 0, 1, 2, 3, 4, 5, 6, 7);
                    switch (s) {
                        case 0: acc[i][j] = mfma_fp4<0>(b, a, acc[i][j], wb[j], wa[i]); break;
                        case 1: acc[i][j] = mfma_fp4<1>(b, a, acc[i][j], wb[j], wa[i]); break;
                        case 2: acc[i][j] = mfma_fp4<2>(b, a, acc[i][j], wb[j], wa[i]); break;
                        default: acc[i][j] = mfma_fp4<3>(b, a, acc[i][j], wb[j], wa[i]); break;
                    }
                }
    }

    // register t of acc[i][j] in lane l is row m = 32 i + l mod 32, column n =
    // 32 j + 8 (t / 4) + 4 (l / 32) + t mod 4: staged 32 rows at a time, read
    // back and stored 16 bytes a lane (8 bf16 or 4 fp32 of a row; M and N are
    // multiples of 32)
    constexpr int kPer = OBF16 ? 8 : 4, kLanes = 64 / kPer;     // columns a lane, lanes a row
    uint8_t* const reg = stage[wave];
    const int lr = lane / kLanes, c = lane % kLanes * kPer;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (32 * i >= rows) break;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<float4*>(reg + l32 * kRow + (32 * j + 8 * q + 4 * h) * 4) =
                    make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int k = 0; k < kLanes / 2; ++k) {
            const int row = 64 / kLanes * k + lr;
            const v4f* const f = reinterpret_cast<const v4f*>(reg + row * kRow + c * 4);
            if (c >= cols) continue;
            const int64_t at = ((int64_t)e * M + m0 + 32 * i + row) * N + n0 + c;
            if constexpr (OBF16) {
                const v4f a = f[0], b = f[1];
                __builtin_nontemporal_store(
                    v4u{bf16_pair(a[0], a[1]), bf16_pair(a[2], a[3]), bf16_pair(b[0], b[1]), bf16_pair(b[2], b[3])},
                    reinterpret_cast<v4u*>(reinterpret_cast<uint16_t*>(C) + at));
            } else {
                __builtin_nontemporal_store(f[0], reinterpret_cast<v4f*>(reinterpret_cast<float*>(C) + at));
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

}  // namespace

hipError_t launch_gemm_depth_short(const uint8_t* aq, const uint8_t* as, const uint8_t* bq, const uint8_t* bs,
                                   const int* offsets, int64_t experts, int64_t rows, int64_t M, int64_t N, void* c,
                                   int out_bf16, hipStream_t st) {
    const int64_t K = 256 * (rows / 256 + experts), tm = (M + kTile - 1) / kTile;
    const bool per_xcd = experts >= kPerXcdExperts;
    const int64_t cols = (N + kTile - 1) / kTile, gx = per_xcd ? cols : (cols + 7) / 8 * 8;
    const GroupArgs ga{offsets, (int)experts, rows};
    const dim3 grid((unsigned)(gx * tm * (per_xcd ? (experts + 7) / 8 * 8 : experts)));
    auto* const k = out_bf16 ? &gemm_mx_depth<true> : &gemm_mx_depth<false>;
    return launch(k, grid, dim3(256), st, aq, as, bq, bs, M, N, K, c, (int)tm, (int)gx, (int)per_xcd, ga);
}

}  // namespace fp4dev
