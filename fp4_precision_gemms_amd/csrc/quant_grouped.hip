// quant_grouped.hip -- MXFP4 quantization of rows grouped by expert, along
// cols (the operands of the forward and Dgrad products), along rows (those of
// Wgrad: each expert's tokens in stages of 256 of their own, the last one
// filled up with zeros) or both from one read.
//
// Bound by HBM like the quantizers without groups, and built the same way: a
// workgroup takes one or two consecutive 32-row units x 256 columns, global ->
// LDS by DMA in 512-byte row segments (16-byte chunks swizzled by row mod 4 so
// that both the column reads and the row reads are free of bank conflicts).
// A unit's rows belong to one expert (grouped.hpp); rows past its last one are
// out-of-range loads and read as zero, so that the rows output holds whole
// 256-token stages, zeros behind an expert's last token, and Wgrad has no tail.
// Along rows a thread owns a column and its 32 values of the unit, along cols
// one 32-element block of a row.  [16384, 4096] over 8 experts along cols 37 us
// (4.6 TB/s), along rows 40; [16384, 14336] both ways 142 us (5.0 TB/s).
#include "fp4_launch.hpp"
#include "grouped.hpp"
#include "mx_device.hpp"

namespace fp4dev {
namespace {

typedef __attribute__((address_space(3))) void lds_void_t;

constexpr int kCols = 256;
constexpr uint32_t kOob = 0x80000000u;

struct Rotation {
    uint32_t sign_word;
    float norm;
};

// HADN: rotation size along the axis (0 = none); with both outputs it is the
// rows output's and the cols output is not rotated.
// A workgroup takes kUnits units at a time, kTurns times.
template <int HADN, bool SR, bool ROWS, bool COLS, int kUnits, int kTurns>
__global__ __launch_bounds__(kCols) void quant_grouped(
    const uint16_t* __restrict__ x, const int* __restrict__ offsets, int experts, int64_t rows, int cols,
    Rotation rot, uint64_t sr_rows, uint64_t sr_cols, uint8_t* __restrict__ codes_r, uint8_t* __restrict__ scales_r,
    uint8_t* __restrict__ codes_c, uint8_t* __restrict__ scales_c) {
    __shared__ __attribute__((aligned(1024))) uint16_t tile[kUnits][32 * kCols];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // units of the cols output, blocks of the rows output
    const int64_t units = rows / 32 + experts, blocks = 8 * (rows / 256 + experts), nbc = cols / 32;
    const int gx = (cols + kCols - 1) / kCols;
    // (workgroups past the last unit find nothing live)
    const uint32_t wg = blockIdx.y * gridDim.x + blockIdx.x;
    const int c0 = (int)(wg % gx) * kCols;
    const int64_t q0 = (int64_t)(wg / gx) * (kUnits * kTurns);
    // units of one stage belong to one expert
    const int stage_expert = ROWS ? expert_of_unit<256>(offsets, experts, rows, q0 / 8) : -1;
    for (int turn = 0; turn < kTurns; ++turn) {
        const int64_t p0 = q0 + turn * kUnits;
        int64_t r0[kUnits], local[kUnits];
        int expert[kUnits], left[kUnits];                  // rows of the unit
        bool live[kUnits];                                 // whether anything is written for it
#pragma unroll
        for (int t = 0; t < kUnits; ++t) {
            const int64_t p = p0 + t;
            left[t] = 0;
            r0[t] = local[t] = 0;
            live[t] = false;
            if (ROWS) expert[t] = stage_expert;
            else expert[t] = p < units ? expert_of_unit<32>(offsets, experts, rows, p) : -1;
            if (expert[t] < 0) continue;
            const RowRange rr = expert_rows(offsets, expert[t], rows);
            local[t] = p - (ROWS ? 8 * (rr.lo / 256 + expert[t]) : rr.lo / 32 + expert[t]);
            r0[t] = rr.lo + 32 * local[t];
            left[t] = rr.hi - r0[t] >= 32 ? 32 : rr.hi > r0[t] ? (int)(rr.hi - r0[t]) : 0;
            left[t] = __builtin_amdgcn_readfirstlane(left[t]);
            live[t] = left[t] > 0 || (ROWS && local[t] / 8 * 256 < rr.hi - rr.lo);
        }
        if (!live[0] && !live[kUnits - 1]) return;     // nor is anything after them in the stage
#pragma unroll
        for (int t = 0; t < kUnits; ++t) {
            if (left[t] == 0) continue;
            const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
                (void*)(x + r0[t] * cols), (short)0, left[t] * cols * 2, 0x00020000);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int j = wave * 4 + k, row = 2 * j + (lane >> 5);
                const int chunk = (lane & 31) ^ (row & 3);
                const uint32_t o = (uint32_t)(row * cols + c0) * 2 + chunk * 16;
                const bool in = row < left[t] && c0 + 8 * chunk < cols;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void_t*)((uint8_t*)tile[t] + j * 1024), 16,
                                                         in ? o : kOob, 0, 0, 0);
            }
        }
        __builtin_amdgcn_s_waitcnt(0x0F70);                // the DMA has landed
        __syncthreads();
        int colpos[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) colpos[q] = (((tid >> 3) ^ q) << 3) | (tid & 7);
        const int col = c0 + tid;
        uint32_t bytes = 0;
#pragma unroll
        for (int t = 0; t < kUnits; ++t) {
            if (!live[t]) continue;
            if constexpr (ROWS) {
                if (col < cols) {
                    const int64_t p = p0 + t;
                    uint32_t wd[4] = {}, byte = 0;             // what a block of zeros gives
                    if (left[t] > 0) {
                        float a[32];
#pragma unroll
                        for (int r = 0; r < 32; ++r)
                            a[r] = __uint_as_float((uint32_t)tile[t][r * kCols + colpos[r & 3]] << 16);
                        const uint64_t g = ((uint64_t)col * (uint64_t)(32 * blocks) + (uint64_t)(32 * p)) >> 2;
                        byte = quant_block32<HADN, SR>(a, rot.sign_word, rot.norm, sr_rows, g, wd);
                    }
                    *reinterpret_cast<uint4*>(codes_r + tiled_offset(col, p, blocks)) =
                        make_uint4(wd[0], wd[1], wd[2], wd[3]);
                    bytes |= byte << (8 * t);
                }
            }
            if constexpr (COLS) {
                const int grp = lane >> 4;
                const int r = 8 * wave + 4 * (grp & 1) + ((lane >> 2) & 3), b = 4 * (grp >> 1) + (lane & 3);
                const int64_t cb = c0 + 32 * b;
                if (r < left[t] && cb < cols) {
                    float a[32];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint4 v =
                            *reinterpret_cast<const uint4*>(&tile[t][r * kCols + (((4 * b + k) ^ (r & 3)) << 3)]);
                        a[8 * k + 0] = bf16_lo(v.x); a[8 * k + 1] = bf16_hi(v.x);
                        a[8 * k + 2] = bf16_lo(v.y); a[8 * k + 3] = bf16_hi(v.y);
                        a[8 * k + 4] = bf16_lo(v.z); a[8 * k + 5] = bf16_hi(v.z);
                        a[8 * k + 6] = bf16_lo(v.w); a[8 * k + 7] = bf16_hi(v.w);
                    }
                    uint32_t wd[4];
                    const uint64_t g = ((uint64_t)(r0[t] + r) * (uint64_t)cols + (uint64_t)cb) >> 2;
                    const uint32_t byte =
                        quant_block32<ROWS ? 0 : HADN, SR>(a, rot.sign_word, rot.norm, sr_cols, g, wd);
                    const int64_t first = r0[t] - 32 * local[t];          // the expert's first row
                    const int64_t pr = 32 * (first / 32 + expert[t] + local[t]) + r, blk = cb / 32;
                    *reinterpret_cast<uint4*>(codes_c + tiled_offset(pr, blk, nbc)) =
                        make_uint4(wd[0], wd[1], wd[2], wd[3]);
                    scales_c[((blk >> 3) * (32 * units) + pr) * 8 + (blk & 7)] = (uint8_t)byte;
                }
            }
        }
        // a column's scales: all blocks are written (a stage is written whole)
        if constexpr (ROWS)
            if (col < cols) {
                uint8_t* const s = scales_r + ((p0 >> 3) * cols + col) * 8 + (p0 & 7);
                if constexpr (kUnits == 2) *reinterpret_cast<uint16_t*>(s) = (uint16_t)bytes;
                else *s = (uint8_t)bytes;
            }
        if (kTurns > 1) __syncthreads();               // the tile has been read
    }
}

// Units per workgroup: two (pairs of codes and scale bytes leave together),
// one where that leaves CUs idle and a unit's latency is the time (1999 rows
// over 40 experts, 736 and 1120 columns: 8.2 and 6.8 us, 14.3 and 15.1 with two).
// Along rows, where most units of many experts are the zeros that fill their
// stages, a workgroup takes a whole stage, two units a turn: 8000 rows over 128
// experts, 2048 columns, both ways 22 us, 35 without; 4000 over 64 17 and 20; but
// 8000 over 64, 4096 columns 31.6 and 29.8.
constexpr int64_t kFewWorkgroups = 1024;

template <int HADN, bool SR, bool ROWS, bool COLS>
hipError_t launch_one(const void* x, const int* offsets, int64_t experts, int64_t rows, int64_t cols, Rotation rot,
                      uint64_t sr_rows, uint64_t sr_cols, uint8_t* cr, uint8_t* sr, uint8_t* cc, uint8_t* sc,
                      hipStream_t st) {
    const int64_t units = ROWS ? 8 * (rows / 256 + experts) : rows / 32 + experts;
    const int64_t gx = (cols + kCols - 1) / kCols;
    if constexpr (ROWS)
        if (rows < 96 * experts && gx * units / 8 >= kFewWorkgroups / 2)
            return launch(&quant_grouped<HADN, SR, ROWS, COLS, 2, 4>, grid_of(gx * (units / 8), kCols), dim3(kCols),
                          st, (const uint16_t*)x, offsets, (int)experts, rows, (int)cols, rot, sr_rows, sr_cols, cr, sr,
                          cc, sc);
    if (gx * units / 2 < kFewWorkgroups)
        return launch(&quant_grouped<HADN, SR, ROWS, COLS, 1, 1>, grid_of(gx * units, kCols), dim3(kCols), st,
                      (const uint16_t*)x, offsets, (int)experts, rows, (int)cols, rot, sr_rows, sr_cols, cr, sr, cc, sc);
    return launch(&quant_grouped<HADN, SR, ROWS, COLS, 2, 1>, grid_of(gx * ((units + 1) / 2), kCols), dim3(kCols), st,
                  (const uint16_t*)x, offsets, (int)experts, rows, (int)cols, rot, sr_rows, sr_cols, cr, sr, cc, sc);
}

template <int HADN, bool SR, typename... A>
hipError_t launch_axes(bool r, bool c, A... a) {
    if (r && c) return launch_one<HADN, SR, true, true>(a...);
    if (r) return launch_one<HADN, SR, true, false>(a...);
    return launch_one<HADN, SR, false, true>(a...);
}

}  // namespace

hipError_t launch_quant_grouped(const void* x, const int* offsets, int64_t experts, int64_t rows, int64_t cols,
                                int had_n, int had, uint64_t sign_seed, int rnd, uint64_t sr_rows, uint64_t sr_cols,
                                uint8_t* codes_r, uint8_t* scales_r, uint8_t* codes_c, uint8_t* scales_c,
                                hipStream_t st) {
    const bool r = codes_r != nullptr, c = codes_c != nullptr, sr = rnd == 1;
    const int n = had == 0 ? 0 : had_n;
    const Rotation rot{host_sign_word(had, sign_seed),
                       n == 16 ? 0.25f : __builtin_bit_cast(float, 0x3E3504F3u)};   // fl(1 / sqrt(n))
#define FP4_GROUPED(N)                                                                                             \
    return sr ? launch_axes<N, true>(r, c, x, offsets, experts, rows, cols, rot, sr_rows, sr_cols, codes_r, scales_r, \
                                     codes_c, scales_c, st)                                                       \
              : launch_axes<N, false>(r, c, x, offsets, experts, rows, cols, rot, sr_rows, sr_cols, codes_r, scales_r, \
                                      codes_c, scales_c, st)
    if (n == 0) FP4_GROUPED(0);
    if (n == 16) FP4_GROUPED(16);
    FP4_GROUPED(32);
#undef FP4_GROUPED
}

}  // namespace fp4dev
