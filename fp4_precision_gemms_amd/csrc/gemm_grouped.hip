// gemm_grouped.hip -- scaled MXFP4 products grouped by expert on the large tiles
// of gemm_mx.hip: C[m, n] = sum_k a[m, k] b[n, k] where
//   kRowGroups   -- the rows of A and C belong to experts, each with a B of its
//                   own (forward, Dgrad);
//   kDepthGroups -- each expert owns whole 256-element stages of the contraction
//                   and an output of its own (Wgrad).
// (fp4_quantize_grouped writes the layouts, grouped.hpp says where an expert
// starts.)
//
// One persistent workgroup of 4 waves per CU, a tile of BM = 32 FM rows x 256
// columns, V_MFMA_SCALE_F32_32X32X64_F8F6F4 with B as first operand, A through
// a ring of four 256-k stage slots in LDS, B straight to registers 8 k-steps
// ahead, as gemm_mx.hip explains; what the groups change:
//   - The tiles.  Row groups: each workgroup counts the experts' row tiles up in
//     LDS when it starts (offsets are known on the device only); a tile never
//     crosses into the next expert.  Depth groups: experts one after another,
//     each one's tiles spread over all XCDs, since experts are of unequal length.
//   - Loads have no tails: code rows past the operand read as zero, scale rows
//     as whatever follows them (they reach no output that is stored), stages
//     past the last or before the first as the nearest one.
//   - A contraction that is no multiple of four stages.  Row groups, all of one
//     length, have a kernel for each remainder, whose tiles start at another
//     slot of the ring.  An expert's depth is known on the device only, so depth
//     groups start with up to three stages that are not of the tile, load but
//     do not multiply them: see the tile loop.
//   - The epilogue stores through a buffer that ends with the tile's last row,
//     16 bytes a lane, so a partial tile takes no branch and the next tile's
//     first stages are always in flight by then.
// Bound like the product without groups, by the card's power limit: 16384 rows
// over 8 experts, 14336 x 4096: 496 us (3.9 PFLOP/s; the same rows as one dense
// product 465 on that box, and 6 % more tiles), the weight gradient 581 us.
#include "fp4_device.hpp"
#include "fp4_launch.hpp"
#include "gemm_tile.hpp"
#include "grouped.hpp"
#include "mx_mfma.hpp"

#include <type_traits>

namespace fp4dev {
namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kBN = 256;            // tile columns: 64 per wave
constexpr int kKS = 4;              // MFMA k-steps (64 k each) per 256-k stage
constexpr int kSlots = 4;           // A stage ring
constexpr int kRing = 8;            // B register ring depth, in k-steps
constexpr int kEpiRow = 64 * 4 + 16;            // a staged row of a wave's 64 fp32 columns, padded
constexpr int kEpiRegion = 32 * kEpiRow;        // 32 rows per wave

// The kernel's lambdas, some with several large callers: left to its own
// judgement the compiler keeps calls, and the accumulators in memory.
#define FP4_INLINE __attribute__((always_inline))

enum { kRowGroups = 1, kDepthGroups = 2 };

// One int per expert in LDS; Which tells several arrays apart.
template <int Which>
__device__ __forceinline__ int* expert_ints() {
    __shared__ int v[kMaxExperts];
    return v;
}

// M: rows of A's scale layout; K: elements per row of A's and B's layouts;
// tiles_m: row tiles of an expert's output (depth groups).
// PHASE: the ring slot of a tile's first stage, for row groups such that the
// last one falls into slot 3 (0 for depth groups).
template <int FM, bool OBF16, int GROUP, int PHASE>
__global__ __launch_bounds__(kThreads) void gemm_mx_grouped(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ SA, const uint8_t* __restrict__ B,
    const uint8_t* __restrict__ SB, int64_t M, int64_t N, int64_t K, void* __restrict__ C, int tiles_m,
    int tiles_n, const GroupArgs ga) {
    constexpr int BM = 32 * FM, FN = 2;
    constexpr int kACodes = FM * 4096;                 // FM row groups x 8 chunks of 512 B
    constexpr int kAScales = 2048;                     // 256 rows x 8 B at most
    constexpr int kSlot = (kACodes + kAScales) > kWaves * kEpiRegion ? (kACodes + kAScales)
                                                                     : kWaves * kEpiRegion;
    // VMEM instructions per wave per stage: A codes (FM) and scales (1) by DMA,
    // B codes (two per k-step) and B scales (two)
    constexpr int kVmStage = FM + 1 + 2 * kKS + 2;
    static_assert(FM >= 4 && FM <= 8, "tile rows");
    constexpr int kWaitStage = 2 * kVmStage - 2;
    static_assert(kWaitStage <= 63, "vmcnt range");
    static_assert(kSlots * kSlot + 3 * 4 * kMaxExperts <= 160 * 1024, "LDS");
    // Stage slots as distinct arrays: the compiler can then tell that
    // fragment reads of one do not wait on DMA still landing in another.
    __shared__ __attribute__((aligned(1024))) uint8_t lds0[kSlot];
    __shared__ __attribute__((aligned(1024))) uint8_t lds1[kSlot];
    __shared__ __attribute__((aligned(1024))) uint8_t lds2[kSlot];
    __shared__ __attribute__((aligned(1024))) uint8_t lds3[kSlot];
    uint8_t* const slots[kSlots] = {lds0, lds1, lds2, lds3};

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // wave-uniform
    const int h = lane >> 5, l32 = lane & 31;
    const int64_t nb = K / 32;                         // blocks per row of the layout
    const uint32_t gstride = (uint32_t)(nb * 512);     // bytes per 32-row group of codes
    int ntiles;
    // of the tile: k-steps, 256-k stages, and the first of the stages (depth
    // groups: 0 or less, their count rounded up to a multiple of the ring)
    int nks = (int)((nb + 1) / 2);
    int nk = (int)((nb + 7) / 8);
    int kfirst = 0;
    if constexpr (GROUP == kRowGroups) {
        // ends[e]: row tiles of experts 0 .. e
        int* const los = expert_ints<0>();
        int* const his = expert_ints<1>();
        int* const ends = expert_ints<2>();
        if (wave == 0) {
            int before = 0;
            for (int base = 0; base < ga.experts; base += 64) {
                const int e = base + lane;
                int n = 0;
                if (e < ga.experts) {
                    const RowRange r = expert_rows(ga.offsets, e, ga.rows);
                    los[e] = (int)r.lo;
                    his[e] = (int)r.hi;
                    n = (int)((r.hi - r.lo + BM - 1) / BM);
                }
#pragma unroll
                for (int o = 1; o < 64; o <<= 1) {
                    const int v = __shfl_up(n, o);
                    if (lane >= o) n += v;
                }
                n += before;
                if (e < ga.experts) ends[e] = n;
                before = __shfl(n, 63);
            }
        }
        __syncthreads();
        tiles_m = __builtin_amdgcn_readfirstlane(ends[ga.experts - 1]);
        ntiles = tiles_m * tiles_n;
        if ((int)blockIdx.x >= ntiles) return;
    } else {
        int* const los = expert_ints<0>();
        int* const his = expert_ints<1>();
        for (int e = tid; e < ga.experts; e += kThreads) {
            const RowRange r = expert_rows(ga.offsets, e, ga.rows);
            los[e] = (int)r.lo;
            his[e] = (int)r.hi;
        }
        __syncthreads();
        ntiles = tiles_m * tiles_n * ga.experts;       // the grid has no more workgroups
    }

    // Per-lane parts of the buffer offsets (the stage / k-step part goes in the
    // scalar offset): A chunk d of this wave's k-step of a stage, B fragment j
    // (row group 2 wave + j) of a k-step, A scales (16 bytes of this wave's
    // 128-row run), B scales (this lane's row of fragment j).
    uint32_t offa[FM], offb[FN], offsb[FN];
#pragma unroll
    for (int d = 0; d < FM; ++d) offa[d] = (uint32_t)d * gstride + (uint32_t)lane * 16;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        offb[j] = (uint32_t)(2 * wave + j) * gstride + (uint32_t)lane * 16;
        offsb[j] = (uint32_t)((64 * wave + 32 * j + l32) * 8);
    }
    const uint32_t offsa = (uint32_t)(((wave & 1) ? (BM - 128) * 8 : 0) + lane * 16);

    int64_t n0 = 0, rows_a = 0;
    // the tile's first row in C, and what comes before its expert's output
    int64_t c0 = 0, cbase = 0;
    __amdgpu_buffer_rsrc_t ra = raw_buffer(A, 0);
    __amdgpu_buffer_rsrc_t rb = ra, rsa = ra, rsb = ra;
    auto set_tile = [&](int t) FP4_INLINE {
        int tile_m, tile_n, e = 0;
        if constexpr (GROUP == kDepthGroups) {
            const int per = tiles_m * tiles_n;
            e = __builtin_amdgcn_readfirstlane(t / per);
            tile_of_block<kGroupRows>(t - e * per, per, tiles_m, tiles_n, tile_m, tile_n);
        } else {
            tile_of_block<kGroupRows>(t, ntiles, tiles_m, tiles_n, tile_m, tile_n);
        }
        tile_m = __builtin_amdgcn_readfirstlane(tile_m);
        tile_n = __builtin_amdgcn_readfirstlane(tile_n);
        n0 = (int64_t)tile_n * kBN;
        const int64_t rows_b = (N - n0) < kBN ? (N - n0) : kBN;
        int64_t m0;
        const uint8_t* sa_tile = SA;
        const uint8_t* sb_tile = SB;
        if constexpr (GROUP == kRowGroups) {
            const int* const ends = expert_ints<2>();
            for (int base = 0; base < ga.experts; base += 64)
                e += __popcll(__ballot(base + lane < ga.experts && ends[base + lane] <= tile_m));
            e = __builtin_amdgcn_readfirstlane(e);
            const int first = e ? __builtin_amdgcn_readfirstlane(ends[e - 1]) : 0;
            const int lo = __builtin_amdgcn_readfirstlane(expert_ints<0>()[e]);
            const int hi = __builtin_amdgcn_readfirstlane(expert_ints<1>()[e]);
            const int64_t local = (int64_t)(tile_m - first) * BM;
            m0 = 32 * ((int64_t)lo / 32 + e) + local;
            c0 = lo + local;
            rows_a = (hi - c0) < BM ? (hi - c0) : BM;
            const int64_t groups = (N + 31) / 32;      // of an expert's B
            ra = raw_buffer(A + (m0 / 32) * (int64_t)gstride, ((rows_a + 31) / 32) * (int64_t)gstride);
            rb = raw_buffer(B + (e * groups + n0 / 32) * (int64_t)gstride, ((rows_b + 31) / 32) * (int64_t)gstride);
            sb_tile = SB + (int64_t)e * nk * N * 8;
        } else {
            const int lo = __builtin_amdgcn_readfirstlane(expert_ints<0>()[e]);
            const int hi = __builtin_amdgcn_readfirstlane(expert_ints<1>()[e]);
            m0 = c0 = (int64_t)tile_m * BM;
            rows_a = (M - m0) < BM ? (M - m0) : BM;
            nk = (hi - lo + 255) / 256;
            nks = 4 * nk;
            kfirst = -((kSlots - nk % kSlots) % kSlots);
            const int64_t q0 = lo / 256 + e;
            cbase = (int64_t)e * M * N;
            sa_tile = SA + q0 * M * 8;
            sb_tile = SB + q0 * N * 8;
            // an expert's span of each 32-row group: up to its last stage (one
            // without rows still loads a stage, which stays unused)
            const int64_t span = (nk ? nk : 1) * 4096;
            ra = raw_buffer(A + (m0 / 32) * (int64_t)gstride + q0 * 4096,
                            ((rows_a + 31) / 32 - 1) * (int64_t)gstride + span);
            rb = raw_buffer(B + (n0 / 32) * (int64_t)gstride + q0 * 4096,
                            ((rows_b + 31) / 32 - 1) * (int64_t)gstride + span);
        }
        // stage q of the tile's rows starts q R 8 bytes further on
        const int64_t stages = nk ? nk : 1;
        rsa = raw_buffer(sa_tile + m0 * 8, (stages * M - m0) * 8);
        rsb = raw_buffer(sb_tile + n0 * 8, (stages * N - n0) * 8);
    };
    // the stage loaded in place of stage kt
    auto stage_of = [&](int kt) FP4_INLINE { return kt < 0 ? 0 : kt < nk ? kt : nk ? nk - 1 : 0; };

    // ---- loads ---------------------------------------------------------
    // A DMA of stage kt into `slot`: chunk d (row group d, k-step `wave` of the
    // stage) for d in [d0, d1), and the scales when `scales`: 16-byte-per-lane
    // DMAs of 128 rows, rows 0..127 (waves 0, 2) and the last 128 rows of the
    // tile (waves 1, 3; the repeated DMA writes the same bytes and keeps every
    // wave's instruction count, hence its waits, identical).
    auto dma_a = [&](int kt, uint8_t* slot, int d0, int d1, bool scales) FP4_INLINE {
        const int kc = stage_of(kt);
        const int soff = __builtin_amdgcn_readfirstlane((4 * kc + wave) * 1024);
#pragma unroll
        for (int d = 0; d < FM; ++d)
            if (d >= d0 && d < d1) dma16_to_lds(ra, slot + d * 4096 + wave * 1024, offa[d], soff);
        if (scales) {
            const int ss = __builtin_amdgcn_readfirstlane((int)((int64_t)kc * M * 8));
            dma16_to_lds(rsa, slot + kACodes + ((wave & 1) ? (BM - 128) * 8 : 0), offsa, ss);
        }
    };
    // B fragment j of k-step s (global index) into registers.
    auto load_b = [&](int s, int j) FP4_INLINE -> v4i {
        const int soff =
            __builtin_amdgcn_readfirstlane((s < 0 ? 0 : s < nks ? s : nks ? nks - 1 : 0) * 1024);
        return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rb, offb[j], soff, 0));
    };
    // B scales of stage kt: this lane's row of fragment j, 8 bytes.
    struct BSc { uint32_t w[FN][2]; };
    auto load_bsc = [&](int kt) FP4_INLINE -> BSc {
        const int ss = __builtin_amdgcn_readfirstlane((int)((int64_t)stage_of(kt) * N * 8));
        BSc r;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const auto v = __builtin_amdgcn_raw_buffer_load_b64(rsb, offsb[j], ss, 0);
            r.w[j][0] = v[0];
            r.w[j][1] = v[1];
        }
        return r;
    };

    // ---- registers -----------------------------------------------------
    v16f acc[FM][FN];
    v4i fa[2][FM];                 // A fragments of two k-steps (k-step parity)
    v4i fb[kRing][FN];             // B fragments, k-step s in fb[(s + 4 PHASE) mod 8]
    BSc bsc[kSlots];               // B scales, stage kt in bsc[(kt - kfirst + PHASE) mod 4]
    struct ASc { uint32_t w[FM][2]; };
    ASc asc[2];                    // A scales of the current and next stage

    // Per-slot lane bases of the LDS reads (see gemm_mx.hip).
    uint32_t lo16 = (uint32_t)lane * 16, lo8 = (uint32_t)l32 * 8;
    asm volatile("" : "+v"(lo16), "+v"(lo8));
    const uint8_t* fbase[kSlots];
    const uint8_t* sbase[kSlots];
#pragma unroll
    for (int q = 0; q < kSlots; ++q) {
        fbase[q] = slots[q] + lo16;
        sbase[q] = slots[q] + kACodes + lo8;
    }
    auto read_afrags = [&](int q, int s, int set) FP4_INLINE {
#pragma unroll
        for (int i = 0; i < FM; ++i)
            fa[set][i] = *reinterpret_cast<const v4i*>(fbase[q] + i * 4096 + s * 1024);
    };
    auto read_ascales = [&](int q, ASc& sc) FP4_INLINE {
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const uint2 v = *reinterpret_cast<const uint2*>(sbase[q] + i * 32 * 8);
            sc.w[i][0] = v.x;
            sc.w[i][1] = v.y;
        }
    };
    // Row groups: the bytes of the last stage's scale words (byte s: block
    // 2 s + h of the stage) that are of blocks of the operand.
    const int last_bytes = (int)(nb - 8 * (nk - 1) - h + 1) / 2;
    const uint32_t last_keep = last_bytes >= 4 ? ~0u : (1u << (8 * last_bytes)) - 1;
    struct SWords { uint32_t a[FM], b[FN]; };
    auto stage_words = [&](const ASc& sa, const BSc& sb, int kt) FP4_INLINE -> SWords {
        SWords w;
#pragma unroll
        for (int i = 0; i < FM; ++i) w.a[i] = stage_scale_word(sa.w[i][0], sa.w[i][1], h);
#pragma unroll
        for (int j = 0; j < FN; ++j) w.b[j] = stage_scale_word(sb.w[j][0], sb.w[j][1], h);
        if constexpr (GROUP == kRowGroups) {
            // Blocks past the last one hold whatever follows: with both scales
            // 2^-127 their products vanish.
            const uint32_t keep = kt == nk - 1 ? last_keep : ~0u;
#pragma unroll
            for (int i = 0; i < FM; ++i) w.a[i] &= keep;
#pragma unroll
            for (int j = 0; j < FN; ++j) w.b[j] &= keep;
        }
        return w;
    };
    // MFMAs of k-step s (0..3) of a stage: A fragments set, B ring slot r.
    auto mfmas = [&](int s, int set, int r, const SWords& sw) FP4_INLINE {
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const v8i af = __builtin_shufflevector(fa[set][i], v4i{0, 0, 0, 0}, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const v8i bf = __builtin_shufflevector(fb[r][j], v4i{0, 0, 0, 0}, 0, 1, 2, 3, 4, 5, 6, 7);
                switch (s) {
                    case 0: acc[i][j] = mfma_fp4<0>(bf, af, acc[i][j], sw.b[j], sw.a[i]); break;
                    case 1: acc[i][j] = mfma_fp4<1>(bf, af, acc[i][j], sw.b[j], sw.a[i]); break;
                    case 2: acc[i][j] = mfma_fp4<2>(bf, af, acc[i][j], sw.b[j], sw.a[i]); break;
                    default: acc[i][j] = mfma_fp4<3>(bf, af, acc[i][j], sw.b[j], sw.a[i]); break;
                }
            }
        }
    };

    // A chunk DMAs of a stage are spread over k-steps 0..2: k-step s issues
    // chunks [kdma(s), kdma(s + 1)) (the scale run goes with k-step 0).
    auto kdma = [](int s) { return s * FM / 3 < FM ? s * FM / 3 : FM; };

    // One stage from slot u (its k-step 0 fragments and scales already in
    // registers).  Stage kt + 3 is loaded into slot (u + 3) mod 4, B scales
    // of stage kt + 2 into the B scale ring, B k-steps 8 ahead into the B
    // ring.  Without `live`: these loads alone.
    auto run_stage = [&](int u, int kt, bool live = true) FP4_INLINE {
        uint8_t* const ahead = slots[(u + 3) % kSlots];
        ASc& nsa = asc[(u + 1) & 1];
        const SWords sw = stage_words(asc[u & 1], bsc[u], kt);
#pragma unroll
        for (int s = 0; s < kKS - 1; ++s) {
            read_afrags(u, s + 1, (s + 1) & 1);
            if (live) mfmas(s, s & 1, (4 * u + s) % kRing, sw);
#pragma unroll
            for (int j = 0; j < FN; ++j) fb[(4 * u + s) % kRing][j] = load_b(4 * kt + s + kRing, j);
            dma_a(kt + 3, ahead, kdma(s), kdma(s + 1), s == 0);
            if (s == 0) bsc[(u + 2) % kSlots] = load_bsc(kt + 2);
            // interleave: one MFMA, then a DS read and a VMEM op spread evenly
            constexpr int kM = FM * FN;
            const int nvm = FN + (kdma(s + 1) - kdma(s)) + (s == 0 ? 1 + FN : 0);
#pragma unroll
            for (int t = 0; t < kM; ++t) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);        // MFMA
                if ((t + 1) * FM / kM > t * FM / kM)
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);    // DS read
                if ((t + 1) * nvm / kM > t * nvm / kM)
                    __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);    // VMEM read
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        // this wave's DMA of stage kt + 1 (issued two stages ago) has landed,
        // and its fragment reads of the current one are done; the barrier
        // publishes every wave's part of stage kt + 1.  At least
        // 2 kVmStage - 2 VMEM instructions follow the last one of stage
        // kt + 1: all of stage kt - 1, stage kt up to here, the B loads
        // closing stage kt - 2 (the prologue's order gives exactly that count
        // for the first stages).
        __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(kWaitStage));
        barrier_after_wait();
        read_ascales((u + 1) % kSlots, nsa);
        read_afrags((u + 1) % kSlots, 0, 0);
        if (live) mfmas(kKS - 1, 1, (4 * u + 3) % kRing, sw);
#pragma unroll
        for (int j = 0; j < FN; ++j) fb[(4 * u + 3) % kRing][j] = load_b(4 * kt + 3 + kRing, j);
        constexpr int kM = FM * FN, kDs = 2 * FM;
#pragma unroll
        for (int t = 0; t < kM; ++t) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);            // MFMA
            if ((t + 1) * kDs / kM > t * kDs / kM) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            if ((t + 1) * kDs / kM > t * kDs / kM + 1) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            if ((t + 1) * FN / kM > t * FN / kM) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };

    // The first stages of a tile: A stages kfirst .. kfirst+2 into the slots
    // from PHASE on, B scales of the first two stages, B k-steps of the first two
    // stages, in stage order, so that the wait for stage kfirst counts
    // everything after its A part (the scheduling barriers keep this order).
    auto prologue = [&]() FP4_INLINE {
        dma_a(kfirst, slots[PHASE], 0, FM, true);
        __builtin_amdgcn_sched_barrier(0);
        bsc[PHASE] = load_bsc(kfirst);
#pragma unroll
        for (int s = 0; s < kKS; ++s)
#pragma unroll
            for (int j = 0; j < FN; ++j) fb[(4 * PHASE + s) % kRing][j] = load_b(4 * kfirst + s, j);
        __builtin_amdgcn_sched_barrier(0);
        dma_a(kfirst + 1, slots[(PHASE + 1) % kSlots], 0, FM, true);
        __builtin_amdgcn_sched_barrier(0);
        bsc[(PHASE + 1) % kSlots] = load_bsc(kfirst + 1);
#pragma unroll
        for (int s = kKS; s < 2 * kKS; ++s)
#pragma unroll
            for (int j = 0; j < FN; ++j) fb[(4 * PHASE + s) % kRing][j] = load_b(4 * kfirst + s, j);
        __builtin_amdgcn_sched_barrier(0);
        dma_a(kfirst + 2, slots[(PHASE + 2) % kSlots], 0, FM, true);
        __builtin_amdgcn_sched_barrier(0);
    };
    // VMEM issued after stage kfirst's A part in the prologue: its B scales,
    // the B loads of two stages, two more A stages and one more B scale load
    constexpr int kPro = FN + 2 * kKS * FN + 2 * (FM + 1) + FN;
    // stores of an epilogue per wave: 16 bytes a lane, so 8 rows of bf16 or 4 of
    // fp32 per instruction (8 bytes of bf16 a lane, and integer rounding, took
    // 540 us where this takes 496: 8 experts of 2048 rows, 14336 x 4096)
    constexpr int kEpiRows = OBF16 ? 8 : 4, kEpiStores = FM * (32 / kEpiRows);
    constexpr int kOut = OBF16 ? 2 : 4;

    // Staggered start, as in gemm_mx.hip: the tile boundaries of the workgroups
    // do not all fall at the same moment (8 experts of 4096 x 4096, 1024 uneven
    // rows 81 us, 92 without; 16 of them, weight gradient, 1024 rows 201 and 227).
    // The last workgroup starts 7 us late, the time of a short tile, so that row
    // groups of two rounds or few stages shorten it by their stages (8 experts of
    // 4096 x 256, 512 rows 18.6 with the whole, 12.3 us with 1/16; 32 of 2048 x
    // 512, 250 rows 18.7 and 14.4; but 8 of 4096 x 1024, 1000 rows, four rounds,
    // 35.2 and 42).
    if (ntiles > (int)gridDim.x) {
        int delay = blockIdx.x;
        if constexpr (GROUP == kRowGroups)
            if (nk < 16 && (ntiles <= 2 * (int)gridDim.x || (int64_t)ntiles * nk * FM <= 32 * (int)gridDim.x))
                delay = delay * nk / 16;
        for (int q = 0; q < delay; ++q) __builtin_amdgcn_s_sleep(1);
    }
    // The first tile's prologue goes out here and every later one during the
    // previous tile's epilogue, which leaves the loop a single prologue site.
    set_tile(blockIdx.x);
    prologue();
    __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(0));
    for (int t = blockIdx.x; t < ntiles; t += gridDim.x) {
        // the prologue went out before the previous tile's kEpiStores stores
        // (the memory counter completes in order)
        __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(kPro + kEpiStores < 63 ? kPro + kEpiStores : 63));
        barrier_after_wait();
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
        read_ascales(PHASE, asc[PHASE & 1]);
        read_afrags(PHASE, 0, 0);
        // The tile's stages and its epilogue, after `dead` stages that are not
        // of the tile (loads only).
        auto tile = [&](auto dead) FP4_INLINE {
            constexpr int D = decltype(dead)::value;
            int kt = kfirst;
            if constexpr (PHASE > 0) {
                if constexpr (PHASE < 2) run_stage(1, kt++);
                if constexpr (PHASE < 3) run_stage(2, kt++);
                run_stage(3, kt++);
            }
            if constexpr (D > 0) {
                run_stage(0, kt, false);
                run_stage(1, kt + 1, D < 2);
                run_stage(2, kt + 2, D < 3);
                run_stage(3, kt + 3);
                kt += kSlots;
            }
            for (; kt < nk; kt += kSlots) {
                run_stage(0, kt);
                run_stage(1, kt + 1);
                run_stage(2, kt + 2);
                run_stage(3, kt + 3);
            }

            // the prefetches past the last stage must land before the slots are
            // refilled (and before the workgroup goes away)
            __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(0));
            __syncthreads();                           // all fragment reads of the tile are done

            // The tile's rows of C as one buffer; this lane's offset in its
            // first row, out of range for columns past N.  What lies past the
            // last row is past the buffer's end.  Non-temporal (8 experts of
            // 512 rows, 14336 x 4096, in bf16 on 128-row tiles: 156 us, 180 with
            // plain stores; 8 of 2000 rows and 8160 x 4064, whose rows are no
            // whole lines: 271 and 303, their weight gradient 321 and 372).
            const int er = lane / (64 / kEpiRows), ec = lane % (64 / kEpiRows) * kEpiRows;
            const uint32_t row_bytes = (uint32_t)N * kOut;
            const __amdgpu_buffer_rsrc_t rc = raw_buffer(
                (uint8_t*)C + (cbase + c0 * N + n0) * kOut, (rows_a * N - n0) * kOut);
            const uint32_t offc = n0 + 64 * wave + ec < N
                                      ? (uint32_t)er * row_bytes + (uint32_t)(64 * wave + ec) * kOut
                                      : kOob;

            // The next tile's first stages go out now, into three slots (this
            // epilogue stages in the fourth); waited for at the next tile's start.
            const int tn = t + (int)gridDim.x;
            if (tn < ntiles) {
                set_tile(tn);
                prologue();
            }

            // acc[i][j] holds C^T of a 32x32 tile: register r of lane l is
            // n = 8 (r / 4) + 4 (l / 32) + r mod 4, m = l mod 32.  Each wave
            // stages 32 rows x its 64 columns at a time in its quarter of that
            // slot (rows padded by 16 bytes), then reads back whole row segments.
            uint8_t* const reg = slots[(PHASE + 3) % kSlots] + wave * kEpiRegion;
#pragma unroll
            for (int i = 0; i < FM; ++i) {
#pragma unroll
                for (int j = 0; j < FN; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int cn = j * 32 + 8 * q + 4 * h;
                        *reinterpret_cast<float4*>(reg + l32 * kEpiRow + cn * 4) =
                            make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                                        acc[i][j][4 * q + 3]);
                    }
                v4u o[32 / kEpiRows];
#pragma unroll
                for (int k = 0; k < 32 / kEpiRows; ++k) {
                    const v4f* const f = reinterpret_cast<const v4f*>(reg + (kEpiRows * k + er) * kEpiRow + ec * 4);
                    if constexpr (OBF16) {
                        const v4f a = f[0], b = f[1];
                        o[k] = v4u{bf16_pair(a[0], a[1]), bf16_pair(a[2], a[3]), bf16_pair(b[0], b[1]),
                                   bf16_pair(b[2], b[3])};
                    } else {
                        o[k] = __builtin_bit_cast(v4u, f[0]);
                    }
                }
#pragma unroll
                for (int k = 0; k < 32 / kEpiRows; ++k) {
                    const uint32_t at = offc + (uint32_t)(32 * i + kEpiRows * k) * row_bytes;
                    __builtin_amdgcn_raw_buffer_store_b128(o[k], rc, at, 0, 2);
                }
            }
        };
        if constexpr (GROUP == kDepthGroups) {
            // Up to three stages multiplied in vain cost: 8 experts of 2048
            // tokens, 14336 x 4096 632 us with them, 581 without.  Each count
            // has code of its own from the first stage to the last store: where
            // the accumulators of two paths met, the compiler spilled hundreds
            // of registers.
            switch (-kfirst) {
                case 1: tile(std::integral_constant<int, 1>{}); break;
                case 2: tile(std::integral_constant<int, 2>{}); break;
                case 3: tile(std::integral_constant<int, 3>{}); break;
                default: tile(std::integral_constant<int, 0>{}); break;
            }
        } else {
            tile(std::integral_constant<int, 0>{});
        }
    }
}

template <int FM, int GROUP, int PHASE>
hipError_t launch_grouped(const uint8_t* aq, const uint8_t* as, const uint8_t* bq, const uint8_t* bs, int64_t M,
                          int64_t N, int64_t K, void* c, int out_bf16, int64_t most, int64_t tm, int64_t tn,
                          const GroupArgs& ga, hipStream_t st) {
    const int64_t cus = cu_count();
    const dim3 grid((unsigned)(most < cus ? most : cus));
    auto* const k = out_bf16 ? &gemm_mx_grouped<FM, true, GROUP, PHASE> : &gemm_mx_grouped<FM, false, GROUP, PHASE>;
    return launch(k, grid, dim3(kThreads), st, aq, as, bq, bs, M, N, K, c, (int)tm, (int)tn, ga);
}

template <int FM, typename... T>
hipError_t launch_rows(int64_t stages, T... a) {
    switch (stages % kSlots) {
        case 1: return launch_grouped<FM, kRowGroups, 3>(a...);
        case 2: return launch_grouped<FM, kRowGroups, 2>(a...);
        case 3: return launch_grouped<FM, kRowGroups, 1>(a...);
        default: return launch_grouped<FM, kRowGroups, 0>(a...);
    }
}

}  // namespace

// Whether the tiles' 32-bit offsets hold: rows of C in whole 16-byte pieces, a
// tile of C and an operand's scales within 2 GiB.
bool row_groups_fit(int64_t experts, int64_t rows, int64_t N, int64_t K) {
    const int64_t M = 32 * (rows / 32 + experts);
    return N % 8 == 0 && N < (INT64_C(1) << 21) && (K + 255) / 256 * (M > N ? M : N) * 8 < (INT64_C(1) << 31);
}

hipError_t launch_gemm_row_groups(const uint8_t* aq, const uint8_t* as, const int* offsets, int64_t experts,
                                  int64_t rows, const uint8_t* wq, const uint8_t* ws, int64_t N, int64_t K, void* c,
                                  int out_bf16, hipStream_t st) {
    const int64_t M = 32 * (rows / 32 + experts), tn = (N + kBN - 1) / kBN, cus = cu_count();
    const int64_t stages = (K + 255) / 256;
    const GroupArgs ga{offsets, (int)experts, rows};
    // Tile rows: rounds of the persistent grid times a tile's time, with half a
    // tile per expert for its last one, and a whole one where that is all it has
    // (64 experts of 1408 x 1408, 40 rows each: 20 us, 29 without this).  A tile of 128 rows takes 0.53-0.62 of
    // one of 256 (it loads as much of B): 8 experts of 14336 x 4096, 256 rows
    // each 92 against 100 us, 2048 rows 574 against 526; 32 experts of 2048 x
    // 2048, 200 rows 33 against 40.
    auto rounds = [&](int64_t bm) {
        const int64_t half = rows / bm + (experts + 1) / 2;
        return ((half > experts ? half : experts) * tn + cus - 1) / cus;
    };
    if (58 * rounds(128) < 100 * rounds(256))
        return launch_rows<4>(stages, aq, as, wq, ws, M, N, K, c, out_bf16, (rows / 128 + experts) * tn, 0, tn,
                                             ga, st);
    return launch_rows<8>(stages, aq, as, wq, ws, M, N, K, c, out_bf16, (rows / 256 + experts) * tn, 0, tn, ga,
                                         st);
}

hipError_t launch_gemm_depth_groups(const uint8_t* aq, const uint8_t* as, const uint8_t* bq, const uint8_t* bs,
                                    const int* offsets, int64_t experts, int64_t rows, int64_t M, int64_t N, void* c,
                                    int out_bf16, hipStream_t st) {
    const int64_t K = 256 * (rows / 256 + experts);             // of the grouped layout
    const int64_t tm = (M + 255) / 256, tn = (N + kBN - 1) / kBN;
    return launch_grouped<8, kDepthGroups, 0>(aq, as, bq, bs, M, N, K, c, out_bf16, tm * tn * experts, tm, tn,
                                           GroupArgs{offsets, (int)experts, rows}, st);
}

}  // namespace fp4dev
