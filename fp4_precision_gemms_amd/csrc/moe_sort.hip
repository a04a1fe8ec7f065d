// moe_sort.hip -- slots sorted by expert: a stable counting sort.
//
// A slot is one choice of a token (slot t k + j).  Keys are the experts 0 .. E - 1
// and E for every id outside of them.  From ids[slots]:
//     offsets[E + 1]   first row of each expert, then the end of the last one's
//     order[slots]     the slot of each row; slots of no expert behind all rows
//     position[slots]  the row of each slot, -1 for one of no expert
//
// A workgroup takes its slots a tile at a time, 64 I consecutive ones a wave, each
// id read once.  The lanes of a wave that share a key are found by ballots over the
// key's bits; a slot's rank among its wave's is the key's count so far plus the
// lanes before it.  Then a thread a key adds up the waves' counts, and a row is the
// key's first row + the counts of the waves before + the rank.  Order is never
// left to an atomic (those that count keys add integers).
//
// One workgroup does a small batch in one launch; else a first kernel counts the
// keys of every workgroup's slots, and each workgroup of the second adds up the
// counts of those before it, all threads at once.
#include "fp4_launch.hpp"
#include "grouped.hpp"
#include "wave.hpp"

namespace fp4dev {
namespace {

constexpr int kWaves = 16, kThreads = 64 * kWaves;
constexpr int kKeys = kMaxExperts + 1;
static_assert(kMaxExperts <= kThreads, "a thread an expert");

typedef uint32_t count_pair_t __attribute__((may_alias));       // two 16-bit counts

__device__ __forceinline__ int key_of(int id, int E) { return id >= 0 && id < E ? id : E; }

// Counts of each workgroup's `run` slots: counts[workgroup][E + 1].
__global__ __launch_bounds__(kThreads) void sort_count(const int* __restrict__ ids, int64_t slots, int E, int64_t run,
                                                       int* __restrict__ counts) {
    __shared__ int count[kKeys];
    for (int e = threadIdx.x; e <= E; e += kThreads) count[e] = 0;
    __syncthreads();
    const int64_t first = blockIdx.x * run, end = first + run < slots ? first + run : slots;
    for (int64_t i = first + threadIdx.x; i < end; i += kThreads) atomicAdd(&count[key_of(ids[i], E)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += kThreads) counts[(int64_t)blockIdx.x * (E + 1) + e] = count[e];
}

// The rows of a workgroup's `run` slots, tiles of kThreads I of them; ONE: of the
// only workgroup, whose slots are one tile (counts is not looked at) and whose order
// goes through LDS, so that it leaves in whole lines.  bits: of the largest key.
template <int I, bool ONE>
__global__ __launch_bounds__(kThreads) void sort_place(const int* __restrict__ ids, int64_t slots, int E, int bits,
                                                       int64_t run, const int* __restrict__ counts,
                                                       int* __restrict__ offsets, int* __restrict__ order,
                                                       int* __restrict__ position) {
    constexpr int kTile = kThreads * I;
    static_assert(kTile <= 65535, "a tile's counts, and its slots, in 16 bits");
    __shared__ uint16_t by_row[ONE ? kTile : 1];
    __shared__ __attribute__((aligned(4))) uint16_t count[kWaves][kKeys + 1];   // of a wave's slots; of the waves before
    __shared__ int next_row[kKeys];                    // of a key's slots that come next
    __shared__ int before_part[kKeys], all_part[kKeys], totals[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_uniform(tid >> 6);
    const int64_t first = blockIdx.x * run, end = first + run < slots ? first + run : slots;
    const int64_t in_tile = wave * (64 * I) + lane;
    uint16_t* const mine = count[wave];
    int id[I], rank[I];
#pragma unroll
    for (int c = 0; c < I; ++c) id[c] = first + in_tile + 64 * c < end ? ids[first + in_tile + 64 * c] : -1;
    // a key's slots of all workgroups and of those before this one: where the keys
    // are fewer than the threads, `groups` threads share a key's workgroups
    const int groups = bits < 10 ? kThreads >> bits : 1;
    if constexpr (!ONE) {
        for (int k = tid; k < kThreads || k <= E; k += kThreads) {
            const int e = groups > 1 ? k & ((1 << bits) - 1) : k;
            int before = 0, all = 0;
            if (e <= E) {
#pragma unroll 8
                for (int b = groups > 1 ? k >> bits : 0; b < (int)gridDim.x; b += groups) {
                    const int n = counts[(int64_t)b * (E + 1) + e];
                    before += b < (int)blockIdx.x ? n : 0;
                    all += n;
                }
            }
            before_part[k] = before;
            all_part[k] = all;
        }
    }
    for (int64_t tile = first; tile < end; tile += kTile) {
        if (tile != first) {
#pragma unroll
            for (int c = 0; c < I; ++c) id[c] = tile + in_tile + 64 * c < end ? ids[tile + in_tile + 64 * c] : -1;
            __syncthreads();                           // count and next_row have been read
        }
        for (int e = lane; 2 * e <= E; e += 64) reinterpret_cast<count_pair_t*>(mine)[e] = 0;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        // the rank of each slot among its wave's of the same key
#pragma unroll
        for (int c = 0; c < I; ++c) {
            const bool in = tile + in_tile + 64 * c < end;
            id[c] = key_of(id[c], E);
            uint64_t same = __ballot(in);
            for (int b = 0; b < bits; ++b) {
                const bool one = (id[c] >> b) & 1;
                const uint64_t ones = __ballot(one);
                same &= one ? ones : ~ones;
            }
            // a lane that is `in` finds itself in `same`
            const int before =
                __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0));
            const int so_far = mine[id[c]];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (in && before == 0) mine[id[c]] = (uint16_t)(so_far + __popcll(same));
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            rank[c] = so_far + before;
        }
        __syncthreads();
        // a thread a key (one of them two, where E is 1024): the counts of the waves
        // before each, and the tile's
        int n[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int e = tid + k * kThreads;
            if (e > E) continue;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const int v = count[w][e];
                count[w][e] = (uint16_t)n[k];
                n[k] += v;
            }
        }
        if (tile == first) {
            int all[2] = {n[0], n[1]}, before[2] = {0, 0};
            if constexpr (!ONE) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    all[k] = 0;
                    const int e = tid + k * kThreads;
                    if (e > E) continue;
                    for (int g = 0; g < groups; ++g) {
                        before[k] += before_part[(g << bits) + e];
                        all[k] += all_part[(g << bits) + e];
                    }
                }
            }
            const int own = tid < E ? all[0] : 0, sum = wave_scan(own);
            if (lane == 63) totals[wave] = sum;
            __syncthreads();
            int row = sum - own, total = 0;            // the first row of expert tid, and the end of the last one
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                row += w < wave ? totals[w] : 0;
                total += totals[w];
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int e = tid + k * kThreads;
                if (e > E) continue;
                if (e == E) row = total;
                next_row[e] = row + before[k];
                if (blockIdx.x == 0) offsets[e] = row;
            }
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < I; ++c) {
            const int64_t i = tile + in_tile + 64 * c;
            if (i >= end) continue;
            const int row = next_row[id[c]] + mine[id[c]] + rank[c];
            if constexpr (ONE) by_row[row] = (uint16_t)i;
            else order[row] = (int)i;
            position[i] = id[c] < E ? row : -1;
        }
        if constexpr (ONE) {
            __syncthreads();
            for (int row = tid; row < (int)end; row += kThreads) order[row] = by_row[row];
            return;
        }
        if (tile + kTile < end) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (tid + k * kThreads <= E) next_row[tid + k * kThreads] += n[k];
        }
    }
}

// One launch up to this many slots (4096 of 64 experts 5.0 us, 6.1 with two; 6000 of
// 256 8.3 and 7.3).
constexpr int64_t kOneWorkgroup = 4096;
// A thread's slots of a tile, with several workgroups: 16384 slots of 8 experts 6.7 us
// with one and 7.4 with two, 49152 of 64 7.9 and 8.1, 131072 of 256 11.7 and 10.2, of
// 1024 19.7 and 14.7.
int64_t tile_items(int64_t slots) { return slots <= 65536 ? 1 : 2; }

template <int I, bool ONE>
hipError_t launch_place(const int* ids, int64_t slots, int64_t experts, int64_t workgroups, int64_t run,
                        const int* counts, int* offsets, int* order, int* position, hipStream_t st) {
    return launch(&sort_place<I, ONE>, dim3((unsigned)workgroups), dim3(kThreads), st, ids, slots, (int)experts,
                  32 - __builtin_clz((unsigned)experts), run, counts, offsets, order, position);
}

}  // namespace

int64_t moe_sort_workgroups(int64_t slots) {
    if (slots <= kOneWorkgroup) return 1;
    const int64_t tile = kThreads * tile_items(slots), n = (slots + tile - 1) / tile;
    return n < 256 ? n : 256;
}

hipError_t launch_moe_sort(const int* ids, int64_t slots, int64_t experts, int* offsets, int* order, int* position,
                           int* counts, hipStream_t st) {
    const int64_t n = moe_sort_workgroups(slots);
    if (n == 1) {
        // as few slots a thread as take them: 96 slots 2.7 us with one and 4.2 with four,
        // 1800 3.6 with two and 4.6
        auto* const place = slots <= kThreads       ? &launch_place<1, true>
                            : slots <= 2 * kThreads ? &launch_place<2, true>
                                                    : &launch_place<4, true>;
        return place(ids, slots, experts, 1, slots, nullptr, offsets, order, position, st);
    }
    const int64_t tile = kThreads * tile_items(slots), run = ((slots + n - 1) / n + tile - 1) / tile * tile;
    const hipError_t e =
        launch(&sort_count, dim3((unsigned)n), dim3(kThreads), st, ids, slots, (int)experts, run, counts);
    if (e != hipSuccess) return e;
    auto* const place = tile == kThreads ? &launch_place<1, false> : &launch_place<2, false>;
    return place(ids, slots, experts, n, run, counts, offsets, order, position, st);
}

}  // namespace fp4dev
