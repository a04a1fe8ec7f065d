// moe_sort.hip -- slots sorted by expert: a stable counting sort.
//
// A slot is one choice of a token (slot t k + j).  Keys are the experts 0 .. E - 1
// and E for every id outside of them.  From ids[slots]:
//     offsets[E + 1]   first row of each expert, then the end of the last one's
//     order[slots]     the slot of each row; slots of no expert behind all rows
//     position[slots]  the row of each slot, -1 for one of no expert
//
// Every wave owns a run of consecutive slots, 64 at a time.  It counts its keys,
// learns how many of each the runs before it hold, and walks over its run again:
// the lanes that share a key are found by ballots over the key's bits, and a
// slot's row is the key's cursor plus the lanes before it.  No atomic decides an
// order (those on the counts add integers), so the result is the sorted order.
//
// One workgroup does a small batch in one launch; else a first kernel counts the
// keys of each workgroup's slots and every workgroup of the second adds up the
// counts of those before it.
#include "fp4_launch.hpp"
#include "grouped.hpp"
#include "wave.hpp"

namespace fp4dev {
namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kKeys = kMaxExperts + 1;

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

// The rows of a workgroup's `run` slots (a multiple of kThreads); counts null for
// the only workgroup.
__global__ __launch_bounds__(kThreads) void sort_place(const int* __restrict__ ids, int64_t slots, int E, int64_t run,
                                                       const int* __restrict__ counts, int* __restrict__ offsets,
                                                       int* __restrict__ order, int* __restrict__ position) {
    __shared__ int cursor[kWaves][kKeys], first_row[kKeys];
    const int lane = threadIdx.x & 63, wave = wave_uniform((int)threadIdx.x >> 6);
    for (int e = threadIdx.x; e <= E; e += kThreads) {
#pragma unroll
        for (int w = 0; w < kWaves; ++w) cursor[w][e] = 0;
    }
    __syncthreads();
    const int64_t first = blockIdx.x * run + wave * (run / kWaves);
    int64_t end = first + run / kWaves;
    end = end < slots ? end : slots;
    for (int64_t i = first + lane; i < end; i += 64) atomicAdd(&cursor[wave][key_of(ids[i], E)], 1);
    __syncthreads();
    // per key: the counts of the waves before each, of the workgroups before this
    // one, and of all
    for (int e = threadIdx.x; e <= E; e += kThreads) {
        int before = 0, all = 0;
        if (counts) {
            for (unsigned b = 0; b < gridDim.x; ++b) {
                const int n = counts[(int64_t)b * (E + 1) + e];
                before += b < blockIdx.x ? n : 0;
                all += n;
            }
        }
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const int n = cursor[w][e];
            cursor[w][e] = before;
            before += n;
        }
        first_row[e] = counts ? all : before;
    }
    __syncthreads();
    if (wave == 0) {                                   // counts to first rows
        int carry = 0;
        for (int e0 = 0; e0 <= E; e0 += 64) {
            const int e = e0 + lane, n = e <= E ? first_row[e] : 0;
            const int sum = wave_scan(n);
            if (e <= E) first_row[e] = carry + sum - n;
            carry += __builtin_amdgcn_readlane(sum, 63);
        }
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= E; e += kThreads) offsets[e] = first_row[e];
    int bits = 32 - __builtin_clz(E);                  // of the largest key, E >= 1
    int* const mine = cursor[wave];
    for (int64_t i0 = first; i0 < end; i0 += 64) {
        const int64_t i = i0 + lane;
        const bool in = i < end;
        const int key = in ? key_of(ids[i], E) : 0;
        uint64_t same = __ballot(in);
        for (int b = 0; b < bits; ++b) {
            const bool one = (key >> b) & 1;
            const uint64_t ones = __ballot(one);
            same &= one ? ones : ~ones;
        }
        // a lane that is `in` finds itself in `same`
        const int rank = __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0));
        if (in) {
            const int at = mine[key], row = first_row[key] + at + rank;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (rank == 0) mine[key] = at + __popcll(same);
            order[row] = (int)i;
            position[i] = key < E ? row : -1;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// One launch up to this many slots.
constexpr int64_t kOneWorkgroup = 4096;

}  // namespace

int64_t moe_sort_workgroups(int64_t slots) {
    if (slots <= kOneWorkgroup) return 1;
    const int64_t n = (slots + 4095) / 4096;
    return n < 256 ? n : 256;
}

hipError_t launch_moe_sort(const int* ids, int64_t slots, int64_t experts, int* offsets, int* order, int* position,
                           int* counts, hipStream_t st) {
    const int64_t n = moe_sort_workgroups(slots);
    const int64_t run = ((slots + n - 1) / n + kThreads - 1) / kThreads * kThreads;
    if (n > 1) {
        const hipError_t e =
            launch(&sort_count, dim3((unsigned)n), dim3(kThreads), st, ids, slots, (int)experts, run, counts);
        if (e != hipSuccess) return e;
    }
    return launch(&sort_place, dim3((unsigned)n), dim3(kThreads), st, ids, slots, (int)experts, run,
                  (const int*)(n > 1 ? counts : nullptr), offsets, order, position);
}

}  // namespace fp4dev
