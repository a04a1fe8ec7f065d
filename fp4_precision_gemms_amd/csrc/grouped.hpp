// grouped.hpp -- rows grouped by expert: where an expert's rows sit in the
// operands, from the row offsets alone.
//
// offsets[0 .. experts]: expert e owns rows [offsets[e], offsets[e + 1]) of a
// tensor of `rows` rows.  In a layout with units of U rows expert e starts at
// unit offsets[e] / U + e.  Its ceil(count / U) units always fit before the
// next expert's first one: floor((o + n) / U) + 1 >= floor(o / U) + ceil(n / U).
// So no prefix sum over the experts, no plan and no look at the counts on the
// host is needed, and rows / U + experts units hold any split.
// U is 32 (a row group of the tiled codes) where the rows are the operand's
// rows, 256 (a stage of the GEMMs) where they are its contraction.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp4dev {

constexpr int kMaxExperts = 1024;

struct RowRange {
    int64_t lo, hi;
};

// What a grouped product needs besides its operands; `rows` are those of the
// tensor that the offsets split.
struct GroupArgs {
    const int* offsets;
    int experts;
    int64_t rows;
};

// Rows of expert e, clamped to the tensor whatever the offsets say.
__device__ __forceinline__ RowRange expert_rows(const int* offsets, int e, int64_t rows) {
    int64_t lo = offsets[e], hi = offsets[e + 1];
    lo = lo < 0 ? 0 : lo > rows ? rows : lo;
    hi = hi < lo ? lo : hi > rows ? rows : hi;
    return {lo, hi};
}

// The expert whose span of U-row units holds unit p (the last one that starts
// at or before p; -1 if none does).  Called by whole waves: each lane looks at
// the first of up to 16 experts, then 16 lanes at those of the last such group
// that starts at or before p.  (Whatever the offsets say, the expert found
// starts at or before p.  1000 experts, 6000 rows of 1024 columns quantized along
// cols: 14.7 us, 28.3 with 64 experts looked at a time.)
template <int U>
__device__ __forceinline__ int expert_of_unit(const int* offsets, int experts, int64_t rows, int64_t p) {
    static_assert(kMaxExperts <= 64 * 64, "two looks");
    const int lane = threadIdx.x & 63;
    auto last_before = [&](int e, bool in) -> int {
        bool before = false;
        if (in) {
            int64_t lo = offsets[e];
            lo = lo < 0 ? 0 : lo > rows ? rows : lo;
            before = lo / U + e <= p;
        }
        return 63 - (int)__clzll((long long)__ballot(before));
    };
    const int step = (experts + 63) / 64;
    int e = last_before(lane * step, lane * step < experts) * step;
    if (e >= 0 && step > 1) e += last_before(e + lane, lane < step && e + lane < experts);
    return __builtin_amdgcn_readfirstlane(e < 0 ? -1 : e);
}

}  // namespace fp4dev
