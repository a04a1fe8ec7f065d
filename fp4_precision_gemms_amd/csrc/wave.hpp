// wave.hpp -- reductions over a 64-lane wave by data-parallel moves (DPP), the
// result in every lane by way of a scalar register: no LDS traffic and no
// latency of one (a sum of a wave takes 7 vector instructions; the same by __shfl_xor
// 6 trips through the LDS pipe).  The norm keeps a sum of its own by __shfl_xor, also
// of binary64 numbers, whose order its results go by.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp4dev {

constexpr int kRowShr1 = 0x111, kRowShr2 = 0x112, kRowShr4 = 0x114, kRowShr8 = 0x118;   // within 16 lanes
constexpr int kRowRor1 = 0x121, kRowRor2 = 0x122, kRowRor4 = 0x124, kRowRor8 = 0x128;   // rotated within 16
constexpr int kRowBcast15 = 0x142, kRowBcast31 = 0x143;      // lane 15 of a row, lane 31, to the rows behind

// `v` of the lane that CTRL names; `old` where there is none or ROWS leaves the row out.
template <int CTRL, int ROWS>
__device__ __forceinline__ int moved(int old, int v) {
    return __builtin_amdgcn_update_dpp(old, v, CTRL, ROWS, 0xF, false);
}

// The sum's order is fixed: pairs of lanes, of pairs, ... of each 16, then the
// four 16s.
__device__ __forceinline__ float wave_sum(float v) {
    auto add = [](float a, int b) { return a + __int_as_float(b); };
    v = add(v, moved<kRowShr1, 0xF>(0, __float_as_int(v)));
    v = add(v, moved<kRowShr2, 0xF>(0, __float_as_int(v)));
    v = add(v, moved<kRowShr4, 0xF>(0, __float_as_int(v)));
    v = add(v, moved<kRowShr8, 0xF>(0, __float_as_int(v)));
    v = add(v, moved<kRowBcast15, 0xA>(0, __float_as_int(v)));
    v = add(v, moved<kRowBcast31, 0xC>(0, __float_as_int(v)));
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Of each 16 lanes, in all of them (the same bits: the two sums that meet are the
// same pair).
__device__ __forceinline__ float row_sum(float v) {
    auto add = [](float a, int b) { return a + __int_as_float(b); };
    v = add(v, moved<kRowRor8, 0xF>(0, __float_as_int(v)));
    v = add(v, moved<kRowRor4, 0xF>(0, __float_as_int(v)));
    v = add(v, moved<kRowRor2, 0xF>(0, __float_as_int(v)));
    v = add(v, moved<kRowRor1, 0xF>(0, __float_as_int(v)));
    return v;
}

// The largest of 16 lanes or of the wave, in all of them; a NaN is none.
template <int LANES>
__device__ __forceinline__ float token_max(float v) {
    auto larger = [](float a, int b) { return fmaxf(a, __int_as_float(b)); };
    auto bits = [](float a) { return __float_as_int(a); };
    v = larger(v, moved<kRowRor1, 0xF>(bits(v), bits(v)));
    v = larger(v, moved<kRowRor2, 0xF>(bits(v), bits(v)));
    v = larger(v, moved<kRowRor4, 0xF>(bits(v), bits(v)));
    v = larger(v, moved<kRowRor8, 0xF>(bits(v), bits(v)));
    if constexpr (LANES == 64) {
        v = larger(v, moved<kRowBcast15, 0xF>(bits(v), bits(v)));
        v = larger(v, moved<kRowBcast31, 0xF>(bits(v), bits(v)));
        v = __int_as_float(__builtin_amdgcn_readlane(bits(v), 63));
    }
    return v;
}

// Inclusive prefix sums over the lanes.
__device__ __forceinline__ int wave_scan(int v) {
    v += moved<kRowShr1, 0xF>(0, v);
    v += moved<kRowShr2, 0xF>(0, v);
    v += moved<kRowShr4, 0xF>(0, v);
    v += moved<kRowShr8, 0xF>(0, v);
    v += moved<kRowBcast15, 0xA>(0, v);
    v += moved<kRowBcast31, 0xC>(0, v);
    return v;
}

__device__ __forceinline__ int wave_uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint32_t wave_uniform(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
}

}  // namespace fp4dev
