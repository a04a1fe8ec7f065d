// mx_mfma.hpp -- what the MXFP4 products share: vector types, raw buffers, the
// scaled FP4 MFMA and its scale words.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp4dev {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kBufferWord3 = 0x00020000;   // raw buffer, 32-bit data format
constexpr uint32_t kOob = 0x80000000u;     // a buffer offset past any range: reads zero

__device__ __forceinline__ __amdgpu_buffer_rsrc_t raw_buffer(const void* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, kBufferWord3);
}
__device__ __forceinline__ v4i load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// Scaled FP4 MFMA (32x32x64, both operands E2M1, fp32 accumulate) taking the
// E8M0 scales from byte S of the scale registers.
template <int S>
__device__ __forceinline__ v16f mfma_fp4(v8i b, v8i a, v16f c, uint32_t sb, uint32_t sa) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, c, 4, 4, S, (int)sb, S, (int)sa);
}

// The scale word a lane feeds the MFMAs of one 256-k stage: the stage's 8
// block scales of its row are bytes 0..7 of (hi:lo); k-step s uses block
// 2 s + (lane / 32), so lane half h keeps bytes h, 2 + h, 4 + h, 6 + h, and
// k-step s reads byte s of the word -- one byte permute per stage instead of
// a shift before every MFMA.  Formed when the stage starts: at load time it
// would wait for loads issued stages ahead.
__device__ __forceinline__ uint32_t stage_scale_word(uint32_t lo, uint32_t hi, int h) {
    return __builtin_amdgcn_perm(hi, lo, h ? 0x07050301u : 0x06040200u);
}

// Bytes of a scale word for blocks first .. first+3 that lie at or past nb
// (the unused tail of the last k-group) set to 127 (2^0; their codes are
// zero).
__device__ __forceinline__ uint32_t mask_scale_word(uint32_t w, int64_t first, int64_t nb) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (first + i >= nb) w = (w & ~(0xFFu << (8 * i))) | (127u << (8 * i));
    return w;
}

}  // namespace fp4dev
