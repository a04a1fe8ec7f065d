// mx_device.hpp -- device-side pieces the MX quantizing kernels share: quad
// permutes, the in-register Hadamard butterflies, block maxima, 16 bytes of bf16,
// the E2M1 and E4M3 encoders of 8 elements and of a whole 32-element block, and
// the tiled code layout.
#pragma once

#include "fp4_device.hpp"

namespace fp4dev {

// Quad permutes: partner lane q^1 and q^2 inside each group of four lanes.
__device__ __forceinline__ uint32_t quad_xor1(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false);   // [1,0,3,2]
}
__device__ __forceinline__ uint32_t quad_xor2(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false);   // [2,3,0,1]
}
__device__ __forceinline__ float quad_xor1f(float v) { return __uint_as_float(quad_xor1(__float_as_uint(v))); }
__device__ __forceinline__ float quad_xor2f(float v) { return __uint_as_float(quad_xor2(__float_as_uint(v))); }

// In-register butterflies with strides 1 .. N/2 over a[0..N-1].
template <int N>
__device__ __forceinline__ void butterflies(float* a) {
#pragma unroll
    for (int h = 1; h < N; h <<= 1) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i & h) continue;
            const float x = a[i], y = a[i + h];
            a[i] = x + y;
            a[i + h] = x - y;
        }
    }
}

// Largest |a_i| of n values as binary32 bits (NaN > Inf > finite).
template <int N>
__device__ __forceinline__ uint32_t max_abs_bits(const float* a) {
    uint32_t m = 0;
#pragma unroll
    for (int t = 0; t < N; ++t) m = max(m, __float_as_uint(a[t]) & 0x7FFFFFFFu);
    return m;
}

// Codes of 8 values y[0..7] under scale byte `byte` (1..254): hardware
// round-to-nearest-even of y / 2^(byte-127), element 2k in nibble 2k.
__device__ __forceinline__ uint32_t encode8_hw(const float* y, uint32_t byte) {
    const float s = __uint_as_float(byte << 23);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[0], y[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[2], y[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[4], y[5], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[6], y[7], s, 3);
    return w;
}

// Loads and stores of 16 and 8 bytes, non-temporal with NT.
typedef uint32_t word4_t __attribute__((ext_vector_type(4)));
typedef uint32_t word2_t __attribute__((ext_vector_type(2)));
template <bool NT>
__device__ __forceinline__ uint4 load16(const uint4* p) {
    if constexpr (!NT) return *p;
    const word4_t v = __builtin_nontemporal_load(reinterpret_cast<const word4_t*>(p));
    return make_uint4(v.x, v.y, v.z, v.w);
}
template <bool NT>
__device__ __forceinline__ uint2 load8(const uint2* p) {
    if constexpr (!NT) return *p;
    const word2_t v = __builtin_nontemporal_load(reinterpret_cast<const word2_t*>(p));
    return make_uint2(v.x, v.y);
}
template <bool NT>
__device__ __forceinline__ void store16(uint4* p, uint4 v) {
    if constexpr (!NT) *p = v;
    else __builtin_nontemporal_store(word4_t{v.x, v.y, v.z, v.w}, reinterpret_cast<word4_t*>(p));
}
template <bool NT>
__device__ __forceinline__ void store8(void* p, uint2 v) {
    if constexpr (!NT) *static_cast<uint2*>(p) = v;
    else __builtin_nontemporal_store(word2_t{v.x, v.y}, static_cast<word2_t*>(p));
}

// Eight bf16 values of 16 bytes, and back (rounded to nearest even).
__device__ __forceinline__ void unpack8(const uint4& w, float* a) {
    a[0] = bf16_lo(w.x); a[1] = bf16_hi(w.x); a[2] = bf16_lo(w.y); a[3] = bf16_hi(w.y);
    a[4] = bf16_lo(w.z); a[5] = bf16_hi(w.z); a[6] = bf16_lo(w.w); a[7] = bf16_hi(w.w);
}

__device__ __forceinline__ uint4 pack8(const float* a) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16_pair(a[2 * i], a[2 * i + 1]);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Codes of 8 values under scale byte `byte` (not 255) as E4M3: the hardware
// conversion rounds to nearest even but turns what lies beyond 464 into NaN,
// so the scaled value is clamped to +-448 first.
__device__ __forceinline__ uint2 encode8_e4m3(const float* y, uint32_t byte) {
    const float inv = inv_scale_from_e8m0(byte);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __builtin_amdgcn_fmed3f(y[i] * inv, -448.0f, 448.0f);
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
    return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// Integer encoders: v_t = y_t * 2^-(byte-127) in binary32, then RTN or SR.
template <bool SR>
__device__ __forceinline__ uint32_t encode8_sw(const float* y, uint32_t byte, uint4 u0, uint4 u1) {
    const float inv = inv_scale_from_e8m0(byte);
    uint32_t w = 0;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        const float v = y[t] * inv;
        uint32_t c;
        if constexpr (SR) c = e2m1_sr(v, word_of(t < 4 ? u0 : u1, t & 3));
        else c = e2m1_rtn(v);
        w |= c << (4 * t);
    }
    return w;
}

// Byte offset of the 16 code bytes of (row r, block b) in the 32-row tiled
// layout of an operand with nb blocks per row: chunk (r / 32, b) of 512
// bytes, row r mod 32 at 16 (r mod 32).
__device__ __forceinline__ int64_t tiled_offset(int64_t r, int64_t b, int64_t nb) {
    return ((r >> 5) * nb + b) * 512 + (r & 31) * 16;
}

// Rotation, scale and codes of one 32-element block held by one thread: a[]
// holds the block's values in order; gbase is the logical index (in the
// quantized [R, C] layout) of the block's first element divided by 4, the SR
// counter of its first four elements.  Returns the scale byte; wd gets the
// 16 code bytes (zero for a NaN / infinite block).
template <int HADN, bool SR>
__device__ __forceinline__ uint32_t quant_block32(float* a, uint32_t sign_word, float norm,
                                                  uint64_t sr_seed, uint64_t gbase, uint32_t* wd) {
    if constexpr (HADN != 0) {
#pragma unroll
        for (int r = 0; r < 32; ++r) a[r] = flip_if(a[r], (sign_word >> (r % HADN)) & 1u);
#pragma unroll
        for (int o = 0; o < 32; o += HADN) butterflies<HADN>(a + o);
    }
    uint32_t m = max_abs_bits<32>(a);
    if constexpr (HADN != 0) {
        m = __float_as_uint(__uint_as_float(m) * norm) & 0x7FFFFFFFu;
#pragma unroll
        for (int r = 0; r < 32; ++r) a[r] = a[r] * norm;
    }
    const uint32_t byte = e8m0_from_amax_bits(m);
#pragma unroll
    for (int k = 0; k < 4; ++k) wd[k] = 0;
    if (byte != 255u) {
        if (!SR && byte != 0u) {
#pragma unroll
            for (int k = 0; k < 4; ++k) wd[k] = encode8_hw(a + 8 * k, byte);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
                if constexpr (SR) {
                    u0 = stream4(sr_seed, 0u, gbase + 2 * k);
                    u1 = stream4(sr_seed, 0u, gbase + 2 * k + 1);
                }
                wd[k] = encode8_sw<SR>(a + 8 * k, byte, u0, u1);
            }
        }
    }
    return byte;
}

}  // namespace fp4dev
