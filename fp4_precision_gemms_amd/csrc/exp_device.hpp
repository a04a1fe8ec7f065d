// exp_device.hpp -- the exponential of a negative value.
#pragma once

#include <hip/hip_runtime.h>

namespace fp4dev {

// exp(-a), 0 <= a <= 200: 2^n 2^f with n the whole number next to -a log2(e) and f
// what is left, without the rounding of that product (whose error would grow with a,
// to 2^-18); |f| <= 1/2, so the hardware's exp2 is off by a step.  Values below 2^-126
// are kept, down to 2^-149: they may meet large factors next.
__device__ __forceinline__ float exp_minus_to_200(float a) {
    constexpr float kLog2e = 1.44269504f, kRest = 1.92596303e-8f;   // log2(e) in two parts
    constexpr float kWhole = 0x1.8p23f;                // n added to it is its last bits
    const float m = __builtin_fmaf(a, -kLog2e, kWhole);
    const float f = __builtin_fmaf(a, -kRest, __builtin_fmaf(a, -kLog2e, kWhole - m));
    return __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(f), __float_as_int(m) - 0x4B400000);
}

// exp(-a), a >= 0; zero where a is infinite; a NaN stays one.
__device__ __forceinline__ float exp_minus(float a) { return exp_minus_to_200(a > 200.0f ? 200.0f : a); }

}  // namespace fp4dev
