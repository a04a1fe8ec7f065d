// exp_device.hpp -- the exponential of a negative value.
#pragma once

#include <hip/hip_runtime.h>

namespace fp4dev {

// exp(-a), 0 <= a <= 200: 2^t by the hardware's exp2 with what the product a log2(e)
// rounds off put back (without it the error grows with a, to 2^-18).  Below 2^-126
// the hardware gives 0.
__device__ __forceinline__ float exp_minus_to_200(float a) {
    constexpr float kLog2e = 1.44269504f, kRest = 1.92596303e-8f;   // log2(e) in two parts
    const float t = a * kLog2e;
    const float rest = __builtin_fmaf(a, kLog2e, -t) + a * kRest;
    return __builtin_amdgcn_exp2f(-t) * __builtin_fmaf(rest, -0.693147181f, 1.0f);
}

// exp(-a), a >= 0; zero where a is infinite; a NaN stays one.
__device__ __forceinline__ float exp_minus(float a) { return exp_minus_to_200(a > 200.0f ? 200.0f : a); }

}  // namespace fp4dev
