// fp4_check.hpp -- argument checks and status codes the C ABI's files share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4.h"

namespace fp4abi {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// a * b stays far from int64 overflow (byte counts of bf16 / fp32 tensors)
inline bool product_ok(int64_t a, int64_t b) { return a > 0 && b > 0 && a <= (INT64_C(1) << 60) / b; }

constexpr int64_t kMaxContraction = INT64_C(1) << 24;
constexpr int64_t kMaxTiles = INT64_C(1) << 24;

inline fp4_status from_hip(hipError_t e) { return e == hipSuccess ? FP4_OK : FP4_ERR_LAUNCH; }

}  // namespace fp4abi
