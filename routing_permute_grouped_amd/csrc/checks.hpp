// Argument checks shared by the C ABI entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe.h"
#include "kernels.hpp"

namespace moe {

constexpr int kMaxExperts = 1024;
constexpr int kMaxK = kMaxTopK;
constexpr int kMaxDim = 1 << 16;

inline bool aligned16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool dim_ok(int d) { return d >= 64 && d <= kMaxDim && d % 64 == 0; }
inline bool mtile_ok(int mt) {
  return mt == 16 || mt == 32 || mt == 64 || mt == 128 || mt == 256;
}
inline bool dtype_ok(int dt) { return dt == MOE_F32 || dt == MOE_BF16; }
inline bool tk_ok(int T, int k) { return T >= 1 && (int64_t)T * k <= (1 << 30); }
// masked slabs: a multiple of 16 rows each, E*cap rows addressable with int32
inline bool cap_ok(int E, int cap) {
  return cap >= 16 && cap % 16 == 0 && (int64_t)E * cap <= INT32_MAX;
}

inline moe_status_t hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_EHIP; }

}  // namespace moe
