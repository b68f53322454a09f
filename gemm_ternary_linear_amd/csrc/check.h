// Host-side argument checks shared by the C ABI's translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/ternary.h"
#include "internal.h"

namespace ternary {

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// [a, a+na) and [b, b+nb) overlap (byte ranges; empty ranges never overlap).
inline bool overlap(const void *a, int64_t na, const void *b, int64_t nb)
{
    if (na <= 0 || nb <= 0)
        return false;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + (uintptr_t)nb && b0 < a0 + (uintptr_t)na;
}

inline int hip_status(hipError_t e)
{
    if (e == hipSuccess)
        return TERNARY_OK;
    return e == kErrCaptureWorkspace ? TERNARY_ERR_WORKSPACE : TERNARY_ERR_HIP;
}

// Largest M, N or K accepted: kernels index channels, tokens and K with
// 32-bit ints (element offsets are 64-bit) and grids stay far inside the
// launch limits.
constexpr int64_t kMaxDim = (int64_t)1 << 24;

}  // namespace ternary
