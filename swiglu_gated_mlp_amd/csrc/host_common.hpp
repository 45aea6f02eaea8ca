// Host helpers that the library's entry points share: argument checks (no HIP
// calls), the device's CU count and the per-thread record of a failed HIP call.
#pragma once

#include "swiglu.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

namespace swh {

extern thread_local int g_last_hip_error;   // swiglu_last_hip_error()

inline swiglu_status hip_fail(hipError_t e) {
    g_last_hip_error = (int)e;
    return SWIGLU_ERR_HIP;
}

constexpr int64_t kMaxDim = (int64_t)1 << 30;   // every dimension fits int32 with room
constexpr int64_t kMaxK = (int64_t)1 << 22;     // 256 rows of activations stay below 2 GiB

// ---------------------------------------------------------------------------
// argument checks (host only, no HIP calls)
// ---------------------------------------------------------------------------
inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

struct Range {
    uintptr_t lo, hi;   // [lo, hi)
};

inline Range range_of(const void* p, int64_t bytes) {
    return Range{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes};
}

inline bool overlap(Range a, Range b) {
    if (a.lo == a.hi || b.lo == b.hi) return false;
    return a.lo < b.hi && b.lo < a.hi;
}

inline swiglu_status check_shape(int64_t M, int64_t K, int64_t N) {
    if (M < 0 || K <= 0 || N <= 0) return SWIGLU_ERR_BAD_SHAPE;
    if (M > kMaxDim || K > kMaxDim || N > kMaxDim) return SWIGLU_ERR_BAD_SHAPE;
    if (M * N > ((int64_t)1 << 40) || K * N > ((int64_t)1 << 40) || M * K > ((int64_t)1 << 40))
        return SWIGLU_ERR_BAD_SHAPE;
    if ((K % 8) != 0 || (N % 8) != 0) return SWIGLU_ERR_UNSUPPORTED_SHAPE;
    if (K > kMaxK) return SWIGLU_ERR_UNSUPPORTED_SHAPE;
    return SWIGLU_OK;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---------------------------------------------------------------------------
// device facts
// ---------------------------------------------------------------------------
inline int cu_count_now() {
    static std::mutex mu;
    static int cache[64] = {0};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lock(mu);
    if (cache[dev] == 0) {
        int n = 0;
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return 0;
        cache[dev] = n;
    }
    return cache[dev];
}

}  // namespace swh
