// kdn_check.h -- host-side argument checks shared by the C ABI sources.
#pragma once

#include "kdn.h"

#include <stdint.h>

namespace kdn {

inline bool aligned(const void *p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// [a, a+na) and [b, b+nb) overlap (byte ranges, empty ranges never overlap)
inline bool overlap(const void *a, long long na, const void *b, long long nb) {
    if (!a || !b || na <= 0 || nb <= 0)
        return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

inline bool valid_dtype(int d) { return d == KDN_F32 || d == KDN_BF16; }
inline bool valid_dim(int d) { return d == 64 || d == 128; }

}  // namespace kdn
