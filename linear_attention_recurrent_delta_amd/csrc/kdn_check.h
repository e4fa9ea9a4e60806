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

struct Range {
    const void *p;
    long long n;
};

inline long long up256(long long n) { return (n + 255) / 256 * 256; }

// A launch has less than 2^32 work-items: of more the runtime starts what their
// low 32 bits say, and reports no error.
inline bool launchable(long long workgroups, int threads) {
    return workgroups * threads < (1LL << 32);
}

// Bytes from the first to the last element of `rows` strided rows.
inline long long span(long long rows, long long stride, long long row, long long es) {
    return rows > 0 ? ((rows - 1) * stride + row) * es : 0;
}

// Outputs overlap no input and no other output.
inline bool clash(const Range *outs, int no, const Range *ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlap(outs[i].p, outs[i].n, ins[j].p, ins[j].n))
                return true;
        for (int j = i + 1; j < no; ++j)
            if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return true;
    }
    return false;
}

inline bool valid_dtype(int d) { return d == KDN_F32 || d == KDN_BF16; }
inline bool valid_dim(int d) { return d == 64 || d == 128; }

}  // namespace kdn
