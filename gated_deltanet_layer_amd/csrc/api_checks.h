// api_checks.h -- host-side helpers of the C ABI's argument checks.
#pragma once
#include <stdint.h>

namespace gdn_checks {

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};

inline bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1u)) == 0; }
inline bool aligned16(const void *p) { return aligned(p, 16); }

inline Range range(const void *p, unsigned long long bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, lo + (uintptr_t)bytes};
}

inline bool overlap(Range a, Range b) {
    if (a.lo == a.hi || b.lo == b.hi) return false;
    return a.lo < b.hi && b.lo < a.hi;
}

// n = a * b * c * d without overflow past 2^62, or -1.
inline long long prod(long long a, long long b, long long c = 1, long long d = 1) {
    const long long lim = 1LL << 62;
    long long n = a;
    for (long long f : {b, c, d}) {
        if (f != 0 && n > lim / f) return -1;
        n *= f;
    }
    return n;
}

} // namespace gdn_checks
