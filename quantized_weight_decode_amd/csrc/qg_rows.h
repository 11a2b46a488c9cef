// qg_rows.h -- whether two sets of rows share a byte (host only).
#pragma once

#include <stdint.h>

namespace qg {

// Rows of bytes: n of `width`, `ld` apart.  The comparison is exact, so that
// columns of one buffer may be x and others y.
struct Rows {
    uintptr_t p;
    long long n, width, ld;
};

inline Rows rows_of(const void *p, long long n, long long width, long long ld)
{
    return {(uintptr_t)p, p ? n : 0, width, ld};
}
inline Rows block(const void *p, long long bytes) { return rows_of(p, bytes > 0, bytes, bytes); }

inline long long floor_div(long long a, long long b) { return a / b - (a % b < 0); }

inline bool overlap(Rows a, Rows b)
{
    if (a.n < 1 || b.n < 1) return false;
    if (a.n > b.n) {
        const Rows t = a;
        a = b;
        b = t;
    }
    const uintptr_t a_end = a.p + (a.n - 1) * a.ld + a.width;
    const uintptr_t b_end = b.p + (b.n - 1) * b.ld + b.width;
    if (a_end <= b.p || b_end <= a.p) return false;
    const long long d = (long long)(b.p - a.p);
    if (a.ld == b.ld) {
        // row j of b starts r bytes behind the start of row j + k of a
        const long long k = floor_div(d, a.ld), r = d - k * a.ld;
        auto some = [&](long long k) {                   // both rows j and j + k exist
            return (k < 0 ? -k : 0) < (b.n < a.n - k ? b.n : a.n - k);
        };
        return (r < a.width && some(k)) || (r + b.width > a.ld && some(k + 1));
    }
    // each row of a: the first row of b that ends behind its start
    for (long long i = 0; i < a.n; i++) {
        const long long lo = i * a.ld - d;               // from b's first row
        const long long j = lo < b.width ? 0 : floor_div(lo - b.width, b.ld) + 1;
        if (j < b.n && j * b.ld < lo + a.width) return true;
    }
    return false;
}

inline bool overlaps_any(const Rows &y, const Rows *others, int n)
{
    for (int i = 0; i < n; i++)
        if (overlap(y, others[i])) return true;
    return false;
}

}  // namespace qg
