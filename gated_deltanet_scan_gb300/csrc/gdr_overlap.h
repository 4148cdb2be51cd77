// Whether strided rows overlap one another (plain C++, no CUDA).
#pragma once

#include <stdint.h>

namespace gdr {
namespace attn {

// True if some two of the n0 x n1 pieces of d values at i * s0 + j * s1 overlap.
inline bool overlap(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int d) {
    if (n0 <= 1) s0 = INT64_MAX;  // a stride that is never used
    if (n1 <= 1) s1 = INT64_MAX;
    if (s0 > s1) return overlap(n1, s1, n0, s0, d);
    if (s0 < d) return true;
    if (n1 <= 1 || (s1 - d) / s0 >= n0 - 1) return false;  // a run of n0 ends before the next one starts
    // runs reach into each other: piece j of the longer stride against the nearest two of the first run
    for (int64_t j = 1; j < n1; ++j) {
        const unsigned __int128 at = (unsigned __int128)j * (uint64_t)s1;
        const unsigned __int128 i = at / (uint64_t)s0;
        if (i > (uint64_t)n0 - 1) return false;
        const int64_t past = (int64_t)(at % (uint64_t)s0);
        if (past < d || (i + 1 < (uint64_t)n0 && s0 - past < d)) return true;
    }
    return false;
}

}  // namespace attn
}  // namespace gdr
