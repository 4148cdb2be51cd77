// Trees of drafted tokens, from the parents of their nodes.
//
// A sequence's tree is n <= 64 rows; parents[j] is -1 (a child of the last committed
// token), an earlier row, or -2 (no node).  The mask of node j is A_j, the set of j and its
// ancestors, as bits; a row that is no node has mask 0.  Parents come before their
// children, so the bits of A_j in rising order are the path to j, and |A_j| is its length.
//
// A warp holds the tree: lane l has rows l and l + 32.  Masks come by pointer jumping:
// every row adds what the row its pointer names has gathered, and takes over that row's
// pointer, so a path of 64 takes six steps, whatever the tree looks like (a walk would take
// a dependent load per ancestor).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gdr {
namespace tree {

constexpr int kMaxNodes = 64;

__device__ __forceinline__ uint64_t shfl64(uint64_t v, int lane) {
    const uint32_t lo = __shfl_sync(0xffffffffu, (uint32_t)v, lane);
    const uint32_t hi = __shfl_sync(0xffffffffu, (uint32_t)(v >> 32), lane);
    return (uint64_t)hi << 32 | lo;
}

struct Masks {
    uint64_t a[2];  // of rows lane and lane + 32
    bool bad;       // one of them has a parent that cannot be one
};

// Parents of rows lane and lane + 32.
__device__ __forceinline__ int2 load_parents(const int32_t *parents, int n, int lane) {
    return make_int2(lane < n ? parents[lane] : -2, lane + 32 < n ? parents[lane + 32] : -2);
}

// Of a tree of n rows with these parents, by a whole warp.  With SUMS, `sum` holds a number for
// each of the lane's rows, and gets the sum of those of the row's path (0 for no node).
template <bool SUMS = false>
__device__ __forceinline__ Masks masks(int2 parents, int n, int lane, double *sum = nullptr) {
    Masks m;
    int to[2] = {parents.x, parents.y};
    m.bad = false;
    bool node[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = lane + 32 * i;
        if (to[i] < -2 || to[i] >= j) {
            m.bad = m.bad || j < n;
            to[i] = -2;
        }
        node[i] = to[i] != -2;
        m.a[i] = node[i] ? 1ull << j : 0;
        if (SUMS && !node[i]) sum[i] = 0.0;
    }
    if (n <= 32) {
#pragma unroll 1
        for (int step = 1; step < n; step <<= 1) {
            const uint32_t up = __shfl_sync(0xffffffffu, (uint32_t)m.a[0], to[0] & 31);
            const int next = __shfl_sync(0xffffffffu, to[0], to[0] & 31);
            double more = 0.0;
            if (SUMS) more = __shfl_sync(0xffffffffu, sum[0], to[0] & 31);
            if (to[0] >= 0) {
                m.a[0] |= up;
                to[0] = next;
                if (SUMS) sum[0] += more;
            }
        }
    } else {
#pragma unroll 1
        for (int step = 1; step < n; step <<= 1) {
            uint64_t up[2];
            int next[2];
            double more[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint64_t u0 = shfl64(m.a[0], to[i] & 31), u1 = shfl64(m.a[1], to[i] & 31);
                const int t0 = __shfl_sync(0xffffffffu, to[0], to[i] & 31);
                const int t1 = __shfl_sync(0xffffffffu, to[1], to[i] & 31);
                up[i] = to[i] & 32 ? u1 : u0;
                next[i] = to[i] & 32 ? t1 : t0;
                if (SUMS) {
                    const double s0 = __shfl_sync(0xffffffffu, sum[0], to[i] & 31);
                    const double s1 = __shfl_sync(0xffffffffu, sum[1], to[i] & 31);
                    more[i] = to[i] & 32 ? s1 : s0;
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (to[i] >= 0) {
                    m.a[i] |= up[i];
                    to[i] = next[i];
                    if (SUMS) sum[i] += more[i];
                }
            }
        }
    }
    // a path that ends in a row that is no node
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (node[i] && to[i] == -2) {
            m.bad = true;
            m.a[i] = 0;
            if (SUMS) sum[i] = 0.0;
        }
    }
    return m;
}

__device__ __forceinline__ Masks masks(const int32_t *parents, int n, int lane) {
    return masks(load_parents(parents, n, lane), n, lane);
}

// The mask of row j (the same or another for every lane).
__device__ __forceinline__ uint64_t mask_of(const Masks &m, int j) {
    const uint64_t a0 = shfl64(m.a[0], j & 31), a1 = shfl64(m.a[1], j & 31);
    return j & 32 ? a1 : a0;
}

// Ancestors of row j, or -1 where it is no node; `bad`: one of them, or the row, has a parent that cannot be
// one.  By a whole warp, a step per ancestor.
__device__ __forceinline__ int depth_of(int2 parents, int j, bool &bad) {
    int at = j;
    bad = false;
#pragma unroll 1
    for (int depth = 0;; ++depth) {
        const int lo = __shfl_sync(0xffffffffu, parents.x, at & 31), hi = __shfl_sync(0xffffffffu, parents.y, at & 31);
        const int up = at & 32 ? hi : lo;
        if (up == -1) return depth;
        if (up < 0 || up >= at) {
            bad = up != -2 || depth > 0;
            return -1;
        }
        at = up;
    }
}

// 32 bits of what a node sees from slot `rel` on, relative to the tree's first slot: all
// before the tree, then its mask.
__device__ __forceinline__ uint32_t sees32(uint64_t mask, int rel) {
    if (rel <= -32) return ~0u;
    if (rel < 0) return (uint32_t)(mask << -rel) | ((1u << -rel) - 1u);
    return rel < 64 ? (uint32_t)(mask >> rel) : 0u;
}

}  // namespace tree
}  // namespace gdr
