// What the kernels of the rule over a tree of drafted tokens share.
//
// Math.  With A_j the path to node j (itself included), G_j the sum of g over A_j and S_0 the
// state before the tree, unrolling S_j = e^{g_j} (I - beta_j k_j k_j^T) S_parent + beta_j k_j v_j^T
// along the path gives S_j = e^{G_j} S_0 + sum_{i in A_j} e^{G_j - G_i} k_i u_i^T, so
//     u_j = beta_j (v_j - e^{G_j} S_0^T k_j) - sum_{i in A_j, i < j} N_ji u_i,  N_ji = beta_j e^{G_j - G_i} k_j . k_i
//     o_j = e^{G_j} S_0^T q_j + sum_{i in A_j} P_ji u_i,                       P_ji = e^{G_j - G_i} q_j . k_i
// which is a chunk of the rule with the chain's triangle replaced by the tree's paths.
#pragma once

#include "gdr_common.cuh"
#include "gdr_internal.h"
#include "gdr_tree.cuh"

namespace gdr {
namespace tree {

// A sequence's tree and gates of one V head, in shared memory.
struct Nodes {
    uint64_t mask[kMaxNodes];
    float2 sum[kMaxNodes];  // G_j as the sum of two floats
    float grown[kMaxNodes];  // e^{G_j}
    float beta[kMaxNodes];
    uint8_t order[kMaxNodes];      // the nodes level by level
    uint8_t start[kMaxNodes + 1];  // where a level starts among them
    int levels;
};

// e^{G_t - G_i}.  Sums of 64 gates reach -100 and more, where a float is 2^-18 coarse; their
// difference may be small, and the exponential takes it as a relative error.  So sums are
// doubles, kept as two floats each.
__device__ __forceinline__ float decay(float2 t, float2 i) { return expf((t.x - i.x) + (t.y - i.y)); }

// A gate as it enters the sums.  e^{-10^4} is zero, and so is every factor over such a gate; what is
// lower (minus infinity, a state that is forgotten) would leave no difference of sums behind it.
__device__ __forceinline__ double gate(float g) { return g < -1e4f ? -1e4 : (double)g; }

// By one warp; `lead`: of the block that reports what is wrong with the tree.
__device__ __forceinline__ void load_nodes(Nodes &s, const Args &a, int seq, int h, int32_t *err, bool lead) {
    const int lane = threadIdx.x & 31, n = a.fixed_len;
    const int64_t row0 = (int64_t)seq * n;
    double sum[2];
    float b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = lane + 32 * i;
        sum[i] = j < n ? gate(a.g[(row0 + j) * a.h_v + h]) : 0.0;
        b[i] = j < n ? a.beta[(row0 + j) * a.h_v + h] : 0.f;
    }
    const Masks m = masks<true>(load_parents(a.parents + row0, n, lane), n, lane, sum);
    if (lead && m.bad) atomicCAS(err, 0, (int32_t)GDR_ERR_INVALID_ARG);
    int depth[2], deepest = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = lane + 32 * i;
        depth[i] = __popcll(m.a[i]);
        deepest = max(deepest, depth[i]);
        const float hi = (float)sum[i], lo = (float)(sum[i] - (double)hi);
        s.mask[j] = m.a[i];
        s.sum[j] = make_float2(hi, lo);
        s.grown[j] = expf(hi) * (1.f + lo);
        s.beta[j] = a.beta_logits ? 1.f / (1.f + expf(-b[i])) : b[i];
    }
    deepest = __reduce_max_sync(0xffffffffu, deepest);
    int at = 0;
    const uint32_t below = (1u << lane) - 1u;
    for (int d = 1; d <= deepest; ++d) {
        const uint32_t b0 = __ballot_sync(0xffffffffu, depth[0] == d), b1 = __ballot_sync(0xffffffffu, depth[1] == d);
        if (lane == 0) s.start[d - 1] = (uint8_t)at;
        if (depth[0] == d) s.order[at + __popc(b0 & below)] = (uint8_t)lane;
        if (depth[1] == d) s.order[at + __popc(b0) + __popc(b1 & below)] = (uint8_t)(lane + 32);
        at += __popc(b0) + __popc(b1);
    }
    if (lane == 0) {
        s.start[deepest] = (uint8_t)at;
        s.levels = deepest;
    }
}

// The corrections and outputs, level by level: the nodes of a level depend on none of each
// other, so the block's threads take COLS columns of THREADS / COLS of them at a time, and a
// tree of a few levels has a few dependent steps whatever it holds.  Only a node's ancestors
// are looked at: what the others hold (infinities, NaNs) cannot reach it.
//   su   [n][LD] in: beta_j (v_j - e^{G_j} S_0^T k_j); out: u_j
//   so   [n][LD] e^{G_j} S_0^T q_j
//   np   [n][ld_np] N and P
// Starts and ends with a barrier of the block.
template <int COLS, int THREADS, int LD>
__device__ __forceinline__ void sweep(const Nodes &s, float *su, const float *so, const float2 *np, int ld_np,
                                      const Args &a, int64_t row0, int h, int col0) {
    constexpr int AT_ONCE = THREADS / COLS;
    const int c = threadIdx.x % COLS, w = threadIdx.x / COLS, n = a.fixed_len;
    auto store = [&](int t, float o, float u) {
        const int64_t at = ((row0 + t) * a.h_v + h) * a.d + col0 + c;
        store_out(a.o, at, o, a.out_bf16);
        if (a.deltas) a.deltas[at] = u;
    };
    for (int t = w; t < n; t += AT_ONCE)
        if (s.mask[t] == 0) store(t, 0.f, 0.f);
    __syncthreads();
    for (int level = 0; level < s.levels; ++level) {
        const int end = s.start[level + 1];
        for (int x = s.start[level] + w; x < end; x += AT_ONCE) {
            const int t = s.order[x];
            const float2 *const row = np + t * ld_np;
            float u = su[t * LD + c], o = so[t * LD + c];
            uint64_t up = s.mask[t] & ~(1ull << t);
            int left = __popcll(up);
            auto next = [&] {
                const int i = __ffsll((long long)up) - 1;
                up &= up - 1;
                return i;
            };
            for (; left >= 4; left -= 4) {
                int i[4];
                float2 f[4];
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) i[e] = next();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[e] = row[i[e]];
                    v[e] = su[i[e] * LD + c];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    u = fmaf(-f[e].x, v[e], u);
                    o = fmaf(f[e].y, v[e], o);
                }
            }
            for (; left > 0; --left) {
                const int i = next();
                const float2 f = row[i];
                const float v = su[i * LD + c];
                u = fmaf(-f.x, v, u);
                o = fmaf(f.y, v, o);
            }
            su[t * LD + c] = u;
            store(t, a.scale * fmaf(row[t].y, u, o), u);
        }
        __syncthreads();
    }
}

}  // namespace tree
}  // namespace gdr
