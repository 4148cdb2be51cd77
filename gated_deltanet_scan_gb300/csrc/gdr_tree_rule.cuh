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
    float2 sum[kMaxNodes];   // G_j as the sum of two floats
    float grown[kMaxNodes];  // e^{G_j}
    float beta[kMaxNodes];
    uint16_t start[kMaxNodes + 1];  // where the list of a node's path starts
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
    int at = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = lane + 32 * i, length = __popcll(m.a[i]);
        const float hi = (float)sum[i], lo = (float)(sum[i] - (double)hi);
        s.mask[j] = m.a[i];
        s.sum[j] = make_float2(hi, lo);
        s.grown[j] = expf(hi) * (1.f + lo);
        s.beta[j] = a.beta_logits ? 1.f / (1.f + expf(-b[i])) : b[i];
        int upto = length;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += y;
        }
        s.start[j] = (uint16_t)(at + upto - length);
        at += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane == 0) s.start[kMaxNodes] = (uint16_t)at;
}

}  // namespace tree
}  // namespace gdr
