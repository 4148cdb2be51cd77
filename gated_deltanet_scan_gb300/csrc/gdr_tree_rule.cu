// The gated delta rule over trees of drafted tokens: the kernel of every type and head size,
// and the commit of an accepted path.
//
// Formulas: gdr_tree_rule.cuh.  The state is only read (4 d^2 bytes a V head; a chain's
// verify block, which leaves the state after its last token and a snapshot, moves three
// times that): a tree has no last token.
//
// tree_kernel is the plain one, in fp32 on CUDA cores: a block of 256 threads has one
// (sequence, V head, 32 columns), its queries and keys as floats and its 32 columns of the
// state in shared memory, a column per lane.
#include "gdr_attn.h"
#include "gdr_tree_rule.cuh"

namespace gdr {
namespace {

constexpr int NT = 256;
constexpr int BV = 32;

template <int D>
struct Shape {
    static constexpr int LDK = D + 4;
    // floats, for n rows: state, K, Q, corrections, outputs, N and P
    static size_t bytes(int n) { return 4 * (size_t)(D * BV + 2 * n * LDK + 2 * n * BV + 2 * n * n); }
};

template <int D>
__global__ void __launch_bounds__(NT) tree_kernel(const __grid_constant__ Args a, int32_t *err) {
    using Sh = Shape<D>;
    extern __shared__ __align__(16) float smem[];
    __shared__ tree::Nodes s;
    const int n = a.fixed_len;
    float *const sS = smem, *const sK = sS + D * BV, *const sQ = sK + n * Sh::LDK, *const sU = sQ + n * Sh::LDK,
                 *const sO = sU + n * BV;
    float2 *const sNP = reinterpret_cast<float2 *>(sO + n * BV);
    constexpr int ncb = D / BV;
    const int cb = blockIdx.x % ncb, h = blockIdx.x / ncb % a.h_v, seq = blockIdx.x / (ncb * a.h_v);
    const int hq = h / (a.h_v / a.h_qk), col0 = cb * BV;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row0 = (int64_t)seq * n;
    const float *const state = a.state + ((int64_t)seq * a.h_v + h) * D * D + col0;

    for (int e = tid; e < D * (BV / 4); e += NT)
        reinterpret_cast<float4 *>(sS)[e] = *reinterpret_cast<const float4 *>(state + e / (BV / 4) * D + e % (BV / 4) * 4);
    if (warp == 0) tree::load_nodes(s, a, seq, h, err, cb == 0 && h == 0);
    for (int e = tid; e < n * D; e += NT) {
        const int t = e / D, x = e % D;
        sK[t * Sh::LDK + x] = load_in(a.k, ((row0 + t) * a.h_qk + hq) * D + x, a.in_bf16);
        sQ[t * Sh::LDK + x] = load_in(a.q, ((row0 + t) * a.h_qk + hq) * D + x, a.in_bf16);
    }
    __syncthreads();
    if (a.qk_norm) {
        for (int r = warp; r < 2 * n; r += NT / 32) {
            float *const x = sK + r * Sh::LDK;  // Q's rows follow K's
            float sq = 0.f;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) sq = fmaf(x[lane + 32 * e], x[lane + 32 * e], sq);
            const float f = l2norm_scale(warp_sum(sq));
#pragma unroll
            for (int e = 0; e < D / 32; ++e) x[lane + 32 * e] *= f;
        }
        __syncthreads();
    }
    // S^T k and S^T q: a column per lane, rows warp, warp + 8, ...
    for (int t0 = warp; t0 < n; t0 += 32) {
        float ks[4] = {0.f, 0.f, 0.f, 0.f}, qs[4] = {0.f, 0.f, 0.f, 0.f};
        for (int x = 0; x < D; x += 4) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = sS[(x + e) * BV + lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = min(t0 + 8 * i, n - 1);
                const float4 k = *reinterpret_cast<const float4 *>(sK + t * Sh::LDK + x);
                const float4 q = *reinterpret_cast<const float4 *>(sQ + t * Sh::LDK + x);
                ks[i] = fmaf(k.x, v[0], fmaf(k.y, v[1], fmaf(k.z, v[2], fmaf(k.w, v[3], ks[i]))));
                qs[i] = fmaf(q.x, v[0], fmaf(q.y, v[1], fmaf(q.z, v[2], fmaf(q.w, v[3], qs[i]))));
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = t0 + 8 * i;
            if (t >= n) break;
            const float v = load_in(a.v, ((row0 + t) * a.h_v + h) * D + col0 + lane, a.in_bf16);
            sU[t * BV + lane] = s.beta[t] * (v - s.grown[t] * ks[i]);
            sO[t * BV + lane] = s.grown[t] * qs[i];
        }
    }
    // N and P where there is a path
    for (int e = tid; e < n * n; e += NT) {
        const int t = e / n, i = e - t * n;
        if (!(s.mask[t] >> i & 1)) continue;
        float kk = 0.f, qk = 0.f;
        for (int x = 0; x < D; x += 4) {
            const float4 k = *reinterpret_cast<const float4 *>(sK + t * Sh::LDK + x);
            const float4 q = *reinterpret_cast<const float4 *>(sQ + t * Sh::LDK + x);
            const float4 y = *reinterpret_cast<const float4 *>(sK + i * Sh::LDK + x);
            kk = fmaf(k.x, y.x, fmaf(k.y, y.y, fmaf(k.z, y.z, fmaf(k.w, y.w, kk))));
            qk = fmaf(q.x, y.x, fmaf(q.y, y.y, fmaf(q.z, y.z, fmaf(q.w, y.w, qk))));
        }
        const float f = tree::decay(s.sum[t], s.sum[i]);
        sNP[e] = make_float2(s.beta[t] * f * kk, f * qk);
    }
    tree::sweep<BV, NT, BV>(s, sU, sO, sNP, n, a, row0, h, col0);
}

// --- commit: S = e^{G_a} S + sum_{i in A_a} e^{G_a - G_i} k_i u_i^T ------------------------------
//
// Bound by HBM: the state is read and written once.  A block of 256 threads has ROWS rows of one
// (sequence, V head)'s state, a thread four columns of ROWS / RSTEP of them; their loads are on
// their way before the path is known.  The path's keys, times their weights, are in shared
// memory, its corrections pass through registers four nodes at a time.
template <int D, int ROWS>
__global__ void __launch_bounds__(NT) tree_commit_kernel(const __grid_constant__ Args a, int32_t *err) {
    constexpr int Q4 = D / 4, RSTEP = NT / Q4, NR = ROWS / RSTEP, NPART = D / ROWS;
    static_assert(NR >= 1 && NR * RSTEP == ROWS && NPART * ROWS == D, "rows of a thread");
    __shared__ float sK[tree::kMaxNodes][ROWS];
    __shared__ float sW[tree::kMaxNodes];
    __shared__ int sNode[tree::kMaxNodes];
    __shared__ int sCount;
    __shared__ float sGrown;
    const int part = blockIdx.x % NPART, h = blockIdx.x / NPART % a.h_v, seq = blockIdx.x / (NPART * a.h_v);
    const int hq = h / (a.h_v / a.h_qk), n = a.fixed_len, rbase = part * ROWS;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cq = tid % Q4, r0 = tid / Q4;
    const int64_t row0 = (int64_t)seq * n;
    float4 *const state = reinterpret_cast<float4 *>(a.state + (((int64_t)seq * a.h_v + h) * D + rbase) * D);
    float4 x[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) x[i] = state[(r0 + i * RSTEP) * Q4 + cq];
    if (warp == 0) {
        const int last = a.last[seq];
        double sum[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = lane + 32 * i;
            sum[i] = j < n ? (double)a.g[(row0 + j) * a.h_v + h] : 0.0;
        }
        const tree::Masks m = tree::masks<true>(tree::load_parents(a.parents + row0, n, lane), n, lane, sum);
        uint64_t path = tree::mask_of(m, last & 63);
        if (last < 0 || last >= n) path = 0;
        const int count = __popcll(path);
        const double s0 = __shfl_sync(0xffffffffu, sum[0], last & 31), s1 = __shfl_sync(0xffffffffu, sum[1], last & 31);
        const double total = last & 32 ? s1 : s0;
        if ((m.bad || last < -1 || (last >= 0 && count == 0)) && part == 0 && h == 0)
            atomicCAS(err, 0, (int32_t)GDR_ERR_INVALID_ARG);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = lane + 32 * i;
            if (!(path >> j & 1)) continue;
            const int at = __popcll(path & ((1ull << j) - 1));
            sNode[at] = j;
            sW[at] = expf((float)(total - sum[i]));
        }
        if (lane == 0) {
            sCount = count;
            sGrown = expf((float)total);
        }
    }
    __syncthreads();
    const int count = sCount;
    if (count == 0) return;  // nothing accepted: the state stays as it is
    if (a.qk_norm) {
        for (int i = warp; i < count; i += NT / 32) {
            float sq = 0.f;
            for (int e = lane; e < D; e += 32) {
                const float v = load_in(a.k, ((row0 + sNode[i]) * a.h_qk + hq) * D + e, a.in_bf16);
                sq = fmaf(v, v, sq);
            }
            sq = warp_sum(sq);
            if (lane == 0) sW[i] *= l2norm_scale(sq);
        }
        __syncthreads();
    }
    for (int e = tid; e < count * ROWS; e += NT) {
        const int i = e / ROWS, r = e % ROWS;
        sK[i][r] = sW[i] * load_in(a.k, ((row0 + sNode[i]) * a.h_qk + hq) * D + rbase + r, a.in_bf16);
    }
    __syncthreads();
    const float grown = sGrown;
#pragma unroll
    for (int i = 0; i < NR; ++i) x[i] = make_float4(grown * x[i].x, grown * x[i].y, grown * x[i].z, grown * x[i].w);
    constexpr int U = 4;
    for (int i0 = 0; i0 < count; i0 += U) {
        float4 u[U];
#pragma unroll
        for (int e = 0; e < U; ++e)
            u[e] = *reinterpret_cast<const float4 *>(
                a.deltas + ((row0 + sNode[min(i0 + e, count - 1)]) * a.h_v + h) * D + 4 * cq);
#pragma unroll
        for (int e = 0; e < U; ++e) {
            if (i0 + e >= count) break;
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const float k = sK[i0 + e][r0 + i * RSTEP];
                x[i].x = fmaf(k, u[e].x, x[i].x);
                x[i].y = fmaf(k, u[e].y, x[i].y);
                x[i].z = fmaf(k, u[e].z, x[i].z);
                x[i].w = fmaf(k, u[e].w, x[i].w);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) state[(r0 + i * RSTEP) * Q4 + cq] = x[i];
}

template <int D>
cudaError_t launch_plain(const Args &a, int32_t *err, cudaStream_t s) {
    const size_t bytes = Shape<D>::bytes(a.fixed_len);
    static attn::SmemOptIn opt_in;
    const cudaError_t e =
        opt_in.set(reinterpret_cast<const void *>(tree_kernel<D>), (int)Shape<D>::bytes(tree::kMaxNodes));
    if (e != cudaSuccess) return e;
    tree_kernel<D><<<(unsigned)((int64_t)a.n_seqs * a.h_v * (D / BV)), NT, bytes, s>>>(a, err);
    return cudaGetLastError();
}

template <int D, int ROWS>
cudaError_t launch_commit_as(const Args &a, int32_t *err, cudaStream_t s) {
    tree_commit_kernel<D, ROWS><<<(unsigned)((int64_t)a.n_seqs * a.h_v * (D / ROWS)), NT, 0, s>>>(a, err);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree(const Args &a, int32_t *err, cudaStream_t s) {
    if (a.in_bf16) return launch_tree_tc(a, err, s);
    if (a.d == 32) return launch_plain<32>(a, err, s);
    if (a.d == 64) return launch_plain<64>(a, err, s);
    return launch_plain<128>(a, err, s);
}

cudaError_t launch_tree_commit(const Args &a, int32_t *err, cudaStream_t s) {
    if (a.d == 32) return launch_commit_as<32, 32>(a, err, s);
    if (a.d == 64) return launch_commit_as<64, 16>(a, err, s);
    return launch_commit_as<128, 16>(a, err, s);
}

}  // namespace gdr
