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
#include "gdr_attn_ptx.cuh"
#include "gdr_tree_rule.cuh"
#include "tc_ptx.cuh"

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
// Bound by HBM: the state is read and written once.  Before it can change, the tree, the gates'
// sums, the keys and the corrections are four dependent loads, about 4 us, so what matters is
// how many bytes of states an SM has on their way meanwhile.  tree_commit_kernel, for batches,
// has a block of 256 threads per (sequence, V head) and brings its whole state into shared
// memory with bulk copies, 192 KiB an SM.  tree_commit_rows_kernel, for a few, has ROWS rows of a
// state in registers, so that one sequence spreads over the GPU.

// The accepted path of a sequence for one V head, by a warp: its nodes in rising order and their
// weights e^{G_a - G_i}.  Returns their number; `grown` is e^{G_a}.
struct Path {
    int node[tree::kMaxNodes];
    float weight[tree::kMaxNodes];
    float grown;
    int count;
};
__device__ __forceinline__ void load_path(Path &s, const Args &a, int seq, int h, int32_t *err, bool lead) {
    const int lane = threadIdx.x & 31, n = a.fixed_len;
    const int64_t row0 = (int64_t)seq * n;
    const int last = a.last[seq];
    const int2 parents = tree::load_parents(a.parents + row0, n, lane);
    double sum[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = lane + 32 * i;
        sum[i] = j < n ? tree::gate(a.g[(row0 + j) * a.h_v + h]) : 0.0;
    }
    const tree::Masks m = tree::masks<true>(parents, n, lane, sum);
    uint64_t path = tree::mask_of(m, last & 63);
    if (last < 0 || last >= n) path = 0;
    const int count = __popcll(path);
    if ((m.bad || last < -1 || (last >= 0 && count == 0)) && lead) atomicCAS(err, 0, (int32_t)GDR_ERR_INVALID_ARG);
    const double s0 = __shfl_sync(0xffffffffu, sum[0], last & 31), s1 = __shfl_sync(0xffffffffu, sum[1], last & 31);
    const double total = last & 32 ? s1 : s0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = lane + 32 * i;
        if (!(path >> j & 1)) continue;
        const int at = __popcll(path & ((1ull << j) - 1));
        s.node[at] = j;
        s.weight[at] = expf((float)(total - sum[i]));
    }
    if (lane == 0) {
        s.grown = expf((float)total);
        s.count = count;
    }
}

// A node's key row at `at`, by a warp: lane's values e, e + 32, ... times its weight (and 1 / |k|).
template <int D>
__device__ __forceinline__ void load_key(float (&k)[D / 32], const Args &a, int64_t at, float weight) {
    const int lane = threadIdx.x & 31;
    float sq = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
        k[e] = load_in(a.k, at + lane + 32 * e, a.in_bf16);
        sq = fmaf(k[e], k[e], sq);
    }
    if (a.qk_norm) weight *= l2norm_scale(warp_sum(sq));
#pragma unroll
    for (int e = 0; e < D / 32; ++e) k[e] *= weight;
}

template <int D, int ROWS>
__global__ void __launch_bounds__(NT) tree_commit_rows_kernel(const __grid_constant__ Args a, int32_t *err) {
    constexpr int Q4 = D / 4, RSTEP = NT / Q4, NR = ROWS / RSTEP, NPART = D / ROWS;
    static_assert(NR >= 1 && NR * RSTEP == ROWS && NPART * ROWS == D && ROWS <= 32, "rows of a thread");
    __shared__ float sK[tree::kMaxNodes][ROWS];
    __shared__ Path s;
    const int part = blockIdx.x % NPART, h = blockIdx.x / NPART % a.h_v, seq = blockIdx.x / (NPART * a.h_v);
    const int hq = h / (a.h_v / a.h_qk), rbase = part * ROWS;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cq = tid % Q4, r0 = tid / Q4;
    const int64_t row0 = (int64_t)seq * a.fixed_len;
    float4 *const state = reinterpret_cast<float4 *>(a.state + (((int64_t)seq * a.h_v + h) * D + rbase) * D);
    float4 x[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) x[i] = state[(r0 + i * RSTEP) * Q4 + cq];
    if (warp == 0) load_path(s, a, seq, h, err, part == 0 && h == 0);
    __syncthreads();
    const int count = s.count;
    if (count == 0) return;  // nothing accepted: the state stays as it is
    constexpr int U = 4;
    float4 u[U];
    const float *const deltas = a.deltas + (row0 * a.h_v + h) * D + 4 * cq;
    auto load_u = [&](int i0) {
#pragma unroll
        for (int e = 0; e < U; ++e)
            u[e] = *reinterpret_cast<const float4 *>(deltas + (int64_t)s.node[min(i0 + e, count - 1)] * a.h_v * D);
    };
    load_u(0);
    for (int i = warp; i < count; i += NT / 32) {
        float k[D / 32];
        load_key<D>(k, a, ((row0 + s.node[i]) * a.h_qk + hq) * D, s.weight[i]);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
            const int r = lane + 32 * e - rbase;
            if (r >= 0 && r < ROWS) sK[i][r] = k[e];
        }
    }
    __syncthreads();
    const float grown = s.grown;
#pragma unroll
    for (int i = 0; i < NR; ++i) x[i] = make_float4(grown * x[i].x, grown * x[i].y, grown * x[i].z, grown * x[i].w);
    for (int i0 = 0; i0 < count; i0 += U) {
#pragma unroll
        for (int e = 0; e < U; ++e) {
            if (i0 + e >= count) break;
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const float w = sK[i0 + e][r0 + i * RSTEP];
                x[i].x = fmaf(w, u[e].x, x[i].x);
                x[i].y = fmaf(w, u[e].y, x[i].y);
                x[i].z = fmaf(w, u[e].z, x[i].z);
                x[i].w = fmaf(w, u[e].w, x[i].w);
            }
        }
        if (i0 + U < count) load_u(i0 + U);
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) state[(r0 + i * RSTEP) * Q4 + cq] = x[i];
}

template <int D>
__global__ void __launch_bounds__(NT) tree_commit_kernel(const __grid_constant__ Args a, int32_t *err) {
    constexpr int Q4 = D / 4, RSTEP = NT / Q4, NR = D / RSTEP;
    constexpr int U = 4, GROUP = 16;  // nodes a thread, and the block, takes at a time
    constexpr uint32_t BYTES = D * D * 4, COPIES = BYTES > 16384 ? BYTES / 16384 : 1;
    extern __shared__ __align__(128) uint8_t held[];
    __shared__ __align__(8) uint64_t s_bar;
    __shared__ Path s;
    float4 *const sS = reinterpret_cast<float4 *>(held);
    float *const sK = reinterpret_cast<float *>(held + BYTES);  // [GROUP / U][D][U]
    const int h = blockIdx.x % a.h_v, seq = blockIdx.x / a.h_v, hq = h / (a.h_v / a.h_qk);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cq = tid % Q4, r0 = tid / Q4;
    const int64_t row0 = (int64_t)seq * a.fixed_len;
    float *const state = a.state + (int64_t)blockIdx.x * D * D;
    const uint32_t bar = tc::smem_u32(&s_bar);
    if (tid == 32) {
        tc::mbar_init(bar, 1);
        tc::fence_mbar_init();
        tc::mbar_arrive_expect_tx(bar, BYTES);
#pragma unroll
        for (uint32_t i = 0; i < COPIES; ++i)
            tc::bulk_load(tc::smem_u32(held) + i * (BYTES / COPIES), state + i * (BYTES / COPIES / 4), BYTES / COPIES, bar);
    }
    if (warp == 0) load_path(s, a, seq, h, err, h == 0);
    __syncthreads();
    const int count = s.count;
    float4 u[U];
    const float *const deltas = a.deltas + (row0 * a.h_v + h) * D + 4 * cq;
    auto load_u = [&](int i0) {
#pragma unroll
        for (int e = 0; e < U; ++e)
            u[e] = __ldcs(reinterpret_cast<const float4 *>(deltas + (int64_t)s.node[min(i0 + e, count - 1)] * a.h_v * D));
    };
    if (count > 0) load_u(0);
    bool ok = true;
    for (int g0 = 0; g0 < count; g0 += GROUP) {
        if (g0 > 0) __syncthreads();  // the group before is done with the keys
        const int g1 = min(g0 + GROUP, count);
        for (int i = g0 + warp; i < ((g1 + U - 1) & ~(U - 1)); i += NT / 32) {
            float k[D / 32];
            load_key<D>(k, a, ((row0 + s.node[min(i, count - 1)]) * a.h_qk + hq) * D, i < g1 ? s.weight[i] : 0.f);
#pragma unroll
            for (int e = 0; e < D / 32; ++e)
                sK[((i - g0) / U * D + lane + 32 * e) * U + (i - g0) % U] = i < g1 ? k[e] : 0.f;
        }
        __syncthreads();
        if (g0 == 0) {
            ok = __syncthreads_and(pair::wait_bounded(bar, 0));
            if (!ok) break;
        }
        for (int i0 = g0; i0 < g1; i0 += U) {
            const bool first = i0 == 0, last = i0 + U >= count;
            const float grown = first ? s.grown : 1.f;
            const float4 *const k = reinterpret_cast<const float4 *>(sK) + (i0 - g0) / U * D;
#pragma unroll
            for (int e = 0; e < U; ++e)
                if (i0 + e >= count) u[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int i = 0; i < NR; ++i) {
                const int r = r0 + i * RSTEP;
                float4 x = sS[r * Q4 + cq];
                const float4 w = k[r];
                x.x = fmaf(w.x, u[0].x, fmaf(w.y, u[1].x, fmaf(w.z, u[2].x, fmaf(w.w, u[3].x, grown * x.x))));
                x.y = fmaf(w.x, u[0].y, fmaf(w.y, u[1].y, fmaf(w.z, u[2].y, fmaf(w.w, u[3].y, grown * x.y))));
                x.z = fmaf(w.x, u[0].z, fmaf(w.y, u[1].z, fmaf(w.z, u[2].z, fmaf(w.w, u[3].z, grown * x.z))));
                x.w = fmaf(w.x, u[0].w, fmaf(w.y, u[1].w, fmaf(w.z, u[2].w, fmaf(w.w, u[3].w, grown * x.w))));
                if (last)
                    __stcs(reinterpret_cast<float4 *>(state) + r * Q4 + cq, x);
                else
                    sS[r * Q4 + cq] = x;
            }
            if (!last) load_u(i0 + U);
        }
    }
    if (count == 0) ok = __syncthreads_and(pair::wait_bounded(bar, 0));  // the copies land before the block goes
    if (!ok && tid == 0) {  // a wait gave up: the state stays as it was
        atomicCAS(err, 0, (int32_t)GDR_ERR_DEVICE_TIMEOUT);
        pair::wait_bounded(bar, 0);
    }
    if (!ok) __syncthreads();
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

// States up to which the kernel of a few rows a block commits them.  Measured on 32-node trees, us, rows
// against whole states: 32 states of d = 128 4.4 / 5.8, 64 4.8 / 6.1, 128 6.1 / 6.1, 256 9.4 / 8.0,
// 2048 65 / 47; of d = 64 4.4 / 4.6, 4.6 / 4.8, 5.1 / 4.8, 7.7 / 5.1, 36 / 15.
constexpr int64_t kFewStates = 64;

template <int D, int ROWS>
cudaError_t launch_commit_as(const Args &a, int32_t *err, cudaStream_t s) {
    const int64_t states = (int64_t)a.n_seqs * a.h_v;
    if (states <= kFewStates) {
        tree_commit_rows_kernel<D, ROWS><<<(unsigned)(states * (D / ROWS)), NT, 0, s>>>(a, err);
        return cudaGetLastError();
    }
    constexpr int bytes = D * D * 4 + 16 * D * 4;
    static attn::SmemOptIn opt_in;
    const cudaError_t e = opt_in.set(reinterpret_cast<const void *>(tree_commit_kernel<D>), bytes);
    if (e != cudaSuccess) return e;
    tree_commit_kernel<D><<<(unsigned)states, NT, bytes, s>>>(a, err);
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
    return launch_commit_as<128, 32>(a, err, s);
}

}  // namespace gdr
