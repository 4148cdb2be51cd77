// The gated delta rule over trees of drafted tokens: the kernel of every type and head size,
// and the commit of an accepted path.
//
// Formulas: gdr_tree_rule.cuh.  The state is only read (4 d^2 bytes a V head; a chain's
// verify block, which leaves the state after its last token and a snapshot, moves three
// times that): a tree has no last token.
//
// tree_kernel, for fp32 inputs, is fp32 on CUDA cores: a block has a (sequence, V head), or 32 of its columns
// where there are few, with its queries and keys in shared memory, in whose rows R and e^G S_0^T q take their
// places.  A warp has 16 columns and every so many rows, a thread four columns of an eighth of the state's
// rows in registers, so that a 16-byte load of a key serves 16 FMAs; the eight sums of a thread go round to one
// a lane in seven shuffles.  N and P are made for the paths' entries, and nodes come after their ancestors, so
// two lanes of a column go through the rows in order, four at once, with no barrier of the block.
// Bound by issue slots (64% of them; the FMAs of S_0^T [K; Q] alone would take 16,400 clocks a pair of 64
// nodes and d = 128, of 70,000): 64 trees of 64 nodes, 32 heads: 506 us, 16 of them 152, 16 chains 274 (64 938), 8
// trees of 41 nodes 51, one of 24 15.4 (level by level, 32 columns a block: 2,300, 599, 1,432, 137 and 16.5).  At
// d = 64 and 32 64 trees of 64 take 225 and 135 us, one of 24 15.5 and 14.0.  It stays on CUDA cores: the tensor-core
// kernel takes K and Q as one bf16 part; three of each would be twice the products that make X and three times the
// operand tiles, for which its shared memory, as it is laid out, has no room.
#include "gdr_attn.h"
#include "gdr_attn_mma.cuh"
#include "gdr_attn_ptx.cuh"
#include "gdr_tree_rule.cuh"
#include "tc_ptx.cuh"

namespace gdr {
namespace {

constexpr int NT = 256;

// For n rows: K (then R, then U), Q (then e^G S_0^T q), N and P, the paths (of at most n (n + 1) / 2 entries).
size_t tree_bytes(int n, int d) { return 4 * (size_t)(2 * n * d) + 9 * (size_t)(n * (n + 1) / 2); }

// p[0] = the sum over lanes of p[i], where i is made of the lane's bits from UNIT on: in 2 HALF - 1 shuffles.
template <int HALF, int UNIT>
__device__ __forceinline__ void sums_to_lanes(float *p, int lane) {
#pragma unroll
    for (int m = HALF; m > 0; m >>= 1) {
        const bool upper = lane & UNIT * m;
#pragma unroll
        for (int e = 0; e < m; ++e)
            p[e] = (upper ? p[m + e] : p[e]) + __shfl_xor_sync(0xffffffffu, upper ? p[e] : p[m + e], UNIT * m);
    }
}

// C: columns of a block.
template <int D, int C>
__global__ void __launch_bounds__(NT, D == 128 ? 2 : D == 64 ? 3 : 4) tree_kernel(const __grid_constant__ Args a, int32_t *err) {
    constexpr int W = NT / 32, Q4 = D / 4;
    constexpr int AT_ONCE = 4, GROUPS = W / (C / 16), STEP = AT_ONCE * GROUPS;  // rows of a warp's step, of the block's
    extern __shared__ __align__(16) float smem[];
    __shared__ tree::Nodes s;
    const int n = a.fixed_len;
    float *const sK = smem, *const sQ = sK + n * D;
    float2 *const sNP = reinterpret_cast<float2 *>(sQ + n * D);
    uint8_t *const sPath = reinterpret_cast<uint8_t *>(sNP + n * (n + 1) / 2);
    const int pair = blockIdx.x / (D / C), col0 = blockIdx.x % (D / C) * C;
    const int h = pair % a.h_v, seq = pair / a.h_v, hq = h / (a.h_v / a.h_qk);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row0 = (int64_t)seq * n;
    for (int e = tid; e < n * Q4; e += NT) {
        const int t = e / Q4, x = e % Q4;
        const int64_t from = ((row0 + t) * a.h_qk + hq) * D + 4 * x;
        attn::cp_async16(tc::smem_u32(sK + 4 * e), static_cast<const float *>(a.k) + from, 16u);
        attn::cp_async16(tc::smem_u32(sQ + 4 * e), static_cast<const float *>(a.q) + from, 16u);
    }
    attn::cp_async_commit();
    const int eighth = lane >> 2, col = warp % (C / 16) * 16 + (lane & 3) * 4;  // of the block's
    float4 state[D / 32][4];
    const float *const from = a.state + ((int64_t)seq * a.h_v + h) * D * D + 4 * eighth * D + col0 + col;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) state[i][e] = *reinterpret_cast<const float4 *>(from + (32 * i + e) * D);
    }
    if (warp == 0) tree::load_nodes(s, a, seq, h, err, h == 0 && col0 == 0);
    attn::cp_async_wait<0>();
    __syncthreads();
    if (a.qk_norm) {
        for (int r = warp; r < 2 * n; r += W) {
            float *const x = sK + r * D;  // Q's rows follow K's
            float sq = 0.f;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) sq = fmaf(x[lane + 32 * e], x[lane + 32 * e], sq);
            const float f = l2norm_scale(warp_sum(sq));
#pragma unroll
            for (int e = 0; e < D / 32; ++e) x[lane + 32 * e] *= f;
        }
    }
    if (tid < n) {
        int at = s.start[tid];
        for (uint64_t up = s.mask[tid]; up; up &= up - 1) sPath[at++] = (uint8_t)(__ffsll((long long)up) - 1);
    }
    __syncthreads();
    // N and P, a row per warp, eight of its entries at a time: their 16 sums over the lanes go round to one a
    // pair of lanes in 16 shuffles (N's in the lower half of the warp)
    constexpr int V = D / 32;
    for (int t = warp; t < n; t += W) {
        const int at = s.start[t], count = s.start[t + 1] - at;
        float k[V], q[V];
#pragma unroll
        for (int x = 0; x < V; ++x) {
            k[x] = sK[t * D + lane + 32 * x];
            q[x] = sQ[t * D + lane + 32 * x];
        }
#pragma unroll 1
        for (int r0 = 0; r0 < count; r0 += 8) {
            float p[16];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float *const y = sK + sPath[at + min(r0 + e, count - 1)] * D + lane;
                p[e] = p[8 + e] = 0.f;
#pragma unroll
                for (int x = 0; x < V; ++x) {
                    p[e] = fmaf(k[x], y[32 * x], p[e]);
                    p[8 + e] = fmaf(q[x], y[32 * x], p[8 + e]);
                }
            }
            sums_to_lanes<8, 2>(p, lane);
            p[0] += __shfl_xor_sync(0xffffffffu, p[0], 1);
            const int r = r0 + (lane >> 1 & 7);
            if ((lane & 1) == 0 && r < count) {
                const float f = tree::decay(s.sum[t], s.sum[sPath[at + r]]);
                reinterpret_cast<float *>(sNP + at + r)[lane >> 4] = (lane < 16 ? s.beta[t] : 1.f) * f * p[0];
            }
        }
    }
    // R and e^G S_0^T q
    const bool is_q = lane & 16;  // the sum that goes to this lane, and its column
    const int own = col + (lane >> 2 & 2) + (lane >> 2 & 1);
    float v[AT_ONCE];
    auto load_v = [&](int t0) {
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
            v[u] = 0.f;
            if (!is_q && t0 + u < n) v[u] = static_cast<const float *>(a.v)[((row0 + t0 + u) * a.h_v + h) * D + col0 + own];
        }
    };
    const int first = warp / (C / 16) * AT_ONCE;
    load_v(first);
#pragma unroll 1
    for (int step = 0; step < n; step += STEP) {
        const int t0 = step + first;
        float z[AT_ONCE];
#pragma unroll
        for (int u0 = 0; u0 < AT_ONCE; u0 += 2) {
            float p[2][8] = {};
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int at = min(t0 + u0 + u, n - 1) * D + 32 * i + 4 * eighth;
                    const float4 k = *reinterpret_cast<const float4 *>(sK + at), q = *reinterpret_cast<const float4 *>(sQ + at);
                    const float kx[4] = {k.x, k.y, k.z, k.w}, qx[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float4 w = state[i][e];
                        p[u][0] = fmaf(kx[e], w.x, p[u][0]);
                        p[u][1] = fmaf(kx[e], w.y, p[u][1]);
                        p[u][2] = fmaf(kx[e], w.z, p[u][2]);
                        p[u][3] = fmaf(kx[e], w.w, p[u][3]);
                        p[u][4] = fmaf(qx[e], w.x, p[u][4]);
                        p[u][5] = fmaf(qx[e], w.y, p[u][5]);
                        p[u][6] = fmaf(qx[e], w.z, p[u][6]);
                        p[u][7] = fmaf(qx[e], w.w, p[u][7]);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                sums_to_lanes<4, 4>(p[u], lane);
                z[u0 + u] = p[u][0];
            }
        }
        __syncthreads();  // all warps have read these rows
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
            const int t = t0 + u;
            if (t >= n) break;
            const float x = s.grown[t] * z[u];
            (is_q ? sQ : sK)[t * D + own] = is_q ? x : s.beta[t] * (v[u] - x);
        }
        load_v(t0 + STEP);
    }
    __syncthreads();
    // u and o, some rows at once: two lanes a column sum every other ancestor each of those before these
    // rows, then the rows' own ancestors among them, the last of their lists, are added in order
    constexpr int G = 4;
    if (tid >= 2 * C) return;
    const int c = tid >> 1, half = tid & 1;
    const int64_t out = (row0 * a.h_v + h) * D + col0 + c, step = (int64_t)a.h_v * D;
#pragma unroll 1
    for (int t0 = 0; t0 < n; t0 += G) {
        float u[G], o[G];
        int at[G], before[G], most = 0;
        uint32_t among[G];
#pragma unroll
        for (int x = 0; x < G; ++x) {
            const uint64_t mask = t0 + x < n ? s.mask[t0 + x] : 0;
            u[x] = o[x] = 0.f;
            at[x] = s.start[min(t0 + x, n)];
            before[x] = __popcll(mask & ((1ull << t0) - 1));
            among[x] = (uint32_t)(mask >> t0);
            most = max(most, before[x]);
        }
#pragma unroll 2
        for (int r = half; r < most; r += 2) {
#pragma unroll
            for (int x = 0; x < G; ++x) {
                const bool there = r < before[x];  // without branches, so that all rows' loads are on their way
                const int e = there ? at[x] + r : 0, i = there ? sPath[e] : 0;
                const float2 np = sNP[e];
                const float y = there ? sK[i * D + c] : 0.f;
                u[x] = fmaf(there ? -np.x : 0.f, y, u[x]);
                o[x] = fmaf(there ? np.y : 0.f, y, o[x]);
            }
        }
#pragma unroll
        for (int x = 0; x < G; ++x) {
            const int t = min(t0 + x, n - 1);
            u[x] += __shfl_xor_sync(0xffffffffu, u[x], 1);
            o[x] += __shfl_xor_sync(0xffffffffu, o[x], 1);
            u[x] += sK[t * D + c];
            o[x] += sQ[t * D + c];
        }
        __syncwarp();  // the rows' R are read
#pragma unroll
        for (int x = 0; x < G; ++x) {
            int r = at[x] + before[x];
#pragma unroll
            for (int y = 0; y < x; ++y) {
                if (among[x] >> y & 1) {
                    const float2 np = sNP[r++];
                    u[x] = fmaf(-np.x, u[y], u[x]);
                    o[x] = fmaf(np.y, u[y], o[x]);
                }
            }
            const bool node = among[x] >> x & 1;
            o[x] = node ? a.scale * fmaf(sNP[r].y, u[x], o[x]) : 0.f;
            u[x] = node ? u[x] : 0.f;
            if (node && half == 0) sK[(t0 + x) * D + c] = u[x];
        }
        __syncwarp();
#pragma unroll
        for (int x = 0; x < G; ++x) {
            if (t0 + x >= n) break;
            if (half == 0)
                store_out(a.o, out + (t0 + x) * step, o[x], a.out_bf16);
            else if (a.deltas)
                a.deltas[out + (t0 + x) * step] = u[x];
        }
    }
}

// --- commit: S = e^{G_a} S + sum_{i in A_a} e^{G_a - G_i} k_i u_i^T ------------------------------
//
// Bound by HBM: the state is read and written once.  Before it can change, the tree, the gates'
// sums, the keys and the corrections are four dependent loads, about 4 us, so what matters is
// how many bytes of states an SM has on their way meanwhile.  tree_commit_kernel, for batches,
// has a block of 256 threads per (sequence, V head) and brings its whole state into shared
// memory with bulk copies, 192 KiB an SM.  tree_commit_rows_kernel, for a few, has ROWS rows of a
// state in registers, so that one sequence spreads over the GPU.  64 trees of 64 nodes, 32 heads of 128: 49.6 us,
// 82% of the measured bandwidth; one tree of 24 6.2 us (its bytes would take 0.6).

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

template <int D, int C>
cudaError_t launch_plain(const Args &a, int32_t *err, cudaStream_t s) {
    static attn::SmemOptIn opt_in;
    const cudaError_t e =
        opt_in.set(reinterpret_cast<const void *>(tree_kernel<D, C>), (int)tree_bytes(tree::kMaxNodes, D));
    if (e != cudaSuccess) return e;
    tree_kernel<D, C><<<(unsigned)((int64_t)a.n_seqs * a.h_v * (D / C)), NT, tree_bytes(a.fixed_len, D), s>>>(a, err);
    return cudaGetLastError();
}
// (Sequence, V head) pairs up to which four blocks share one of d = 128: as many as are resident at once.  Trees of
// 64 nodes, us, one block a pair / four: 16 pairs 46.3 / 28.8, 64 47.2 / 39.0, 80 47.2 / 59.5, 256 78 / 132; of 24
// nodes 20.5 / 14.5, 20.6 / 19.3, 21.7 / 28.8, 30.8 / 57.4.
constexpr int64_t kFewPairs = 2 * 152 / 4;

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
    if (a.d == 32) return launch_plain<32, 32>(a, err, s);
    if (a.d == 64) return launch_plain<64, 64>(a, err, s);
    return (int64_t)a.n_seqs * a.h_v <= kFewPairs ? launch_plain<128, 32>(a, err, s) : launch_plain<128, 128>(a, err, s);
}

cudaError_t launch_tree_commit(const Args &a, int32_t *err, cudaStream_t s) {
    if (a.d == 32) return launch_commit_as<32, 32>(a, err, s);
    if (a.d == 64) return launch_commit_as<64, 16>(a, err, s);
    return launch_commit_as<128, 32>(a, err, s);
}

}  // namespace gdr
