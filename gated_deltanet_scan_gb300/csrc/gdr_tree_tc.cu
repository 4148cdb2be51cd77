// The gated delta rule over trees of drafted tokens, bf16 inputs, on tcgen05 tensor cores.
//
// Formulas: gdr_tree_rule.cuh, with the corrections solved for: the unit triangular I + N, whose
// row j has entries at j's ancestors only, has an inverse T with entries at the same places, so
//     u_j = sum_{i in A_j} T_ji R_i,   o_j = e^{G_j} S_0^T q_j + sum_{i in A_j} W_ji R_i,   W = P T,
// R_j = beta_j (v_j - e^{G_j} S_0^T k_j).  T and W need no state: they are ready when it arrives,
// and the rest is two products a state column enters, both on the tensor cores.
//
// A block of 512 threads has one (sequence, V head), four threads one of the state's columns.
// The first product, X^T = S_0^T [K; Q]^T, has M = d columns, N = 2 n nodes and inner size d, so
// the state is the operand that lives in TMEM: a thread reads its quarter of a column from memory
// (32 lanes, 128 bytes a row), splits each value exactly into three bf16 parts and stores them at
// its lane, and gets its column's products back there.  The second, [U; O]^T = R^T [T; W]^T, has
// inner size n: R, split likewise, is made from the first's results in the same lanes.  Neither
// passes through shared memory.  Of the nine products of parts, the six that reach 2^-24 are made.
//
//   K, Q   cp.async into the swizzled operand layout, rows [0, r) and [r, 2 r), r = n rounded
//          up to 16
//   Gram   [K; Q] K^T, to shared memory, and from there N and P: a list of its ancestors for
//          every node
//   T, W   level by level (a node's row needs its ancestors' rows); an ancestor's own ancestors are
//          the list's first entries, so entry r of node j is -sum_s N_js (entry r of ancestor s)
//   parts  of the state: middle and low, then, over them, high: TMEM holds two parts (128 columns at
//          d = 128) and the products (128) of two blocks an SM; small parts first, so that their
//          sums round small
//
// A node's rows of T and W are zero but at its ancestors, and zero times an infinity or NaN would
// reach it: such values of R (rare) enter the product as zeros and are added afterwards to the
// nodes whose path they are on.
//
// Bound by instructions, which is what every choice here saves: the same sums over the lists of
// ancestors, a thread a column, took 48,000 warp instructions a block at 64 nodes.
//
// d < 128 leaves lanes (and warps) idle.
#include "gdr_attn.h"
#include "gdr_attn_mma.cuh"
#include "gdr_attn_ptx.cuh"
#include "gdr_tree_rule.cuh"
#include "tc_ptx.cuh"

namespace gdr {
namespace {

using namespace tc;

constexpr int NT = 512;
constexpr int kShares = NT / 128;  // threads of a column
constexpr int kNodes = tree::kMaxNodes;
constexpr int GL = kNodes + 1;  // floats of a Gram row in shared memory
constexpr int kEntries = kNodes * (kNodes - 1) / 2;  // of the ancestors' lists
constexpr uint32_t kCols = 256;

// Shared memory: K and Q, then the Gram products.  T and W lie over the end of these, and their
// bf16 parts, [T; W] of 128 rows each, over K, Q and the rest.
struct Shape {
    static constexpr uint32_t BLOCK = 128 * 128;  // 128 rows, 64 columns
    static constexpr uint32_t OFF_GRAM = 2 * BLOCK;
    static constexpr uint32_t OFF_TW = 3 * BLOCK;
    static constexpr uint32_t OFF_LIST = OFF_TW + 16896;  // float4 each
    static_assert(OFF_LIST >= OFF_GRAM + 128 * GL * 4 && OFF_LIST >= OFF_TW + kEntries * 8, "the two fit");
    static constexpr uint32_t OFF_PAIR = OFF_LIST + kNodes * 128 * 4;  // the lists' place holds R, where it is needed
    static_assert(kNodes * 128 * 4 >= kEntries * 16, "the lists");
    static constexpr uint32_t BYTES = OFF_PAIR + kEntries * 4;
    static_assert(3 * BYTES > 228 * 1024, "two blocks, whose TMEM fits, are all that an SM takes");
};

// One, or eight, columns of this thread's lane (complete after pair::tmem_store_wait).
__device__ __forceinline__ void tmem_store8(uint32_t taddr, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_store1(uint32_t taddr, uint32_t r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(r) : "memory");
}

// Eight columns of this thread's lane, complete after pair::tmem_load_wait.
__device__ __forceinline__ void tmem_load8_start(uint32_t taddr, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

// x as three bf16 values whose sum is x (24 bits), two neighbours packed.
__device__ __forceinline__ void split3(float a, float b, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    auto cut = [](float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); };
    hi = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
    const float ra = a - cut(a), rb = b - cut(b);
    mid = __byte_perm(__float_as_uint(ra), __float_as_uint(rb), 0x7632);
    lo = __byte_perm(__float_as_uint(ra - cut(ra)), __float_as_uint(rb - cut(rb)), 0x7632);
}

template <int D, typename Out>
__global__ void __launch_bounds__(NT, 2) tree_tc_kernel(const __grid_constant__ Args a, int32_t *err) {
    using Sh = Shape;
    constexpr uint32_t A0 = 0, A1 = D / 2, X = 128, PART = 32;  // TMEM columns; PART: of R's parts, from 0
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(8) uint64_t s_bar[4];
    __shared__ uint32_t s_tmem;
    __shared__ uint64_t s_mask[kNodes], s_real;  // s_real: the rows that are nodes
    __shared__ float2 s_sum[kNodes];
    __shared__ float s_grown[kNodes], s_beta[kNodes], s_rq[kNodes];
    __shared__ int s_start[kNodes];      // where a node's list starts: the lists lie level by level
    __shared__ int s_level[kNodes + 1];  // where those of a level do
    __shared__ int s_levels;
    __shared__ float4 s_gate[kNodes];   // beta, e^G / |k|, e^G / |q|, P_jj
    float *const s_gram = reinterpret_cast<float *>(smem + Sh::OFF_GRAM);
    float2 *const s_tw = reinterpret_cast<float2 *>(smem + Sh::OFF_TW);
    float4 *const s_list = reinterpret_cast<float4 *>(smem + Sh::OFF_LIST);
    // an entry's node, its ancestor and where the node's list starts: t | i << 8 | start << 16
    uint32_t *const s_pair = reinterpret_cast<uint32_t *>(smem + Sh::OFF_PAIR);
    const uint32_t base = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int h = blockIdx.x % a.h_v, seq = blockIdx.x / a.h_v, hq = h / (a.h_v / a.h_qk);
    const int n = a.fixed_len, nr = (n + 15) & ~15;
    const int64_t row0 = (int64_t)seq * n;
    // the warps of a column block (TMEM lanes) share its inner values, its nodes and its Gram columns
    const int col = tid & 127, share = warp >> 2;
    const bool work = col - lane < D;
    uint32_t bar[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) bar[i] = smem_u32(s_bar + i);

    // ---- every load of the block is on its way before anything is waited for, the tree's first
    int2 parents;
    float gate_in[2], beta_in[2];
    if (warp == 0) {
        parents = tree::load_parents(a.parents + row0, n, lane);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = lane + 32 * i;
            gate_in[i] = j < n ? a.g[(row0 + j) * a.h_v + h] : 0.f;
            beta_in[i] = j < n ? a.beta[(row0 + j) * a.h_v + h] : 0.f;
        }
    }
    {
        constexpr int CPR = D / 8, RPI = NT / CPR;  // 16-byte chunks of a row, rows at a time
        const int c = tid % CPR;
        const int64_t step = (int64_t)a.h_qk * D, first = (row0 * a.h_qk + hq) * D + c * 8;
        const uint32_t to = base + (c >> 3) * Sh::BLOCK;
#pragma unroll 1
        for (int t = tid / CPR; t < n; t += RPI) {
            const int64_t at = first + t * step;
            attn::cp_async16(to + sw128_offset(t, c & 7), static_cast<const uint16_t *>(a.k) + at, 16u);
            attn::cp_async16(to + sw128_offset(nr + t, c & 7), static_cast<const uint16_t *>(a.q) + at, 16u);
        }
        attn::cp_async_commit();
    }
    constexpr int KX = D / kShares, k0w = KX / 2;  // inner values of a thread, and TMEM columns they take
    float x[KX];
    if (work) {
        const float *const state = a.state + (((int64_t)seq * a.h_v + h) * D + share * KX) * D + col;
#pragma unroll
        for (int i = 0; i < KX; ++i) x[i] = __ldcs(state + i * D);
    }
    if (warp == 0) {
        double sum[2] = {(double)gate_in[0], (double)gate_in[1]};
        const tree::Masks m = tree::masks<true>(parents, n, lane, sum);
        if (m.bad && h == 0) atomicCAS(err, 0, (int32_t)GDR_ERR_INVALID_ARG);
        int depth[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = lane + 32 * i;
            const float hi = (float)sum[i], lo = (float)(sum[i] - (double)hi);
            s_mask[j] = m.a[i];
            s_sum[j] = make_float2(hi, lo);
            s_grown[j] = expf(hi) * (1.f + lo);
            s_beta[j] = a.beta_logits ? 1.f / (1.f + expf(-beta_in[i])) : beta_in[i];
            depth[i] = __popcll(m.a[i]);
        }
        const uint32_t real[2] = {__ballot_sync(0xffffffffu, m.a[0] != 0), __ballot_sync(0xffffffffu, m.a[1] != 0)};
        if (lane == 0) s_real = (uint64_t)real[1] << 32 | real[0];
        const int levels = __reduce_max_sync(0xffffffffu, max(depth[0], depth[1]));
        const uint32_t below = (1u << lane) - 1u;
        int at = 0;
#pragma unroll 1
        for (int d = 0; d < levels; ++d) {  // d ancestors
            const uint32_t b0 = __ballot_sync(0xffffffffu, depth[0] == d + 1), b1 = __ballot_sync(0xffffffffu, depth[1] == d + 1);
            if (lane == 0) s_level[d] = at;
            if (depth[0] == d + 1) s_start[lane] = at + __popc(b0 & below) * d;
            if (depth[1] == d + 1) s_start[lane + 32] = at + (__popc(b0) + __popc(b1 & below)) * d;
            at += (__popc(b0) + __popc(b1)) * d;
        }
        if (lane == 0) {
            s_level[levels] = at;
            s_levels = levels;
        }
    } else if (warp == 1) {
        tmem_alloc(smem_u32(&s_tmem), kCols);
        tmem_relinquish();
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) mbar_init(bar[i], 1);
            fence_mbar_init();
        }
        __syncwarp();
    }
    attn::cp_async_wait<0>();
    fence_proxy_async_smem();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = s_tmem, lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint64_t kq = smem_desc_sw128(base, 0, 1024);
    bool ok = true;

    // ---- Gram products [K; Q] K^T, a row per lane; the ancestors' lists beside them
    if (warp == 0 && elect_one()) {
        const uint32_t id = idesc_bf16_f32(128, nr, 0, 0);
#pragma unroll 1
        for (int k = 0; k < D / 16; ++k) {
            const uint64_t at = kq + (((k >> 2) * Sh::BLOCK + (k & 3) * 32) >> 4);
            mma_bf16(tmem + X, at, at, id, k > 0);
        }
        mma_commit(bar[0]);
    }
    __syncwarp();
    if (tid < n && s_mask[tid] != 0) {
        uint64_t up = s_mask[tid] & ~(1ull << tid);
        int e = s_start[tid];
        const uint32_t rest = (uint32_t)e << 16 | tid;
#pragma unroll 1
        for (; up; up &= up - 1) s_pair[e++] = rest | (uint32_t)(__ffsll((long long)up) - 1) << 8;
    }
    if (a.qk_norm) {  // |q_t|: eight lanes a row
        const int r = tid >> 3;
        float sq = 0.f;
#pragma unroll
        for (int c = 0; c < D / 8; c += 8) {
            if (c + (tid & 7) >= D / 8 || r >= n) continue;
            const uint4 w = *reinterpret_cast<const uint4 *>(smem + (c >> 3) * Sh::BLOCK + sw128_offset(nr + r, tid & 7));
            const uint32_t y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float lo = __uint_as_float(y[i] << 16), hi = __uint_as_float(y[i] & 0xFFFF0000u);
                sq = fmaf(lo, lo, fmaf(hi, hi, sq));
            }
        }
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, d);
        if ((tid & 7) == 0 && r < n) s_rq[r] = l2norm_scale(sq);
    }
    __syncwarp();
    ok = pair::wait_bounded(bar[0], 0) && ok;
    __syncwarp();
    tc_fence_after_sync();
    if (16 * share < nr) {
        uint32_t y[16];
        pair::tmem_load16(lanes + X + 16 * share, y);
        if (col < 2 * nr) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s_gram[col * GL + 16 * share + i] = __uint_as_float(y[i]);
        }
    }
    if (tid < n && !a.qk_norm) s_rq[tid] = 1.f;
    tc_fence_before_sync();
    __syncthreads();
    const int levels = s_levels, entries = s_level[levels];
    auto unit = [&](int t) { return a.qk_norm ? l2norm_scale(s_gram[t * GL + t]) : 1.f; };  // 1 / |k_t|
#pragma unroll 1
    for (int e = tid; e < entries; e += NT) {
        const int t = s_pair[e] & 255, i = s_pair[e] >> 8 & 255;
        const float f = tree::decay(s_sum[t], s_sum[i]) * unit(i);
        s_list[e] = make_float4(s_beta[t] * f * unit(t) * s_gram[t * GL + i], f * s_rq[t] * s_gram[(nr + t) * GL + i],
                                __int_as_float(s_start[i]), 0.f);
    }
    if (tid < kNodes) {
        float4 gate = make_float4(0.f, 0.f, 0.f, 0.f);
        if (tid < n) {
            const float rk = unit(tid);
            gate = make_float4(s_beta[tid], s_grown[tid] * rk, s_grown[tid] * s_rq[tid],
                               s_rq[tid] * rk * s_gram[(nr + tid) * GL + tid]);
        }
        s_gate[tid] = gate;
    }
    __syncthreads();

    // ---- T and W: entry r of a node with d ancestors, by the first share's threads
    if (share == 0) {
        auto finish = [&](int e, int t, float m, float w) {
            const float4 f = s_list[e];
            const float y = -(f.x + m);
            s_tw[e] = make_float2(y, fmaf(s_gate[t].w, y, f.y + w));
        };
#pragma unroll 1
        for (int d = 1; d < levels; ++d) {
            const int e0 = s_level[d], e1 = s_level[d + 1];
            if (d <= 8) {  // a thread an entry, its up to seven terms at once
#pragma unroll 1
                for (int e = e0 + tid; e < e1; e += 128) {
                    const uint32_t p = s_pair[e];
                    const int at = p >> 16, r = e - at;
                    float4 f[7];
                    float y[7], m = 0.f, w = 0.f;
#pragma unroll
                    for (int s = 0; s < 7; ++s) {
                        if (s + 1 >= d) break;
                        f[s] = s_list[at + min(r + 1 + s, d - 1)];
                    }
#pragma unroll
                    for (int s = 0; s < 7; ++s) {
                        if (s + 1 >= d) break;
                        y[s] = r + 1 + s < d ? s_tw[__float_as_int(f[s].z) + r].x : 0.f;
                        m = fmaf(f[s].x, y[s], m);
                        w = fmaf(f[s].y, y[s], w);
                    }
                    finish(e, p & 255, m, w);
                }
            } else {  // eight lanes an entry
#pragma unroll 1
                for (int e4 = e0 + (tid >> 5) * 4; e4 < e1; e4 += 16) {  // whole warps
                    const int e = min(e4 + (lane >> 3), e1 - 1), at = s_pair[e] >> 16, r = e - at;
                    float m = 0.f, w = 0.f;
#pragma unroll 1
                    for (int s = r + 1 + (tid & 7); s < d; s += 8) {
                        const float4 f = s_list[at + s];
                        const float y = s_tw[__float_as_int(f.z) + r].x;
                        m = fmaf(f.x, y, m);
                        w = fmaf(f.y, y, w);
                    }
#pragma unroll
                    for (int y = 1; y < 8; y <<= 1) {
                        m += __shfl_xor_sync(0xffffffffu, m, y);
                        w += __shfl_xor_sync(0xffffffffu, w, y);
                    }
                    if ((tid & 7) == 0 && e4 + (lane >> 3) < e1) finish(e, s_pair[e] & 255, m, w);
                }
            }
            named_sync(1, 128);
        }
    }

    // ---- the state's parts, and its products with K and Q
    uint32_t hi[k0w];
    auto store_part = [&](uint32_t at, const uint32_t *w) {
        if constexpr (k0w == 16) {
            pair::tmem_store16(lanes + at + share * 16, w);
        } else {
#pragma unroll
            for (int i = 0; i < k0w; ++i) tmem_store1(lanes + at + share * k0w + i, w[i]);
        }
    };
    if (work) {
        uint32_t mid[k0w], lo[k0w];
#pragma unroll
        for (int i = 0; i < k0w; ++i) split3(x[2 * i], x[2 * i + 1], hi[i], mid[i], lo[i]);
        store_part(A0, lo);
        store_part(A1, mid);
        pair::tmem_store_wait();
    }
    tc_fence_before_sync();
    __syncthreads();
    const uint32_t id_x = idesc_bf16_f32(128, 2 * nr, 0, 0);
    auto products = [&](bool first) {  // the two parts in place, or the last
#pragma unroll 1
        for (int i = 0; i < (first ? 2 : 1) * (D / 16); ++i) {
            const int k = i % (D / 16);
            pair::mma_ts_one(tmem + X, tmem + A0 + i * 8, kq + (((k >> 2) * Sh::BLOCK + (k & 3) * 32) >> 4), id_x,
                             !first || i > 0);
        }
    };
    if (warp == 0) {
        tc_fence_after_sync();
        if (elect_one()) {
            products(true);
            mma_commit(bar[1]);
        }
        __syncwarp();
    }
    // this thread's values on their way
    const int64_t step = (int64_t)a.h_v * D, out0 = (row0 * a.h_v + h) * D + col;
    constexpr int KN = kNodes / kShares;
    const int t0 = share * KN;
    uint32_t v[KN];
    if (work && t0 < n) {
        const uint16_t *const from = static_cast<const uint16_t *>(a.v) + out0;
#pragma unroll
        for (int i = 0; i < KN; ++i) v[i] = from[min(t0 + i, n - 1) * step];
    }
    ok = pair::wait_bounded(bar[1], 0) && ok;
    __syncwarp();
    if (work) {
        tc_fence_after_sync();
        store_part(A0, hi);
        pair::tmem_store_wait();
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after_sync();
        if (elect_one()) {
            products(false);
            mma_commit(bar[2]);
        }
        __syncwarp();
    }

    // ---- R, its parts, and T's and W's
    ok = pair::wait_bounded(bar[2], 0) && ok;
    __syncwarp();
    tc_fence_after_sync();
    // no MMA reads K and Q any more
    for (int x = tid; x < 2 * nr * 8; x += NT) {
#pragma unroll
        for (int p = 0; p < 3; ++p) *reinterpret_cast<uint4 *>(smem + p * Sh::BLOCK + x * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    float qs[KN];
    bool odd = false;  // some R is an infinity or NaN
    static_assert(KN == 16, "a share's nodes are one TMEM load");
    uint32_t r[KN];
    const uint32_t real = (uint32_t)(s_real >> t0);  // bit i: row t0 + i is a node
    if (work && t0 < nr) {
        float most = 0.f;
#pragma unroll
        for (int i0 = 0; i0 < KN; i0 += 8) {
            uint32_t x[16];
            tmem_load8_start(lanes + X + t0 + i0, x);
            tmem_load8_start(lanes + X + nr + t0 + i0, x + 8);
            pair::tmem_load_wait(x);
#pragma unroll
            for (int i = i0; i < i0 + 8; ++i) {
                const float4 gate = s_gate[t0 + i];
                const float y = gate.x * (__uint_as_float(v[i] << 16) - gate.y * __uint_as_float(x[i - i0]));
                r[i] = real >> i & 1 ? __float_as_uint(y) : 0u;
                most = fmaf(__uint_as_float(r[i]), 0.f, most);  // NaN from the first infinity or NaN on
                qs[i] = gate.z * __uint_as_float(x[8 + i - i0]);
            }
        }
        odd = most != 0.f;
    }
    odd = __syncthreads_or(odd);
    float *const s_r = reinterpret_cast<float *>(smem + Sh::OFF_LIST);  // the lists' N and P are no longer needed
    if (work && t0 < nr) {
        uint32_t part[3][KN / 2];
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            if (!odd) break;
            if (t0 + i < n) s_r[(t0 + i) * D + col] = __uint_as_float(r[i]);
            if ((r[i] & 0x7F800000u) == 0x7F800000u) r[i] = 0u;
        }
#pragma unroll
        for (int i = 0; i < KN / 2; ++i)
            split3(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]), part[0][i], part[1][i], part[2][i]);
#pragma unroll
        for (int p = 0; p < 3; ++p) tmem_store8(lanes + p * PART + t0 / 2, part[p]);
        pair::tmem_store_wait();
    }
    for (int e = tid; e < entries + n; e += NT) {  // the ancestors, and the node itself
        const int t = e < entries ? s_pair[e] & 255 : e - entries, i = e < entries ? s_pair[e] >> 8 & 255 : t;
        const float2 f = e < entries ? s_tw[e] : make_float2(1.f, s_gate[t].w);
        uint32_t hi, mid, lo;
        split3(f.x, f.y, hi, mid, lo);
        uint8_t *const at = smem + sw128_offset(t, i >> 3) + (i & 7) * 2, *const aw = smem + sw128_offset(nr + t, i >> 3) + (i & 7) * 2;
        const uint32_t part[3] = {hi, mid, lo};
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            *reinterpret_cast<uint16_t *>(at + p * Sh::BLOCK) = (uint16_t)part[p];
            *reinterpret_cast<uint16_t *>(aw + p * Sh::BLOCK) = (uint16_t)(part[p] >> 16);
        }
    }
    fence_proxy_async_smem();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after_sync();
        if (elect_one()) {
            auto pass = [&](int r_part, int t_part, bool first) {
#pragma unroll
                for (int k = 0; k < kNodes / 16; ++k) {
                    if (k * 16 >= nr) break;
                    pair::mma_ts_one(tmem + X, tmem + r_part * PART + k * 8, kq + ((t_part * Sh::BLOCK + k * 32) >> 4), id_x,
                                     !first || k > 0);
                }
            };
            pass(2, 0, true);
            pass(1, 1, false);
            pass(0, 2, false);
            pass(1, 0, false);
            pass(0, 1, false);
            pass(0, 0, false);
            mma_commit(bar[3]);
        }
        __syncwarp();
    }
    ok = pair::wait_bounded(bar[3], 0) && ok;
    __syncwarp();
    if (work && t0 < n) {
        tc_fence_after_sync();
        uint32_t u[KN], o[KN];
        pair::tmem_load16(lanes + X + t0, u);
        pair::tmem_load16(lanes + X + nr + t0, o);
#pragma unroll
        for (int i = 0; i < KN; ++i) o[i] = __float_as_uint(qs[i] + __uint_as_float(o[i]));
        if (odd) {
#pragma unroll
            for (int i = 0; i < KN; ++i) {
                if (t0 + i >= n) break;
                const uint64_t mask = s_mask[t0 + i];
                const int at = s_start[t0 + i];
                float x = __uint_as_float(u[i]), y = __uint_as_float(o[i]);
                int e = 0;
#pragma unroll 1
                for (uint64_t up = mask; up; up &= up - 1, ++e) {
                    const float w = s_r[(__ffsll((long long)up) - 1) * D + col];
                    if (isfinite(w)) continue;
                    const float2 f = up & (up - 1) ? s_tw[at + e] : make_float2(1.f, s_gate[t0 + i].w);
                    x = fmaf(f.x, w, x);
                    y = fmaf(f.y, w, y);
                }
                u[i] = __float_as_uint(x);
                o[i] = __float_as_uint(y);
            }
        }
        Out *to = static_cast<Out *>(a.o) + out0 + t0 * step;
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            if (t0 + i >= n) break;
            const float y = real >> i & 1 ? a.scale * __uint_as_float(o[i]) : 0.f;
            if constexpr (sizeof(Out) == 2)
                *to = __float2bfloat16_rn(y);
            else
                *to = y;
            to += step;
        }
        if (a.deltas) {
            float *to_u = a.deltas + out0 + t0 * step;
#pragma unroll
            for (int i = 0; i < KN; ++i) {
                if (t0 + i >= n) break;
                *to_u = real >> i & 1 ? __uint_as_float(u[i]) : 0.f;
                to_u += step;
            }
        }
    }
    if (!ok) {
        // a wait gave up: leave the MMAs in flight time to end before their operands go
        atomicCAS(err, 0, (int32_t)GDR_ERR_DEVICE_TIMEOUT);
        const long long t_end = clock64() + 4000000;
        while (clock64() < t_end) {}
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, kCols);
}

template <int D, typename Out>
cudaError_t launch_as(const Args &a, int32_t *err, cudaStream_t s) {
    static attn::SmemOptIn opt_in;
    const cudaError_t e = opt_in.set(reinterpret_cast<const void *>(tree_tc_kernel<D, Out>), (int)Shape::BYTES);
    if (e != cudaSuccess) return e;
    tree_tc_kernel<D, Out><<<(unsigned)((int64_t)a.n_seqs * a.h_v), NT, Shape::BYTES, s>>>(a, err);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch(const Args &a, int32_t *err, cudaStream_t s) {
    return a.out_bf16 ? launch_as<D, __nv_bfloat16>(a, err, s) : launch_as<D, float>(a, err, s);
}

}  // namespace

cudaError_t launch_tree_tc(const Args &a, int32_t *err, cudaStream_t s) {
    if (a.d == 32) return launch<32>(a, err, s);
    if (a.d == 64) return launch<64>(a, err, s);
    return launch<128>(a, err, s);
}

}  // namespace gdr
