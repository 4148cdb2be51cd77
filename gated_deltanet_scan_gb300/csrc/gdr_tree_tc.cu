// The gated delta rule over trees of drafted tokens, bf16 inputs, on tcgen05 tensor cores.
//
// Formulas: gdr_tree_rule.cuh.  A block of 128 threads has one (sequence, V head), a thread one
// of the state's columns.  What the state's columns give is X^T = S_0^T [K; Q]^T, a product of
// M = d columns, N = 2 n nodes and inner size d, so the state is the operand that lives in
// TMEM: a thread reads its column from memory (32 lanes, 128 bytes a row), splits each value
// exactly into three bf16 parts and stores them at its lane, and gets all its column's products
// back there.  The state passes through no shared memory, and the corrections,
// u_j = R_j - sum N_ji u_i over the path, are a column's own business: no barrier between nodes.
//
//   K, Q   cp.async into the swizzled operand layout, rows [0, r) and [r, 2 r), r = n rounded
//          up to 16
//   Gram   [K; Q] K^T, to shared memory, and from there the path's factors: for every node the
//          list of its ancestors, N, P and where their corrections are
//   parts  middle and low, then, over them, high: TMEM holds two parts (128 columns at d = 128) and
//          the products (128) of two blocks an SM; the small parts first, so that their sums round small
//   sweep  nodes in rising order, eight at a time from TMEM; u_i of the ancestors from shared memory
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

constexpr int NT = 128;
constexpr int kNodes = tree::kMaxNodes;
constexpr int GL = kNodes + 1;  // floats of a Gram row in shared memory
constexpr int kEdges = kNodes * (kNodes - 1) / 2;
constexpr uint32_t kCols = 256;

template <int D>
struct Shape {
    static constexpr uint32_t BLOCK = 128 * 128;  // 128 rows, 64 columns
    static constexpr uint32_t KQ = BLOCK * ((D + 63) / 64);
    static constexpr uint32_t OFF_GRAM = KQ;  // later the corrections, [n][D]
    static constexpr uint32_t GRAM = 128 * GL * 4;
    static_assert(GRAM >= kNodes * D * 4, "corrections over the Gram products");
    static constexpr uint32_t OFF_EDGE = OFF_GRAM + GRAM;  // float4 each
    static constexpr uint32_t OFF_PAIR = OFF_EDGE + kEdges * 16;
    static constexpr uint32_t BYTES = OFF_PAIR + kEdges * 2;
    // at least 77 KiB, so that two blocks, whose TMEM fits, are all that an SM takes
    static constexpr uint32_t SMEM = BYTES < 77 * 1024 ? 77 * 1024 : BYTES;
    static constexpr uint32_t A0 = 0, A1 = D / 2, X = 128;  // TMEM columns
};

__device__ __forceinline__ void tmem_load8(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
    pair::tmem_load_wait(r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// x as three bf16 values whose sum is x (24 bits), two neighbours packed.
__device__ __forceinline__ void split3(float a, float b, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    auto cut = [](float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); };
    hi = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
    const float ra = a - cut(a), rb = b - cut(b);
    mid = __byte_perm(__float_as_uint(ra), __float_as_uint(rb), 0x7632);
    lo = __byte_perm(__float_as_uint(ra - cut(ra)), __float_as_uint(rb - cut(rb)), 0x7632);
}

template <int D>
__global__ void __launch_bounds__(NT, 2) tree_tc_kernel(const __grid_constant__ Args a, int32_t *err) {
    using Sh = Shape<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(8) uint64_t s_bar[3];
    __shared__ uint32_t s_tmem;
    __shared__ uint64_t s_mask[kNodes];
    __shared__ float2 s_sum[kNodes];
    __shared__ float s_grown[kNodes], s_beta[kNodes], s_rk[kNodes], s_rq[kNodes];
    __shared__ int s_edge[kNodes + 1];  // where a node's list starts
    __shared__ float4 s_gate[kNodes];   // beta, e^G / |k|, e^G / |q|, P_jj
    float *const s_gram = reinterpret_cast<float *>(smem + Sh::OFF_GRAM);
    float4 *const s_list = reinterpret_cast<float4 *>(smem + Sh::OFF_EDGE);
    uint16_t *const s_pair = reinterpret_cast<uint16_t *>(smem + Sh::OFF_PAIR);
    const uint32_t base = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int h = blockIdx.x % a.h_v, seq = blockIdx.x / a.h_v, hq = h / (a.h_v / a.h_qk);
    const int n = a.fixed_len, nr = (n + 15) & ~15;
    const int64_t row0 = (int64_t)seq * n;
    const bool work = warp < D / 32;
    uint32_t bar[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) bar[i] = smem_u32(s_bar + i);

    // ---- every load of the block is on its way before anything is waited for
    {
        constexpr int CPR = D / 8;
        const uint16_t *const k = static_cast<const uint16_t *>(a.k), *const q = static_cast<const uint16_t *>(a.q);
        for (int e = tid; e < 2 * n * CPR; e += NT) {
            const int r = e / CPR, c = e % CPR, t = r < n ? r : r - n, at = r < n ? t : nr + t;
            attn::cp_async16(base + (c >> 3) * Sh::BLOCK + sw128_offset(at, c & 7),
                             (r < n ? k : q) + ((row0 + t) * a.h_qk + hq) * D + c * 8, 16u);
        }
        attn::cp_async_commit();
    }
    float x[D];
    if (work) {
        const float *const state = a.state + ((int64_t)seq * a.h_v + h) * D * D + tid;
#pragma unroll
        for (int i = 0; i < D; ++i) x[i] = __ldcs(state + i * D);
    }
    if (warp == 0) {
        double sum[2];
        float b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = lane + 32 * i;
            sum[i] = j < n ? (double)a.g[(row0 + j) * a.h_v + h] : 0.0;
            b[i] = j < n ? a.beta[(row0 + j) * a.h_v + h] : 0.f;
        }
        const tree::Masks m = tree::masks<true>(a.parents + row0, n, lane, sum);
        if (m.bad && h == 0) atomicCAS(err, 0, (int32_t)GDR_ERR_INVALID_ARG);
        int before = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = lane + 32 * i;
            const float hi = (float)sum[i], lo = (float)(sum[i] - (double)hi);
            s_mask[j] = m.a[i];
            s_sum[j] = make_float2(hi, lo);
            s_grown[j] = expf(hi) * (1.f + lo);
            s_beta[j] = a.beta_logits ? 1.f / (1.f + expf(-b[i])) : b[i];
            const int edges = max(0, __popcll(m.a[i]) - 1);
            int upto = edges;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, upto, d);
                if (lane >= d) upto += y;
            }
            s_edge[j] = before + upto - edges;
            before += __shfl_sync(0xffffffffu, upto, 31);
        }
        if (lane == 0) s_edge[kNodes] = before;
    } else if (warp == 1) {
        tmem_alloc(smem_u32(&s_tmem), kCols);
        tmem_relinquish();
        if (lane == 0) {
            for (int i = 0; i < 3; ++i) mbar_init(bar[i], 1);
            fence_mbar_init();
        }
        __syncwarp();
    }
    attn::cp_async_wait<0>();
    fence_proxy_async_smem();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = s_tmem, lanes = tmem + ((uint32_t)(warp * 32) << 16);
    const uint64_t kq = smem_desc_sw128(base, 0, 1024);
    bool ok = true;

    // ---- Gram products [K; Q] K^T, a row per lane; the ancestors' lists beside them
    if (warp == 0 && elect_one()) {
        const uint32_t id = idesc_bf16_f32(128, nr, 0, 0);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            const uint64_t at = kq + (((k >> 2) * Sh::BLOCK + (k & 3) * 32) >> 4);
            mma_bf16(tmem + Sh::X, at, at, id, k > 0);
        }
        mma_commit(bar[0]);
    }
    __syncwarp();
    if (tid < n) {
        uint64_t up = s_mask[tid] & ~(1ull << tid);
        for (int e = s_edge[tid]; up; ++e, up &= up - 1)
            s_pair[e] = (uint16_t)(tid << 8 | (__ffsll((long long)up) - 1));
    } else if (a.qk_norm && tid >= 64 && tid < 64 + n) {
        const int t = tid - 64;
        float sq = 0.f;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
            const uint4 w = *reinterpret_cast<const uint4 *>(smem + (c >> 3) * Sh::BLOCK + sw128_offset(nr + t, c & 7));
            const uint32_t y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float lo = __uint_as_float(y[i] << 16), hi = __uint_as_float(y[i] & 0xFFFF0000u);
                sq = fmaf(lo, lo, fmaf(hi, hi, sq));
            }
        }
        s_rq[t] = l2norm_scale(sq);
    }
    __syncwarp();
    ok = pair::wait_bounded(bar[0], 0) && ok;
    __syncwarp();
    tc_fence_after_sync();
#pragma unroll 1
    for (int c = 0; c < nr; c += 16) {
        uint32_t y[16];
        pair::tmem_load16(lanes + Sh::X + c, y);
        if (tid < 2 * nr) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s_gram[tid * GL + c + i] = __uint_as_float(y[i]);
                if (tid < n && c + i == tid) s_rk[tid] = a.qk_norm ? l2norm_scale(__uint_as_float(y[i])) : 1.f;
            }
        }
    }
    if (!a.qk_norm && tid < n) s_rq[tid] = 1.f;

    // ---- the state's parts, and its products with K and Q
    uint32_t hi[D / 2];
    if (work) {
#pragma unroll
        for (int c = 0; c < D / 2; c += 16) {
            uint32_t mid[16], lo[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) split3(x[2 * (c + i)], x[2 * (c + i) + 1], hi[c + i], mid[i], lo[i]);
            pair::tmem_store16(lanes + Sh::A0 + c, lo);
            pair::tmem_store16(lanes + Sh::A1 + c, mid);
        }
        pair::tmem_store_wait();
    }
    tc_fence_before_sync();
    __syncthreads();
    const uint32_t id_x = idesc_bf16_f32(128, 2 * nr, 0, 0);
    auto products = [&](uint32_t part, bool first) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
            pair::mma_ts_one(tmem + Sh::X, tmem + part + k * 8, kq + (((k >> 2) * Sh::BLOCK + (k & 3) * 32) >> 4), id_x,
                             !first || k > 0);
    };
    if (warp == 0) {
        tc_fence_after_sync();
        if (elect_one()) {
            products(Sh::A0, true);
            products(Sh::A1, false);
            mma_commit(bar[1]);
        }
        __syncwarp();
    }
    // the lists' factors, meanwhile
    for (int e = tid; e < s_edge[kNodes]; e += NT) {
        const int t = s_pair[e] >> 8, i = s_pair[e] & 255;
        const float f = tree::decay(s_sum[t], s_sum[i]) * s_rk[i];
        s_list[e] = make_float4(s_beta[t] * f * s_rk[t] * s_gram[t * GL + i], f * s_rq[t] * s_gram[(nr + t) * GL + i],
                                __int_as_float(i * D), 0.f);
    }
    if (tid < n)
        s_gate[tid] = make_float4(s_beta[tid], s_grown[tid] * s_rk[tid], s_grown[tid] * s_rq[tid],
                                  s_rq[tid] * s_rk[tid] * s_gram[(nr + tid) * GL + tid]);
    ok = pair::wait_bounded(bar[1], 0) && ok;
    __syncwarp();
    if (work) {
        tc_fence_after_sync();
#pragma unroll
        for (int c = 0; c < D / 2; c += 16) pair::tmem_store16(lanes + Sh::A0 + c, hi + c);
        pair::tmem_store_wait();
    }
    tc_fence_before_sync();
    __syncthreads();  // and the lists are complete, the Gram products no longer needed
    if (warp == 0) {
        tc_fence_after_sync();
        if (elect_one()) {
            products(Sh::A0, false);
            mma_commit(bar[2]);
        }
        __syncwarp();
    }

    // ---- node by node: this column's corrections and outputs
    if (work) {
        float *const s_u = s_gram + tid;
        const uint16_t *const v = static_cast<const uint16_t *>(a.v) + (row0 * a.h_v + h) * D + tid;
        const int64_t step = (int64_t)a.h_v * D, out0 = (row0 * a.h_v + h) * D + tid;
        uint16_t vn[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) vn[i] = i < n ? v[i * step] : 0;
        ok = pair::wait_bounded(bar[2], 0) && ok;
        __syncwarp();
        tc_fence_after_sync();
#pragma unroll 1
        for (int t0 = 0; t0 < n; t0 += 8) {
            float ks[8], qs[8], vv[8];
            tmem_load8(lanes + Sh::X + t0, ks);
            tmem_load8(lanes + Sh::X + nr + t0, qs);
#pragma unroll
            for (int i = 0; i < 8; ++i) vv[i] = __uint_as_float((uint32_t)vn[i] << 16);
#pragma unroll
            for (int i = 0; i < 8; ++i) vn[i] = t0 + 8 + i < n ? v[(t0 + 8 + i) * step] : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int t = t0 + i;
                if (t >= n) break;
                const float4 gate = s_gate[t];
                float u = gate.x * (vv[i] - gate.y * ks[i]), o = gate.z * qs[i];
                const int end = s_edge[t + 1];
#pragma unroll 4
                for (int e = s_edge[t]; e < end; ++e) {
                    const float4 f = s_list[e];
                    const float w = s_u[__float_as_int(f.z)];
                    u = fmaf(-f.x, w, u);
                    o = fmaf(f.y, w, o);
                }
                s_u[t * D] = u;
                o = a.scale * fmaf(gate.w, u, o);
                if (s_mask[t] == 0) u = o = 0.f;
                store_out(a.o, out0 + t * step, o, a.out_bf16);
                if (a.deltas) a.deltas[out0 + t * step] = u;
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

template <int D>
cudaError_t launch(const Args &a, int32_t *err, cudaStream_t s) {
    static attn::SmemOptIn opt_in;
    const cudaError_t e = opt_in.set(reinterpret_cast<const void *>(tree_tc_kernel<D>), (int)Shape<D>::SMEM);
    if (e != cudaSuccess) return e;
    tree_tc_kernel<D><<<(unsigned)((int64_t)a.n_seqs * a.h_v), NT, Shape<D>::SMEM, s>>>(a, err);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_tc(const Args &a, int32_t *err, cudaStream_t s) {
    if (a.d == 32) return launch<32>(a, err, s);
    if (a.d == 64) return launch<64>(a, err, s);
    return launch<128>(a, err, s);
}

}  // namespace gdr
