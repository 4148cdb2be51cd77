// Position rotation of new queries and keys, and the append of keys and values to
// the paged cache, in one pass.
//
// Math.  A token at position p turns pair i of every query and key head by the
// angle a = p f_i:  (x, y) -> (x cos a - y sin a, x sin a + y cos a).  The angle is
// reduced in 64-bit fixed point: f_i / 2 pi modulo one turn is held as a fraction
// of 2^64 (from the float's bits and the 64 leading bits of 1 / 2 pi: off by 2^-62 of
// itself), p times it wraps around exactly, and the top 32 bits of the product are
// the signed fraction of a turn.  At p = 2^24 they are off by a step or two of 2^-32 turns
// for frequencies of a few hundred (by 2^-21 turns at 2^20, the largest); cos and sin take
// them as a float, off by up to 2^-26 turns.  A 32-bit float product p f would be off by whole
// radians.
//
// Bound by HBM for prompts (every row read once, every output written once) and by
// latency for a few tokens.  One 16-byte vector (8 values) per lane, d / 8 lanes a
// row: a lane keeps the same 8 values of every row it handles, so cos and sin are
// computed once per token and lane and serve all of the token's heads.  A step's
// vectors are loaded a step ahead, the first ones before the token's position is
// known.  A pair's other half is in the same vector (interleaved), in another lane of
// the row (halves a multiple of 8 apart: shuffles) or read again by value (other
// halves).  A row is read whole by its warp before any of it is written, so outputs
// may be the inputs.
//
// Of a tree of drafted tokens a node's position is that of its path's end, and its slot the
// row's: the warp walks up from its row while its first vectors are on their way (32 trees of 64 rows,
// 48 heads of 128: 16.4 us; with the masks of whole trees, which other kernels need, 16.8).
#include "gdr_attn_common.cuh"
#include "gdr_internal.h"
#include "gdr_tree.cuh"

namespace gdr {
namespace attn {
namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 4;  // row vectors in flight per lane

struct Split {
    int tokens;  // consecutive tokens per warp
    int parts;   // warps that share a token's rows
};

// kInterleaved and kShuffle: a lane's 8 values are all rotated or all copied.  kRagged:
// interleaved, the rotated part ends inside a vector.
enum Pairing { kNone, kInterleaved, kRagged, kShuffle, kByValue };

__host__ __device__ constexpr int blocks_per_sm(int pairing) { return pairing == kRagged || pairing == kByValue ? 3 : 5; }

// f / 2 pi modulo 1, as a fraction of 2^64: f = +-M 2^E exactly, and M times the 64
// leading bits of 1 / 2 pi is an integer of 88 bits.
__device__ __forceinline__ uint64_t turn_of(float f) {
    constexpr uint64_t kInvTwoPi = 0x28BE60DB9391054Aull;  // floor(2^64 / (2 pi))
    const uint32_t u = __float_as_uint(f);
    const int e = (u >> 23) & 0xFF;
    const uint64_t m = (u & 0x7FFFFFu) | (e ? 0x800000u : 0u);
    const int down = 150 - (e ? e : 1);  // -E: at least 4 below 2^20
    const uint64_t lo = m * kInvTwoPi, hi = __umul64hi(m, kInvTwoPi);
    const uint64_t t = down <= 0 ? lo : down < 64 ? (lo >> down) | (hi << (64 - down)) : down < 128 ? hi >> (down - 64) : 0;
    return u >> 31 ? 0 - t : t;
}

template <int D, bool F16, int PAIR, bool TREE>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(PAIR))
    append_kernel(const __grid_constant__ Args a, const Split sp) {
    constexpr bool kPaired = PAIR == kInterleaved || PAIR == kRagged;
    constexpr bool kWhole = PAIR == kInterleaved || PAIR == kShuffle;
    constexpr int LPR = D / 8;    // lanes per row
    constexpr int RPW = 32 / LPR;  // rows per warp and step
    const int lane = threadIdx.x & 31;
    const int64_t warp = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t chunk = warp / sp.parts;
    const int part = (int)(warp - chunk * sp.parts);
    const int64_t first = chunk * sp.tokens;
    if (first >= a.t_total) return;
    const int64_t last = min(first + sp.tokens, a.t_total);
    const int vec = lane % LPR, sub = lane / LPR;
    const int e0 = vec * 8;
    const int half = a.rot / 2;

    const int n_q = a.q.p ? a.h_q : 0;
    const int rows = n_q + 2 * a.h_kv;
    const int stride = sp.parts * RPW;  // between a lane's rows
    uint4 next[kUnroll];                // vectors of the step to come
    auto row_of = [&](int64_t t, int r) -> const uint16_t * {
        r = min(r, rows - 1);
        const Rows &x = r < n_q ? a.q : r < n_q + a.h_kv ? a.k : a.v;
        const int h = r < n_q ? r : r < n_q + a.h_kv ? r - n_q : r - n_q - a.h_kv;
        return x.p + t * x.ts + h * x.hs;
    };
    auto load = [&](int64_t t, int r0) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            next[u] = *reinterpret_cast<const uint4 *>(row_of(t, r0 + u * stride + sub) + e0);
    };
    load(first, part * RPW);

    // fractions of a turn per position of this lane's 8 values
    uint64_t turn[kPaired ? 4 : 8];
    if constexpr (PAIR != kNone) {
        constexpr int N = kPaired ? 4 : 8;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int x = kPaired ? e0 / 2 + e : e0 + e;  // pair, or value
            const int i = kPaired ? x : (x < half ? x : x - half);
            turn[e] = i < half ? turn_of(a.inv_freq[i]) : 0;
        }
    }

    const int even = (int)(a.t_total / a.n_seqs);  // tokens per sequence without cu
    int s = a.cu ? find_seq_warp(a.cu, a.n_seqs, first, lane) : (int)(first / even);

    int2 parents = make_int2(-2, -2);
    int parents_of = -1;  // the sequence whose they are

    for (int64_t t = first; t < last; ++t) {
        int64_t t0, t1;
        bool known = true;
        if (!TREE && a.cu) {
            while (s + 1 < a.n_seqs && a.cu[s + 1] <= t) ++s;
            t0 = a.cu[s];
            t1 = a.cu[s + 1];
            known = t0 >= 0 && t0 <= t && t < t1 && t1 <= a.t_total;
        } else {
            while (t >= (int64_t)(s + 1) * even) ++s;
            t0 = (int64_t)s * even;
            t1 = t0 + even;
        }
        int64_t pos = known ? (int64_t)a.kv_lens[s] - (t1 - t) : -1;
        int64_t turned_by = pos;  // the position the angles go by
        if constexpr (TREE) {
            if (s != parents_of) {
                parents_of = s;
                parents = tree::load_parents(a.parents + t0, even, lane);
            }
            const int j = (int)(t - t0);
            bool bad;
            const int depth = tree::depth_of(parents, j, bad);
            if (bad) record_invalid(a.err);
            known = depth >= 0;  // the row is a node
            turned_by = pos - j + depth;
            if (pos < j) pos = -1;  // fewer tokens than the tree has rows
        }
        int64_t slot = -1;  // offset of the token's slot in the cache, in elements
        if (pos >= 0 && pos < (int64_t)a.cache.max_pages * a.cache.page_size) {
            const int pg = (int)pos / a.cache.page_size;
            const int page = a.cache.table[(int64_t)s * a.cache.table_stride + pg];
            if (page >= 0 && page < a.cache.n_pages)
                slot = page * a.cache.page_stride +
                       (int64_t)((int)pos - pg * a.cache.page_size) * a.cache.token_stride;
        }
        if (slot < 0 && (!TREE || known)) record_invalid(a.err);

        float cs[8], sn[8];
        if constexpr (PAIR != kNone) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (kPaired && (e & 1)) {
                    cs[e] = cs[e - 1];
                    sn[e] = -sn[e - 1];
                } else {
                    const int32_t w =
                        (int32_t)(((uint64_t)turned_by * turn[kPaired ? e / 2 : e]) >> 32);
                    sincospif((float)w * 4.656612873077393e-10f, &sn[e], &cs[e]);  // 2^-31 half turns
                    if (kPaired || e0 + e < half) sn[e] = -sn[e];
                }
            }
        }

        for (int r0 = part * RPW; r0 < rows; r0 += stride * kUnroll) {
            uint4 w[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) w[u] = next[u];
            if (r0 + stride * kUnroll < rows)
                load(t, r0 + stride * kUnroll);
            else if (t + 1 < last)
                load(t + 1, part * RPW);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int r = r0 + u * stride + sub;
                if constexpr (PAIR != kNone) {
                    const uint32_t own[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
                    uint32_t oth[4];  // the pairs' other values
                    if constexpr (kPaired) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) oth[i] = __byte_perm(own[i], 0, 0x1032);
                    } else if constexpr (PAIR == kShuffle) {
                        const int h8 = half >> 3;
                        const int from = vec < h8 ? lane + h8 : lane - h8;
#pragma unroll
                        for (int i = 0; i < 4; ++i) oth[i] = __shfl_sync(0xffffffffu, own[i], from & 31);
                    } else {
                        const uint16_t *const src = row_of(t, r);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t o2 = 0;
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const int x = e0 + 2 * i + j;
                                if (x < a.rot && r < n_q + a.h_kv)
                                    o2 |= (uint32_t)src[x < half ? x + half : x - half] << (16 * j);
                            }
                            oth[i] = o2;
                        }
                    }
                    if (r < n_q + a.h_kv && e0 < a.rot) {
                        uint32_t res[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 x = unpack2<F16>(own[i]), y = unpack2<F16>(oth[i]);
                            const float lo = x.x * cs[2 * i] + y.x * sn[2 * i];
                            const float hi = x.y * cs[2 * i + 1] + y.y * sn[2 * i + 1];
                            res[i] = pack2<F16>(lo, hi);
                            if constexpr (!kWhole) {  // values past the rotated part are copied bit for bit
                                const int e = e0 + 2 * i;
                                res[i] = (e < a.rot ? res[i] & 0xFFFFu : own[i] & 0xFFFFu) |
                                         (e + 1 < a.rot ? res[i] & 0xFFFF0000u : own[i] & 0xFFFF0000u);
                            }
                        }
                        w[u] = make_uint4(res[0], res[1], res[2], res[3]);
                    }
                }
            }
            if constexpr (PAIR == kByValue) __syncwarp();  // every value read before any is written
            if (!known) continue;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int r = r0 + u * stride + sub;
                if (r >= rows) continue;
                if (r < n_q) {
                    *reinterpret_cast<uint4 *>(a.q_out.p + t * a.q_out.ts + r * a.q_out.hs + e0) = w[u];
                } else {
                    const bool is_k = r < n_q + a.h_kv;
                    const int h = is_k ? r - n_q : r - n_q - a.h_kv;
                    if (is_k && a.k_out.p)
                        *reinterpret_cast<uint4 *>(a.k_out.p + t * a.k_out.ts + h * a.k_out.hs + e0) = w[u];
                    if (slot >= 0)
                        *reinterpret_cast<uint4 *>((is_k ? a.cache.k : a.cache.v) + slot + h * a.cache.head_stride +
                                                   e0) = w[u];
                }
            }
        }
    }
}

template <int D, bool F16, bool TREE>
void launch_as(const Args &a, int pairing, const Split &sp, unsigned blocks, cudaStream_t s) {
    switch (pairing) {
        case kNone: append_kernel<D, F16, kNone, TREE><<<blocks, kThreads, 0, s>>>(a, sp); break;
        case kInterleaved: append_kernel<D, F16, kInterleaved, TREE><<<blocks, kThreads, 0, s>>>(a, sp); break;
        case kRagged: append_kernel<D, F16, kRagged, TREE><<<blocks, kThreads, 0, s>>>(a, sp); break;
        case kShuffle: append_kernel<D, F16, kShuffle, TREE><<<blocks, kThreads, 0, s>>>(a, sp); break;
        default: append_kernel<D, F16, kByValue, TREE><<<blocks, kThreads, 0, s>>>(a, sp); break;
    }
}
template <int D, bool F16>
void launch(const Args &a, int pairing, const Split &sp, unsigned blocks, cudaStream_t s) {
    if (a.parents)
        launch_as<D, F16, true>(a, pairing, sp, blocks, s);
    else
        launch_as<D, F16, false>(a, pairing, sp, blocks, s);
}

}  // namespace

cudaError_t launch_append(const Args &a, cudaStream_t s) {
    const int rpw = 32 / (a.d / 8);
    const int rows = (a.q.p ? a.h_q : 0) + 2 * a.h_kv;
    const int pairing = a.rot == 0                ? kNone
                        : a.interleaved         ? (a.rot % 8 == 0 ? kInterleaved : kRagged)
                        : (a.rot / 2) % 8 == 0 ? kShuffle
                                               : kByValue;
    // One warp per token and all its rows where there are tokens enough for the warps the
    // GPU holds at once, several tokens per warp beyond that (one wave: 32 warps an SM in
    // one and a half waves took 147 us where one wave takes 124 us, at 29204 tokens); with
    // fewer tokens a token's rows are shared out, down to one step of a warp each.
    const int64_t want = 152 * (kThreads / 32) * blocks_per_sm(pairing);
    Split sp{1, 1};
    if (a.t_total >= want) {
        sp.tokens = (int)((a.t_total + want - 1) / want);
    } else {
        const int64_t steps = (rows + rpw - 1) / rpw;
        const int64_t parts = want / a.t_total;
        sp.parts = (int)(parts < steps ? parts : steps);
    }
    const int64_t warps = (a.t_total + sp.tokens - 1) / sp.tokens * sp.parts;
    const unsigned blocks = (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32));
    if (a.d == 64)
        a.f16 ? launch<64, true>(a, pairing, sp, blocks, s) : launch<64, false>(a, pairing, sp, blocks, s);
    else if (a.d == 128)
        a.f16 ? launch<128, true>(a, pairing, sp, blocks, s) : launch<128, false>(a, pairing, sp, blocks, s);
    else
        a.f16 ? launch<256, true>(a, pairing, sp, blocks, s) : launch<256, false>(a, pairing, sp, blocks, s);
    return cudaGetLastError();
}

}  // namespace attn
}  // namespace gdr
