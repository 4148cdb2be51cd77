// Attention of the last few tokens of every sequence over its paged cache.
//
// Math.  For one key/value head the group's queries of the sequence's n_tok tokens
// are rows r = j group + g of one small matrix Q (rows = n_tok group).  Over tiles
// of 16 tokens, with x = scale log2(e) Q K^T and the running row maximum m,
//     p = 2^(x - m),   l += sum p,   O += P V,
// earlier sums rescaled by 2^(m_old - m) when m grows; o = O / l at the end.  Two
// parts of a row's tokens join the same way from their (m, l, O).
//
// Bound by HBM: keys and values are read once (4 h_kv d bytes a token) and little
// else moves.  Two kernels: this file's, for up to 16 rows (a decode step, a few draft
// tokens), and gdr_attn_wide.cu's for more.  The tiles of all (sequence, key/value head,
// row block) triples lie on one line, cut into equal parts, one per worker, so every
// worker streams the same number of tiles whatever the lengths are.  Here a worker is
// one warp with a ring of shared-memory slots of its own, filled by 16-byte asynchronous
// copies several tiles ahead: no warp waits for another, and while one starts or ends a
// sequence the others of its SM keep the memory busy.  Both products are warp-level
// m16n8k16 MMAs on the 16-bit rows with fp32 sums: at 4 flops a byte the tensor pipes are
// far from busy (26%), so the rows they pad cost nothing.  A sequence that one worker sees
// whole is written by it; the others leave (m, l, O): the workers of a block, next to
// each other on the line, join what they can among themselves, and a second kernel, a
// programmatic dependent launch, joins the blocks' parts from the workspace; always in
// the order of the tokens.
//
// Of a tree of drafted tokens (TREE) a row sees what is before the tree and its own path: the worker makes the
// masks of the tree's nodes (gdr_tree.cuh) when it comes to the sequence, and in the tiles that hold the tree
// a score is selected by its bit.  A row that is no node takes the tokens before the tree with the others
// and is undone at the end: its row of the products costs nothing.  64 trees of 4 nodes, 512 to 8,192 tokens: d = 256,
// 16 / 4 heads 141 us (704 MB, 74% of the measured bandwidth), d = 128, 32 / 8, fp16 134 (77%), d = 64, 16 / 4 51
// (51%); one of 4 over 1,500 tokens, d = 256, 18.5.
//
// P enters P V in 16 bits (its sum l does not): that is the only rounding between the
// inputs and the output's own.  fp16 holds 11 bits of a weight.  bf16 holds 8, which added
// as much error as the output's own rounding (64 sequences of d = 256: 0.00226 of o's rms
// against 0.00166 for that rounding alone), so bf16 weights are two operands, cut and
// rest, of a second product each: error 0.00166, 121.3 us instead of 120.4 (one sequence
// of 131,072 tokens 93.4 / 92.7; 64 of 2,000, d = 128, 98.4 / 97.7; of 4,000, d = 64, 58.1 /
// 55.6).
#include "gdr_attn_line.cuh"
#include "gdr_attn_mma.cuh"
#include "gdr_internal.h"
#include "gdr_tree.cuh"
#include "tc_ptx.cuh"

namespace gdr {
namespace attn {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 16;  // tokens: the MMA's inner size in P V

template <int D>
struct Shape {
    static constexpr uint32_t SLOT = kTile * D * 2;
    static constexpr int FIT = 24576 / (int)SLOT;  // 24 KiB of ring per warp, at most 8 slots
    static constexpr int SLOTS = FIT < 8 ? FIT : 8;
    static constexpr uint32_t SMEM = kWarps * SLOTS * SLOT;
    static_assert(SLOTS * SLOT >= 16 * D * 4, "a ring holds its worker's part");
};

template <int D, bool F16, bool TREE>
__global__ void __launch_bounds__(kThreads, 1) decode_kernel(const __grid_constant__ Args a) {
    using Sh = Shape<D>;
    constexpr Spec sp = spec(kFew, D);
    constexpr int TT = kTile / 8;  // 8-token column tiles of S
    constexpr int KS = D / 16;   // inner steps of Q K^T
    constexpr int NT = D / 8;    // output column tiles
    constexpr int CPR = D / 8;   // 16-byte chunks of a row
    constexpr int RPI = 32 / CPR;  // rows one copy instruction of a warp covers
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ Line<kThreads, kWarps> s_line;
    __shared__ int64_t s_cut[kWarps];     // the triple a worker's part ends in, or -1
    __shared__ float2 s_ml[kWarps * 16];  // m and l of its rows

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, wk = tid >> 5, lane = tid & 31;
    const int rows = a.n_tok * a.group;
    const Layout L = layout(rows, sp, D, (int64_t)a.n_seqs * a.h_kv);
    const Cut cut(s_line.place(a, sp, L.blocks_of_rows), kWarps);
    int me;
    Walk walk = s_line.walk(cut, wk, me);
    if (lane == 0) s_cut[wk] = -1;

    const uint32_t slots = tc::smem_u32(ring) + wk * Sh::SLOTS * Sh::SLOT;
    float2 *const ml_parts = reinterpret_cast<float2 *>(static_cast<uint8_t *>(a.ws) + L.ml);
    float *const o_parts = reinterpret_cast<float *>(static_cast<uint8_t *>(a.ws) + L.o);
    const float sc = a.scale * kLog2e;
    const int r0 = lane >> 2, cq = lane & 3;  // the MMA's row (and row + 8) and column pair of this lane

    Triple tr;
    while (walk.next(a, sp, L.blocks_of_rows, tr)) {
        const int s = tr.s, h = tr.h, len = tr.len, tiles = tr.tiles, tile0 = tr.tile0, tile1 = tr.tile1;
        const int64_t seg0 = tr.seg0;
        const int slot_of_part = cut.start(me) >= seg0 ? 0 : 1;
        const int steps = 2 * (tile1 - tile0);  // keys and values of a tile are a step each
        const int32_t *const pages = a.cache.table + (int64_t)s * a.cache.table_stride;
        const int64_t head = h * a.cache.head_stride;

        // Copies: lane % kTile is a token of the tile; its offset serves keys and values.
        int64_t off = 0;   // of the tile whose copies are being issued
        bool there = false;
        int page_next = 0, slot_next = 0;  // of the tile after it, its page id loaded a tile early
        bool has_next = false;
        auto look_up = [&](int tile) {
            const int64_t p = (int64_t)tile * kTile + lane % kTile;
            has_next = tile < tile1 && p < len;
            if (has_next) {
                const uint32_t pg = (uint32_t)p / (uint32_t)a.cache.page_size;
                slot_next = (int)((uint32_t)p - pg * (uint32_t)a.cache.page_size);
                page_next = pages[pg];
            }
        };
        look_up(tile0);
        // A tree's masks: at most 16 rows, so at most 16 nodes
        tree::Masks nodes;
        if constexpr (TREE) nodes = tree::masks(a.parents + (int64_t)s * a.n_tok, a.n_tok, lane);
        auto issue = [&](int step) {
            if (step < steps) {
                if (!(step & 1)) {
                    there = has_next;
                    if (there && (page_next < 0 || page_next >= a.cache.n_pages)) {
                        record_invalid(a.err);
                        there = false;
                    }
                    off = there ? page_next * a.cache.page_stride + slot_next * a.cache.token_stride + head : 0;
                    look_up(tile0 + (step >> 1) + 1);
                }
                const uint16_t *const from = (step & 1) ? a.cache.v : a.cache.k;
                const uint32_t to = slots + (step % Sh::SLOTS) * Sh::SLOT;
#pragma unroll
                for (int i = 0; i < kTile / RPI; ++i) {
                    const int row = i * RPI + lane / CPR;
                    const int chunk = lane % CPR;
                    const int64_t o = __shfl_sync(0xffffffffu, off, row);
                    const bool ok = __shfl_sync(0xffffffffu, (int)there, row);
                    // no token (past the end, or its page is out of range): zeros
                    cp_async16(to + row * (D * 2) + ((chunk ^ (row & 7)) << 4), from + o + chunk * 8, ok ? 16u : 0u);
                }
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < Sh::SLOTS - 1; ++i) issue(i);
        if (tile0 == 0 && lane == 0) leave_parts(a, sp, L, cut, me, s, h, tr.rb, seg0, tiles);

        // Q: rows lane / 4 and + 8 of this warp's 16, as MMA fragments
        uint32_t qf[KS][4];
        int64_t out_row[2];  // output row, or -1
        int seen[2];         // tokens the row sees; of a tree's node, its mask
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = tr.rb * 16 + r0 + 8 * i;
            out_row[i] = -1;
            seen[i] = 0;
            const uint16_t *src = nullptr;
            if (r < rows) {
                const int j = r / a.group, g = r - j * a.group;
                const int64_t t = (int64_t)s * a.n_tok + j;
                out_row[i] = t * a.h_q + h * a.group + g;
                seen[i] = max(0, len - a.n_tok + j + 1);
                if constexpr (TREE) seen[i] = j;
                src = a.q.p + t * a.q.ts + (int64_t)(h * a.group + g) * a.q.hs;
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qf[k][i] = src ? *reinterpret_cast<const uint32_t *>(src + k * 16 + cq * 2) : 0u;
                qf[k][2 + i] = src ? *reinterpret_cast<const uint32_t *>(src + k * 16 + 8 + cq * 2) : 0u;
            }
        }
        if constexpr (TREE) {
            if (nodes.bad) record_invalid(a.err);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int mask = (int)tree::mask_of(nodes, seen[i]);
                seen[i] = out_row[i] >= 0 ? mask : 0;
            }
        }
        const int base = len - a.n_tok;              // a tree's first slot
        const int all_see = TREE ? base : base + 1;  // tokens every row sees
        // whether row i sees token p of a tile that not all rows see whole (p < len + 16)
        auto sees = [&](int i, int64_t p) {
            if constexpr (TREE)
                return p < base || (seen[i] >> (int)(p - base) & 1);
            else
                return p < seen[i];
        };

        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
        float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};

        for (int tile = tile0; tile < tile1; ++tile) {
            const int step = 2 * (tile - tile0);
            const int64_t p0 = (int64_t)tile * kTile;
            const bool masked = p0 + kTile > all_see;  // some row does not see all of the tile

            // --- keys: x = sc Q K^T
            cp_async_wait<Sh::SLOTS - 2>();
            __syncwarp();
            issue(step + Sh::SLOTS - 1);
            // two column tiles of 8 tokens, each summed in two chains, which hides the MMA's latency
            float x[2][TT][4];
#pragma unroll
            for (int i = 0; i < 2 * TT * 4; ++i) x[i / (TT * 4)][i / 4 % TT][i % 4] = 0.f;
            {
                const uint32_t kb = slots + (step % Sh::SLOTS) * Sh::SLOT;
                const int row = (lane & 7) + ((lane >> 4) << 3);
                // chunk (2 k + b) ^ (row & 7), b = (lane >> 3) & 1: four lane offsets and constants
                uint32_t at[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    at[i] = kb + row * (D * 2) + (((2 * i) ^ ((lane >> 3) & 1) ^ (row & 7)) << 4);
#pragma unroll
                for (int k = 0; k < KS; ++k) {
#pragma unroll
                    for (int t = 0; t < TT; t += 2) {
                        uint32_t b[4];
                        ldsm4(at[k & 3] + t * 8 * D * 2 + (k >> 2) * 128, b);
                        mma16816<F16>(x[k & 1][t], qf[k], b[0], b[1]);
                        mma16816<F16>(x[k & 1][t + 1], qf[k], b[2], b[3]);
                    }
                }
            }
            constexpr int PARTS = F16 ? 1 : 2;
            uint32_t pf[PARTS][TT / 2][4];  // P as MMA operands, bf16 ones in two parts
            float c[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float v[2 * TT];
#pragma unroll
                for (int e = 0; e < 2 * TT; ++e) {
                    v[e] = sc * (x[0][e >> 1][2 * i + (e & 1)] + x[1][e >> 1][2 * i + (e & 1)]);
                    if (masked && !sees(i, p0 + (e >> 1) * 8 + cq * 2 + (e & 1))) v[e] = -CUDART_INF_F;
                }
                float top = v[0];
#pragma unroll
                for (int e = 1; e < 2 * TT; ++e) top = fmaxf(top, v[e]);
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const float mn = next_reference<F16>(m[i], top);
                const float ref = mn == -CUDART_INF_F ? 0.f : mn;  // nothing visible yet: p = 2^-inf
                c[i] = m[i] == mn ? 1.f : tc::fast_exp2(m[i] - ref);
                m[i] = mn;
                l[i] *= c[i];
#pragma unroll
                for (int e = 0; e < TT; ++e) {
                    const float p = tc::fast_exp2(v[2 * e] - ref), q = tc::fast_exp2(v[2 * e + 1] - ref);
                    l[i] += p + q;
                    const int f = (e & 1) * 2 + i;
                    if constexpr (F16)
                        pf[0][e >> 1][f] = pack2<true>(p, q);
                    else
                        split2(p, q, pf[0][e >> 1][f], pf[PARTS - 1][e >> 1][f]);
                }
            }
            if (__any_sync(0xffffffffu, c[0] != 1.f || c[1] != 1.f)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    acc[n][0] *= c[0];
                    acc[n][1] *= c[0];
                    acc[n][2] *= c[1];
                    acc[n][3] *= c[1];
                }
            }

            // --- values: O += P V
            cp_async_wait<Sh::SLOTS - 2>();
            __syncwarp();
            issue(step + Sh::SLOTS);
            const uint32_t vb = slots + ((step + 1) % Sh::SLOTS) * Sh::SLOT;
            if (masked && (TREE || a.n_tok > 1)) {
                // Rows that do not see a draft token have p = 0 for it, and 0 times an
                // infinity or NaN would reach them: such values are added to the rows
                // that see them (p > 0 leaves them as they are) and replaced by zeros.
                bool found = false;
                for (int i = lane; i < kTile * D / 8; i += 32) {
                    uint32_t w[4];
                    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                 : "r"(vb + 16 * i)
                                 : "memory");
                    found = found || any_nonfinite<F16>(w[0], w[1], w[2], w[3]);
                }
                if (__any_sync(0xffffffffu, found)) {
#pragma unroll 1
                    for (int t = 0; t < kTile; ++t) {
                        const int64_t p = p0 + t;
                        if (p >= len) break;
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            uint32_t w;
                            asm volatile("ld.shared.b32 %0, [%1];"
                                         : "=r"(w)
                                         : "r"(vb + t * (D * 2) + ((n ^ (t & 7)) << 4) + cq * 4)
                                         : "memory");
                            if (!nonfinite<F16>(w) && !nonfinite<F16>(w >> 16)) continue;
                            const float2 v = unpack2<F16>(w);
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                if (!sees(i, p)) continue;
                                if (nonfinite<F16>(w)) acc[n][2 * i] += v.x;
                                if (nonfinite<F16>(w >> 16)) acc[n][2 * i + 1] += v.y;
                            }
                        }
                    }
                    __syncwarp();
                    for (int i = lane; i < kTile * D / 2; i += 32) {
                        uint32_t w;
                        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(vb + 4 * i) : "memory");
                        const uint32_t z = cleaned<F16>(w);
                        if (z != w) asm volatile("st.shared.b32 [%0], %1;" ::"r"(vb + 4 * i), "r"(z) : "memory");
                    }
                    __syncwarp();
                }
            }
            {
                const int row = lane & 15;
                uint32_t at[4];  // as for the keys: chunk (n + (lane >> 4)) ^ (row & 7)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    at[i] = vb + row * (D * 2) + (((2 * i) ^ (lane >> 4) ^ (row & 7)) << 4);
#pragma unroll
                for (int t = 0; t < TT / 2; ++t) {
#pragma unroll
                    for (int n = 0; n < NT; n += 2) {
                        uint32_t b[4];
                        ldsm4t(at[(n >> 1) & 3] + t * 16 * D * 2 + (n >> 3) * 128, b);
#pragma unroll
                        for (int i = 0; i < PARTS; ++i) {
                            mma16816<F16>(acc[n], pf[i][t], b[0], b[1]);
                            mma16816<F16>(acc[n + 1], pf[i][t], b[2], b[3]);
                        }
                    }
                }
            }
        }
        cp_async_wait<0>();  // only empty groups are left
        __syncwarp();       // the ring is free for the next triple

#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        }
        if constexpr (TREE) {
            // rows that are no nodes took the tokens before the tree with the others: undone here
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (seen[i] != 0) continue;
                m[i] = -CUDART_INF_F;
                l[i] = 0.f;
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[n][2 * i] = acc[n][2 * i + 1] = 0.f;
            }
        }
        if (tile0 == 0 && tile1 == tiles) {  // the worker saw the whole triple
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (out_row[i] < 0) continue;
                const float inv = seen[i] != 0 ? inverse_sum(l[i]) : 0.f;
                const int64_t t = quotient(out_row[i], a.h_q);
                uint16_t *dst = a.o.p + t * a.o.ts + (out_row[i] - t * a.h_q) * a.o.hs;
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    *reinterpret_cast<uint32_t *>(dst + n * 8 + cq * 2) =
                        pack2<F16>(acc[n][2 * i] * inv, acc[n][2 * i + 1] * inv);
                if (a.lse && cq == 0) a.lse[out_row[i]] = seen[i] != 0 ? kLn2 * (m[i] + log2f(l[i])) : -CUDART_INF_F;
            }
        } else {
            // the part goes to the workspace, or, where the triple goes on in the next worker, to
            // the ring, which this worker has no more use for
            const bool goes_on = tile1 < tiles;
            const int64_t part = ((int64_t)me * 2 + slot_of_part) * L.part_rows;
            float2 *const ml = goes_on ? s_ml + wk * 16 : ml_parts + part;
            float *const po = goes_on ? reinterpret_cast<float *>(ring + wk * Sh::SLOTS * Sh::SLOT) : o_parts + part * D;
            if (goes_on && lane == 0) s_cut[wk] = seg0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (out_row[i] < 0) continue;
                const int r = r0 + 8 * i;
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    *reinterpret_cast<float2 *>(po + r * D + n * 8 + cq * 2) =
                        make_float2(acc[n][2 * i], acc[n][2 * i + 1]);
                if (cq == 0) ml[r] = make_float2(m[i], l[i]);
            }
        }
    }

    // Parts of one triple that end with their workers are joined here, in the order of the
    // tokens, into the first of these workers' part.
    __syncthreads();
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) {
        const int64_t seg0 = s_cut[w];
        if (seg0 < 0 || (w > 0 && s_cut[w - 1] == seg0)) continue;
        int last = w;
        while (last + 1 < kWarps && s_cut[last + 1] == seg0) ++last;
        const int worker = blockIdx.x * cut.per_block + w;
        const int64_t part = ((int64_t)worker * 2 + (cut.start(worker) >= seg0 ? 0 : 1)) * L.part_rows;
        for (int x = tid; x < L.part_rows * (D / 2); x += kThreads) {
            const int r = x / (D / 2), c = x % (D / 2);
            float top = -CUDART_INF_F;
            for (int i = w; i <= last; ++i) top = fmaxf(top, s_ml[i * 16 + r].x);
            const float ref = top == -CUDART_INF_F ? 0.f : top;
            float2 o = make_float2(0.f, 0.f);
            float l = 0.f;
            for (int i = w; i <= last; ++i) {
                const float2 v = s_ml[i * 16 + r];
                const float f = tc::fast_exp2(v.x - ref);
                const float2 y = reinterpret_cast<const float2 *>(ring + i * Sh::SLOTS * Sh::SLOT)[r * (D / 2) + c];
                l += f * v.y;
                o.x += f * y.x;
                o.y += f * y.y;
            }
            reinterpret_cast<float2 *>(o_parts)[(part + r) * (D / 2) + c] = o;
            if (c == 0) ml_parts[part + r] = make_float2(top, l);
        }
    }
}

// What parts of a row add up to, in the order they are added, some at a time.
struct Sum {
    float m, l;
    float4 o;
    __device__ __forceinline__ Sum() : l(0.f), o{0.f, 0.f, 0.f, 0.f} { m = -CUDART_INF_F; }
    // Parts (m, l, x), of which `some` are there.
    template <int U>
    __device__ __forceinline__ void add(const float2 (&ml)[U], const float4 (&x)[U], int some) {
        float top = m;
#pragma unroll
        for (int u = 0; u < U; ++u) top = fmaxf(top, u < some ? ml[u].x : top);
        const float ref = top == -CUDART_INF_F ? 0.f : top;
        const float c0 = m == top ? 1.f : tc::fast_exp2(m - ref);
        m = top;
        l *= c0;
        o = make_float4(o.x * c0, o.y * c0, o.z * c0, o.w * c0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u >= some) break;
            const float c = tc::fast_exp2(ml[u].x - ref);
            l += c * ml[u].y;
            o.x += c * x[u].x;
            o.y += c * x[u].y;
            o.z += c * x[u].z;
            o.w += c * x[u].w;
        }
    }
};
template <bool F16>
__device__ __forceinline__ uint2 pack4(float4 o, float inv) {
    return make_uint2(pack2<F16>(o.x * inv, o.y * inv), pack2<F16>(o.z * inv, o.w * inv));
}

constexpr int kJoinThreads = 256;
template <int D>
constexpr int kJoinRows = 4 * kJoinThreads / D;  // a block's
constexpr int kAtOnce = 4;  // parts added at once

// What the joins' threads would else work out, each for itself.
struct Join {
    const Parts *triples;
    const float2 *ml;
    const float4 *o;
    int part_rows, block_rows, blocks_of_rows;
    uint32_t per_group;  // 2^32 / group, rounded up (rows and groups are below 2^14)
};
struct Joined {  // where a row's result goes
    const Args &a;
    uint32_t per_group;
    int s, h;
    template <bool F16, bool TREE>
    __device__ __forceinline__ void put(int r, int c, const Sum &sum, int64_t len, bool with_lse) const {
        const int j = a.group == 1 ? r : (int)__umulhi((uint32_t)r, per_group), hq = h * a.group + r - j * a.group;
        const int64_t t = (int64_t)s * a.n_tok + j;
        const bool sees = len > 0 && (TREE || len - a.n_tok + j + 1 > 0);  // a tree's rows that are no nodes have l = 0
        reinterpret_cast<uint2 *>(a.o.p + t * a.o.ts + hq * a.o.hs)[c] =
            pack4<F16>(sum.o, sees ? inverse_sum(sum.l) : 0.f);
        if (a.lse && with_lse) a.lse[t * a.h_q + hq] = sees ? kLn2 * (sum.m + log2f(sum.l)) : -CUDART_INF_F;
    }
};

// Joins the parts of every row that more than one worker saw, in the order of the tokens, and
// writes the rows that see nothing.  A block takes the 1024 / D next rows of a triple, a thread four
// columns of a row.  Only parts that are there are loaded (most triples of a batch have two).  Bound by the
// chain of loads, lengths, parts' places, parts, of each wave of blocks.  32 trees of 32 rows, d = 256,
// whole: 84.7 us; two and four rows a thread 83.8 and 84.2, but a long sequence's rows then join one
// after another (30 parts each: 61 us against 29); more blocks an SM, by fewer registers: 87.
template <int D, bool F16, bool TREE>
__global__ void __launch_bounds__(kJoinThreads, 4)
    join_kernel(const __grid_constant__ Args a, const __grid_constant__ Join w) {
    constexpr int TPR = D / 4;
    const uint32_t head = blockIdx.x, triple = head * w.blocks_of_rows + blockIdx.y;
    Joined to{a, w.per_group, (int)(head / (uint32_t)a.h_kv), 0};
    to.h = (int)(head - (uint32_t)to.s * a.h_kv);
    const int r0 = (int)blockIdx.y * w.block_rows, c = threadIdx.x % TPR;
    const int lr = (int)blockIdx.z * kJoinRows<D> + threadIdx.x / TPR;
    const bool live = lr < min(w.part_rows, a.n_tok * a.group - r0);
    const int64_t len = length_of(a, to.s);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!live) return;
    if (len == 0) {
        to.put<F16, TREE>(r0 + lr, c, Sum(), 0, c == 0);
        return;
    }
    const Parts parts = w.triples[triple];
    if (parts.count == 1) return;
    const float2 *const ml = w.ml + lr;
    const float4 *const po = w.o + (int64_t)lr * TPR + c;
    Sum sum;
    if (parts.count == 2) {  // kept short: a batch's rows mostly come here
        const int64_t at0 = parts.row(0, w.part_rows), at1 = (int64_t)parts.w1 * (2 * w.part_rows);
        const float2 v0 = __ldcg(ml + at0), v1 = __ldcg(ml + at1);
        const float4 y0 = __ldcg(po + at0 * TPR), y1 = __ldcg(po + at1 * TPR);
        const float2 v[2] = {v0, v1};
        const float4 y[2] = {y0, y1};
        sum.add<2>(v, y, 2);
        to.put<F16, TREE>(r0 + lr, c, sum, len, c == 0);
        return;
    }
#pragma unroll 1
    for (int i = 0; i < parts.count; i += 2 * kAtOnce) {
        float2 v[2][kAtOnce];
        float4 y[2][kAtOnce];
#pragma unroll
        for (int u = 0; u < 2 * kAtOnce; ++u) {
            if (i + u < parts.count) {
                const int64_t at = parts.row(i + u, w.part_rows);
                v[u / kAtOnce][u % kAtOnce] = __ldcg(ml + at);
                y[u / kAtOnce][u % kAtOnce] = __ldcg(po + at * TPR);
            }
        }
        sum.add<kAtOnce>(v[0], y[0], parts.count - i);
        if (i + kAtOnce < parts.count) sum.add<kAtOnce>(v[1], y[1], parts.count - i - kAtOnce);
    }
    to.put<F16, TREE>(r0 + lr, c, sum, len, c == 0);
}

// The same where rows have many parts (few triples for the blocks): eight warps share the parts of a row.
// (Blocks of 128 columns, twice as many at d = 256, do not all fit the GPU at once: one tree of 24 rows, 16 heads,
// whole: 20.4 us; 18.5 so.)
template <int D, bool F16, bool TREE>
__global__ void __launch_bounds__(kJoinThreads)
    join_many_kernel(const __grid_constant__ Args a, const __grid_constant__ Join j) {
    constexpr int W = kJoinThreads / 32, V = D > 128 ? D / 128 : 1;  // a lane's pieces of four columns
    __shared__ float4 s_o[V][W][32];
    __shared__ float2 s_ml[W];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool mine = lane < D / 4;  // d = 64: half of the lanes
    const uint32_t rows = (uint32_t)a.n_tok * a.group, head = blockIdx.x / rows;
    const int r = (int)(blockIdx.x - head * rows), rb = r / j.block_rows, lr = r - rb * j.block_rows;
    Joined to{a, j.per_group, (int)(head / (uint32_t)a.h_kv), 0};
    to.h = (int)(head - (uint32_t)to.s * a.h_kv);
    const int64_t len = length_of(a, to.s);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (len == 0) {
        if (w < V && mine) to.put<F16, TREE>(r, 32 * w + lane, Sum(), 0, w == 0 && lane == 0);
        return;
    }
    const Parts parts = j.triples[(int64_t)head * j.blocks_of_rows + rb];
    if (parts.count == 1) return;
    Sum sum[V];
#pragma unroll 1
    for (int i = w; i < parts.count; i += W * kAtOnce) {
        float2 v[kAtOnce];
        float4 y[V][kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            if (u > 0 && i + u * W >= parts.count) break;
            const int64_t at = parts.row(i + u * W, j.part_rows) + lr;
            v[u] = __ldcg(j.ml + at);
#pragma unroll
            for (int e = 0; e < V; ++e) y[e][u] = __ldcg(j.o + at * (D / 4) + 32 * e + (mine ? lane : 0));
        }
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e].add<kAtOnce>(v, y[e], (parts.count - i + W - 1) / W);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) s_o[e][w][lane] = sum[e].o;
    if (lane == 0) s_ml[w] = make_float2(sum[0].m, sum[0].l);
    __syncthreads();  // the block is one row: its warps come here together
    if (w >= V) return;
    float2 v[W];
    float4 y[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        v[i] = s_ml[i];
        y[i] = s_o[w][i][lane];
    }
    Sum all;
    all.add<W>(v, y, W);
    if (mine) to.put<F16, TREE>(r, 32 * w + lane, all, len, w == 0 && lane == 0);
}

template <int D, bool F16, bool TREE>
cudaError_t launch_warps(const Args &a, cudaStream_t s) {
    static SmemOptIn opt_in;
    const cudaError_t e = opt_in.set(reinterpret_cast<const void *>(decode_kernel<D, F16, TREE>), (int)Shape<D>::SMEM);
    if (e != cudaSuccess) return e;
    decode_kernel<D, F16, TREE><<<kBlocks, kThreads, Shape<D>::SMEM, s>>>(a);
    return cudaGetLastError();
}

template <int D, bool F16, bool TREE>
cudaError_t launch_as(const Args &a, cudaStream_t s) {
    const int rows = a.n_tok * a.group;
    const int64_t heads = (int64_t)a.n_seqs * a.h_kv;
    const Kind kind = kind_of(rows, D, TREE, heads);
    const cudaError_t e = kind != kFew ? launch_decode_wide(a, s) : launch_warps<D, F16, TREE>(a, s);
    if (e != cudaSuccess) return e;
    const Spec sp = spec(kind, D);
    const Layout L = layout(rows, sp, D, heads);
    const int64_t triples = heads * L.blocks_of_rows;
    const bool many = kBlocks >= 16 * triples;
    char *const ws = static_cast<char *>(a.ws);
    const Join w = {reinterpret_cast<const Parts *>(ws), reinterpret_cast<const float2 *>(ws + L.ml),
                    reinterpret_cast<const float4 *>(ws + L.o), L.part_rows, sp.block_rows, L.blocks_of_rows,
                    (uint32_t)((0x100000000ull + a.group - 1) / a.group)};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = many ? dim3((unsigned)(a.t_total * a.h_q)) : dim3((unsigned)(a.n_seqs * a.h_kv), L.blocks_of_rows, (L.part_rows + kJoinRows<D> - 1) / kJoinRows<D>);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return many ? cudaLaunchKernelEx(&cfg, join_many_kernel<D, F16, TREE>, a, w)
                : cudaLaunchKernelEx(&cfg, join_kernel<D, F16, TREE>, a, w);
}

template <int D, bool F16>
cudaError_t launch(const Args &a, cudaStream_t s) {
    return a.parents ? launch_as<D, F16, true>(a, s) : launch_as<D, F16, false>(a, s);
}

}  // namespace

size_t decode_workspace_bytes(int h_q, int h_kv, int d, int n_seqs, int n_tok, bool tree) {
    const int rows = n_tok * (h_q / h_kv);
    const int64_t heads = (int64_t)n_seqs * h_kv;
    return layout(rows, spec(kind_of(rows, d, tree, heads), d), d, heads).total;
}

cudaError_t launch_decode(const Args &a, cudaStream_t s) {
    if (a.d == 64) return a.f16 ? launch<64, true>(a, s) : launch<64, false>(a, s);
    if (a.d == 128) return a.f16 ? launch<128, true>(a, s) : launch<128, false>(a, s);
    return a.f16 ? launch<256, true>(a, s) : launch<256, false>(a, s);
}

}  // namespace attn
}  // namespace gdr
