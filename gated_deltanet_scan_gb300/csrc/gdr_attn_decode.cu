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

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1) decode_kernel(const __grid_constant__ Args a) {
    using Sh = Shape<D>;
    constexpr Spec sp = spec(false, D);
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
    const Layout L = layout(rows, sp, D, a.n_seqs);
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

        // Q: rows lane / 4 and + 8 of this warp's 16, as MMA fragments
        uint32_t qf[KS][4];
        int64_t out_row[2];  // output row, or -1
        int seen[2];         // tokens the row sees
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
                src = a.q.p + t * a.q.ts + (int64_t)(h * a.group + g) * a.q.hs;
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qf[k][i] = src ? *reinterpret_cast<const uint32_t *>(src + k * 16 + cq * 2) : 0u;
                qf[k][2 + i] = src ? *reinterpret_cast<const uint32_t *>(src + k * 16 + 8 + cq * 2) : 0u;
            }
        }
        const int all_see = len - a.n_tok + 1;  // tokens every row sees

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
                    if (masked && p0 + (e >> 1) * 8 + cq * 2 + (e & 1) >= seen[i]) v[e] = -CUDART_INF_F;
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
            if (masked && a.n_tok > 1) {
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
                                if (p >= seen[i]) continue;
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
        if (tile0 == 0 && tile1 == tiles) {  // the worker saw the whole triple
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (out_row[i] < 0) continue;
                const float inv = seen[i] > 0 ? inverse_sum(l[i]) : 0.f;
                const int64_t t = quotient(out_row[i], a.h_q);
                uint16_t *dst = a.o.p + t * a.o.ts + (out_row[i] - t * a.h_q) * a.o.hs;
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    *reinterpret_cast<uint32_t *>(dst + n * 8 + cq * 2) =
                        pack2<F16>(acc[n][2 * i] * inv, acc[n][2 * i + 1] * inv);
                if (a.lse && cq == 0) a.lse[out_row[i]] = seen[i] > 0 ? kLn2 * (m[i] + log2f(l[i])) : -CUDART_INF_F;
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

// Joins the parts of every row that more than one worker saw, in the order of the
// tokens, and writes the rows that see nothing.  With WPR > 1 a block is WPR warps on 64
// columns of one row, which share the row's parts; else a warp is one row.
template <int D, bool F16, int WPR>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Args a, const bool wide) {
    constexpr int V = WPR > 1 ? 2 : D / 32;  // columns per lane
    constexpr int RPB = 8 / WPR;             // rows per block
    __shared__ float2 s_acc[WPR > 1 ? WPR : 1][32];
    __shared__ float2 s_ml[WPR];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = warp % WPR;
    const uint32_t row = blockIdx.x * RPB + warp / WPR;
    const int word0 = WPR > 1 ? blockIdx.y * 32 + lane : lane;  // this lane's first pair of columns
    if (row >= a.t_total * a.h_q) return;
    const uint32_t t = row / (uint32_t)a.h_q;
    const int hq = (int)(row - t * a.h_q);
    const int s = (int)(t / (uint32_t)a.n_tok), j = (int)(t - (uint32_t)s * a.n_tok);
    const int h = hq / a.group, g = hq - h * a.group;
    const Spec sp = spec(wide, D);
    const Layout L = layout(a.n_tok * a.group, sp, D, a.n_seqs);
    const int r = j * a.group + g, rb = r / sp.block_rows, lr = r - rb * sp.block_rows;
    uint32_t *const dst = reinterpret_cast<uint32_t *>(a.o.p + t * a.o.ts + hq * a.o.hs);
    const bool write_lse = a.lse && lane == 0 && blockIdx.y == 0;
    const int64_t len = length_of(a, s);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (len == 0) {
        if (w == 0) {
#pragma unroll
            for (int e = 0; e < V / 2; ++e) dst[word0 + 32 * e] = 0u;
            if (write_lse) a.lse[row] = -CUDART_INF_F;
        }
        return;
    }
    const int64_t tiles = (len + sp.tile - 1) / sp.tile;
    const int64_t *const line = reinterpret_cast<const int64_t *>(a.ws);
    const int64_t seg0 = line[s] + ((int64_t)h * L.blocks_of_rows + rb) * (tiles + sp.lead);
    const Cut cut(line[a.n_seqs], sp.workers);
    const int w0 = cut.part_of(seg0 + sp.lead), w1 = cut.part_of(seg0 + sp.lead + tiles - 1);
    if (w0 == w1) return;

    const float2 *const ml = reinterpret_cast<const float2 *>(static_cast<const uint8_t *>(a.ws) + L.ml);
    const float2 *const po = reinterpret_cast<const float2 *>(static_cast<const uint8_t *>(a.ws) + L.o);
    // a worker's part is its first where its own start is not before the triple's: so
    // all parts but perhaps the first one's
    // all but the last worker's part are joined within their blocks: the parts are those of the
    // first such worker of every block, and the last worker's
    const int per_block = cut.per_block, b0 = w0 / per_block;
    const int n_parts = (w1 - 1) / per_block - b0 + 2;
    const int64_t row0 = cut.start(w0) >= seg0 ? 0 : L.part_rows;
    auto part_row = [&](int i) {
        const int wk = i == 0 ? w0 : i == n_parts - 1 ? w1 : (b0 + i) * per_block;
        return (int64_t)wk * 2 * L.part_rows + (i == 0 ? row0 : 0) + lr;
    };
    float2 acc[V / 2];
    float m = -CUDART_INF_F, l = 0.f;
#pragma unroll
    for (int e = 0; e < V / 2; ++e) acc[e] = make_float2(0.f, 0.f);
    constexpr int U = 4;  // parts in flight
#pragma unroll 1
    for (int i = w; i < n_parts; i += WPR * U) {
        float2 x[U][V / 2], v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t pr = part_row(min(i + u * WPR, n_parts - 1));
            v[u] = __ldcg(ml + pr);
#pragma unroll
            for (int e = 0; e < V / 2; ++e) x[u][e] = __ldcg(po + pr * (D / 2) + word0 + 32 * e);
        }
        float top = m;
#pragma unroll
        for (int u = 0; u < U; ++u) top = fmaxf(top, i + u * WPR < n_parts ? v[u].x : top);
        const float ref = top == -CUDART_INF_F ? 0.f : top;
        const float c0 = m == top ? 1.f : tc::fast_exp2(m - ref);
        m = top;
        l *= c0;
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
            acc[e].x *= c0;
            acc[e].y *= c0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i + u * WPR >= n_parts) break;
            const float c = tc::fast_exp2(v[u].x - ref);
            l += c * v[u].y;
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
                acc[e].x += c * x[u][e].x;
                acc[e].y += c * x[u][e].y;
            }
        }
    }
    if constexpr (WPR > 1) {
        s_acc[w][lane] = acc[0];
        if (lane == 0) s_ml[w] = make_float2(m, l);
        __syncthreads();  // the block is one row: its warps come here together
        if (w != 0) return;
#pragma unroll
        for (int i = 1; i < WPR; ++i) m = fmaxf(m, s_ml[i].x);
        const float ref = m == -CUDART_INF_F ? 0.f : m;
        l = 0.f;
        acc[0] = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < WPR; ++i) {
            const float c = tc::fast_exp2(s_ml[i].x - ref);
            l += c * s_ml[i].y;
            acc[0].x += c * s_acc[i][lane].x;
            acc[0].y += c * s_acc[i][lane].y;
        }
    }
    const bool sees = len - a.n_tok + j + 1 > 0;
    const float inv = sees ? inverse_sum(l) : 0.f;
#pragma unroll
    for (int e = 0; e < V / 2; ++e) dst[word0 + 32 * e] = pack2<F16>(acc[e].x * inv, acc[e].y * inv);
    if (write_lse) a.lse[row] = sees ? kLn2 * (m + log2f(l)) : -CUDART_INF_F;
}

template <int D, bool F16>
cudaError_t launch_warps(const Args &a, cudaStream_t s) {
    static SmemOptIn opt_in;
    const cudaError_t e = opt_in.set(reinterpret_cast<const void *>(decode_kernel<D, F16>), (int)Shape<D>::SMEM);
    if (e != cudaSuccess) return e;
    decode_kernel<D, F16><<<kBlocks, kThreads, Shape<D>::SMEM, s>>>(a);
    return cudaGetLastError();
}

template <int D, bool F16>
cudaError_t launch(const Args &a, cudaStream_t s) {
    const bool wide = is_wide(a.n_tok * a.group);
    const cudaError_t e = wide ? launch_decode_wide(a, s) : launch_warps<D, F16>(a, s);
    if (e != cudaSuccess) return e;
    // The join: 8 warps on every 64 columns of a row where a row has many parts (few
    // triples for the blocks), else a warp per row.
    const int64_t rows = a.t_total * a.h_q;
    const Layout L = layout(a.n_tok * a.group, spec(wide, D), D, a.n_seqs);
    const bool many = kBlocks >= (int64_t)16 * a.n_seqs * a.h_kv * L.blocks_of_rows;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = many ? dim3((unsigned)rows, D / 64) : dim3((unsigned)((rows + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return many ? cudaLaunchKernelEx(&cfg, join_kernel<D, F16, 8>, a, wide)
                : cudaLaunchKernelEx(&cfg, join_kernel<D, F16, 1>, a, wide);
}

}  // namespace

size_t decode_workspace_bytes(int h_q, int h_kv, int d, int n_seqs, int n_tok) {
    const int rows = n_tok * (h_q / h_kv);
    return layout(rows, spec(is_wide(rows), d), d, n_seqs).total;
}

cudaError_t launch_decode(const Args &a, cudaStream_t s) {
    if (a.d == 64) return a.f16 ? launch<64, true>(a, s) : launch<64, false>(a, s);
    if (a.d == 128) return a.f16 ? launch<128, true>(a, s) : launch<128, false>(a, s);
    return a.f16 ? launch<256, true>(a, s) : launch<256, false>(a, s);
}

}  // namespace attn
}  // namespace gdr
