// Attention of the last few tokens over the paged cache, for more than 16 rows of a
// key/value head (draft blocks, large groups), on tcgen05 tensor cores.
//
// Formulas, line, parts and join are those of gdr_attn_decode.cu.  With 17 rows or more
// the warp-level products of that kernel would bound it (64 rows of d = 256: 55 us against
// 19 of HBM; 255 registers a thread leave two warps a scheduler).  Here one worker per SM
// takes blocks of 128 rows: Q is an operand tile in shared memory, O and two S tiles of 64
// tokens are in TMEM, and P overwrites its S as 16-bit pairs, the second product's operand.
// A tile of 64 tokens takes the tensor pipe 1,024 clocks at d = 256 whatever the rows are,
// against 2,800 that its bytes take at a 152nd of the bandwidth.
//
//   loads    four warps gather K and V rows through the page table, 16-byte asynchronous
//            copies into the swizzled operand layout, as many stages in flight as the ring
//            has; the copies themselves report a stage full when they land, and the MMA warp
//            orders them before its reads (reported by the copying threads two stages from
//            the ring's end instead, 60% of the stages sat landed and unreported: 47 us).
//   Q        three warps, a triple ahead of need where a place for Q is free.
//   MMAs     one warp: S of the next tile before P V of this one.
//   P, O     a warpgroup per block of rows, a row per thread: P of every tile, and O at a triple's end.
// All roles run over the triples' ends, so the loads never stop.
//
// Trees of more than 128 rows (64 nodes, 4 query heads of a key/value head) would read their keys and
// values, and pay for their loads, once per block of rows.  Up to d = 128 TMEM holds O and two S tiles of
// two blocks, so a worker takes both (B = 2, where there are enough of them: kind_of), the products block by block, so that one's P is made
// while the other's run: 16 trees of 64 nodes, contexts up to 16,384, d = 128, 32 / 8 heads: 124 us with a
// block a worker, 113 with two, 107 with two places for Q, 98 with today's join.  While tiles run, the tensor
// pipe and the shared memory it reads (Q again for every 64 tokens) bound it: 1,770 clocks a tile, of which HBM
// would need 1,370.  But a worker's 47 tiles are 42 of the kernel's 87 us, and its tensor pipe works 28% of them:
// the others are its start, one or two changes of triple (256 rows of Q in, O out) and parts of up to 256 rows
// (40 MB written and read again), how much of each is not measured.
//
// P is rounded to its type, fp16's 11 bits or bf16's 8: o is up to 2.8 * 10^-4 or 2.3 * 10^-3 of its norm off 64
// bits, of which its own rounding makes 2.1 * 10^-4 and 1.7 * 10^-3.  A chain as a tree has the bits of gdr_attn_decode where
// both take this kernel on the same cuts.  A second product with what bf16's rounding left, as in
// gdr_attn_decode.cu, would halve o's squared error and take 10% longer (16 draft tokens of 32
// sequences of 2,000, d = 128: 77.6 against 69.5 us; 8 of 512 to 8,192, d = 256: 39.4 / 38.6).
//
// Draft tokens' values that some row does not see are cleaned of infinities and NaNs by
// the threads that copied them, and added at the end to the rows that see them.
#include "gdr_attn_line.cuh"
#include "gdr_attn_mma.cuh"
#include "gdr_attn_ptx.cuh"
#include "gdr_internal.h"
#include "gdr_tree.cuh"
#include "tc_ptx.cuh"

namespace gdr {
namespace attn {
namespace {

using namespace tc;

constexpr int kRows = 128, kTile = 64;
constexpr uint32_t kColsS = 256;  // TMEM: O at 0 (and 128), S tiles at 256 and 320 (and 384 and 448)

// B: blocks of rows that a worker takes at once.
template <int D, int B>
struct Shape {
    static_assert(B == 1 || (B == 2 && D <= 128), "O's columns");
    static constexpr int THREADS = B * 128 + 256;
    static constexpr uint32_t Q_BLOCK = kRows * 128;  // 64 columns
    static constexpr uint32_t Q_BYTES = Q_BLOCK * (D / 64);
    static constexpr uint32_t BOX = kTile * 128;      // 64 tokens, 64 columns
    static constexpr uint32_t STAGE = BOX * (D / 64);
    static constexpr int STAGES = D == 256 ? 5 : D == 128 && B == 2 ? 6 : 8;
    static constexpr int QS = D == 256 ? 1 : 2;  // places for Q, where shared memory has them
    // Rows of a tile that one of the four loading warps copies: 32, two warps for K and two for
    // V, or 16 of either, so that a stage's copies are all on their way sooner.  32 pays waits,
    // arrivals and page ids of a stage half as often, 16 suits few stages: 32 against 16, d = 64
    // 32.3 / 38.1 us, d = 128 63.8 / 70.7, d = 256 42.2 / 38.7.
    static constexpr int LOAD_ROWS = D == 256 ? 16 : 32;
    static constexpr uint32_t OFF_RING = QS * B * Q_BYTES;
    static constexpr uint32_t OFF_BAR = OFF_RING + STAGES * STAGE;
    static constexpr uint32_t OFF_WORDS = OFF_BAR + 8 * 34;  // TMEM address, flag
    static constexpr uint32_t BYTES = OFF_WORDS + 16;
    // at least 116 KiB, so that one block has the SM (and its TMEM) to itself
    static constexpr uint32_t SMEM = BYTES < 116 * 1024 ? 116 * 1024 : BYTES;
};
enum Bar {
    kQFull = 0,                // [places]
    kQEmpty = 2,               // [places]
    kKvFull = 4,               // [stages]
    kKvEmpty = kKvFull + 8,    // [stages]
    kSFull = kKvEmpty + 8,     // [B][2]
    kPFull = kSFull + 4,       // [B][2]
    kPvDone = kPFull + 4,      // [B][2]
    kODone = kPvDone + 4,
    kOFree = kODone + 1,
    kBars = kOFree + 1,
};
static_assert(kBars <= 34, "barrier words");

template <int D, bool F16, bool TREE, int B>
__global__ void __launch_bounds__((Shape<D, B>::THREADS), 1) wide_kernel(const __grid_constant__ Args a) {
    using Sh = Shape<D, B>;
    constexpr int kThreads = Sh::THREADS, kLoads = 4 * B, kMmas = kLoads + 4;  // the roles' first warps
    constexpr Spec sp = spec(B == 2 ? kPaired : kWide, D);
    static_assert(sp.tile == kTile && sp.block_rows == B * kRows, "the line's units");
    constexpr int N = Sh::STAGES, CPR = D / 8;
    extern __shared__ __align__(1024) uint8_t smem[];
    // the line's scan comes before the ring's first use
    Line<kThreads, 1> &s_line = *reinterpret_cast<Line<kThreads, 1> *>(smem + Sh::OFF_RING);
    static_assert(sizeof(Line<kThreads, 1>) <= N * Sh::STAGE, "the scan fits the ring");
    uint32_t *const s_tmem = reinterpret_cast<uint32_t *>(smem + Sh::OFF_WORDS);
    volatile uint32_t *const s_found = s_tmem + 1;  // a cleaned value, in any triple so far
    const uint32_t base = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    auto bar = [&](int i) { return base + Sh::OFF_BAR + 8u * i; };

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 0) {
        for (int i = 0; i < Sh::QS; ++i) {
            mbar_init(bar(kQFull + i), 96);
            mbar_init(bar(kQEmpty + i), 1);
        }
        for (int i = 0; i < N; ++i) {
            mbar_init(bar(kKvFull + i), Sh::LOAD_ROWS == 32 ? 64 : 128);
            mbar_init(bar(kKvEmpty + i), 1);
        }
        for (int i = 0; i < 2 * B; ++i) {
            mbar_init(bar(kSFull + i), 1);
            mbar_init(bar(kPFull + i), 4);
            mbar_init(bar(kPvDone + i), 1);
        }
        mbar_init(bar(kODone), 1);
        mbar_init(bar(kOFree), 4 * B);
        *s_found = 0;
        fence_mbar_init();
    }
    if (warp == kMmas) {
        tmem_alloc(smem_u32(s_tmem), 512);
        tmem_relinquish();
    }
    const int rows = a.n_tok * a.group;
    const Layout L = layout(rows, sp, D, (int64_t)a.n_seqs * a.h_kv);
    const Cut cut(s_line.place(a, sp, L.blocks_of_rows), 1);
    int me;
    Walk walk = s_line.walk(cut, 0, me);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *s_tmem;

    bool ok = true;
    auto wait = [&](int i, uint32_t parity) {
        ok = __all_sync(0xffffffffu, ok && pair::wait_bounded(bar(i), parity & 1)) != 0;
        return ok;
    };
    // Roles count tiles and triples through all of the worker's triples.  Stages of the ring are
    // taken in the order K0, K1, V0, K2, V1, ...; the last value tile leaves one out.
    auto key_stage = [](uint32_t g) { return g == 0 ? 0 : 2 * g - 1; };
    auto value_stage = [](uint32_t g) { return 2 * g + 2; };
    Triple t;

    if (warp < kLoads) {
        // ---- P and O; a thread is a row
        const int row = tid, blk = warp >> 2;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16) + blk * 128;
        const uint32_t s_lanes = lanes + kColsS;  // block 1's S tiles are 128 columns behind block 0's, too
        const float sc = softmax_scale(a.scale);
        float2 *const ml_parts = reinterpret_cast<float2 *>(static_cast<uint8_t *>(a.ws) + L.ml);
        float *const o_parts = reinterpret_cast<float *>(static_cast<uint8_t *>(a.ws) + L.o);
        uint32_t g = 0;  // tiles
        tree::Masks nodes;
        int nodes_of = -1;  // the sequence whose tree they are
        for (int it = 0; ok && walk.next(a, sp, L.blocks_of_rows, t); ++it) {
            const int r = t.rb * sp.block_rows + row;
            const bool live = r < rows;
            const int j = r / a.group, hq = t.h * a.group + r - j * a.group;
            const int tree0 = t.len - a.n_tok;  // a tree's first slot
            const int seen = live ? max(0, tree0 + j + 1) : 0;
            const int all_see = TREE ? tree0 : tree0 + 1;
            uint64_t mask = 0;
            if constexpr (TREE) {
                if (t.s != nodes_of) {
                    nodes_of = t.s;
                    nodes = tree::masks(a.parents + (int64_t)t.s * a.n_tok, a.n_tok, lane);
                    if (nodes.bad) record_invalid(a.err);
                }
                mask = tree::mask_of(nodes, j & 63);
                if (!live) mask = 0;
            }
            const bool any = TREE ? mask != 0 : seen > 0;  // the row sees something
            const bool work = t.rb * sp.block_rows + warp * 32 < rows;  // some row of the warp is live
            float m = -CUDART_INF_F, l = 0.f;
            for (int tile = t.tile0; tile < t.tile1; ++tile, ++g) {
                const int st = g & 1;
                if (!wait(kSFull + 2 * blk + st, g >> 1)) break;
                if (work) {
                    tc_fence_after_sync();
                    const uint32_t s_at = s_lanes + st * kTile;
                    uint32_t x[64];
                    pair::tmem_load32_start(s_at, x);
                    pair::tmem_load32_start(s_at + 32, x + 32);
                    pair::tmem_load_wait(x);
                    const int p0 = tile * kTile;
                    if (p0 + kTile > all_see) {
#pragma unroll
                        for (int c0 = 0; c0 < 64; c0 += 32) {
                            uint32_t sees;
                            if constexpr (TREE) {
                                sees = tree::sees32(mask, p0 + c0 - tree0);
                            } else {
                                const int n = seen - p0 - c0;  // columns seen
                                sees = n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u;
                            }
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!(sees & (1u << c))) x[c0 + c] = 0xFF800000u;
                        }
                    }
                    float top[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                    for (int c = 0; c < 64; c += 8) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            top[e] = pair::max3(top[e], __uint_as_float(x[c + e]), __uint_as_float(x[c + 4 + e]));
                    }
                    const float x_top = sc * fmaxf(pair::max3(top[0], top[1], top[2]), top[3]);
                    const float m_old = m;
                    m = next_reference<F16>(m, x_top);
                    const float ref = m == -CUDART_INF_F ? 0.f : m;  // nothing visible yet: p = 2^-inf
                    const float f = m_old == m ? 1.f : fast_exp2(m_old - ref);
                    if (tile > t.tile0 && __any_sync(0xffffffffu, f != 1.f)) {
                        if (!wait(kPvDone + 2 * blk + ((g - 1) & 1), (g - 1) >> 1)) break;
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            uint32_t o[32];
                            pair::tmem_load32(lanes + c, o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            pair::tmem_store16(lanes + c, o);
                            pair::tmem_store16(lanes + c + 16, o + 16);
                        }
                    }
                    l *= f;
                    uint32_t p[32];
                    float sum[2] = {0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const float u = fast_exp2(fmaf(__uint_as_float(x[2 * c]), sc, -ref));
                        const float v = fast_exp2(fmaf(__uint_as_float(x[2 * c + 1]), sc, -ref));
                        sum[0] += u;
                        sum[1] += v;
                        p[c] = pack2<F16>(u, v);
                    }
                    pair::tmem_store16(s_at, p);
                    pair::tmem_store16(s_at + 16, p + 16);
                    l += sum[0] + sum[1];
                    pair::tmem_store_wait();
                    tc_fence_before_sync();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kPFull + 2 * blk + st));
            }
            if (!ok || !wait(kODone, it)) break;
            tc_fence_after_sync();
            if constexpr (TREE) {
                // a row that is no node took the tokens before the tree with the others: undone here
                if (!any) {
                    m = -CUDART_INF_F;
                    l = 0.f;
                }
            }
            // O, whole or as a part
            const bool whole = t.tile0 == 0 && t.tile1 == t.tiles;
            const bool patch = *s_found != 0;
            const int64_t tok = (int64_t)t.s * a.n_tok + j;
            const int64_t part = ((int64_t)me * 2 + (cut.start(me) >= t.seg0 ? 0 : 1)) * L.part_rows + row;
            const float inv = inverse_sum(l);
            if (work) {
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    pair::tmem_load32(lanes + c, o);
                    if (c + 32 == D) {
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(kOFree));
                    }
                    if (live && whole) {
                        uint16_t *const dst = a.o.p + tok * a.o.ts + (int64_t)hq * a.o.hs + c;
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint4 w;
                            // a row that sees nothing is zero, whatever its O holds
                            w.x = any ? pack2<F16>(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv) : 0u;
                            w.y = any ? pack2<F16>(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv) : 0u;
                            w.z = any ? pack2<F16>(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv) : 0u;
                            w.w = any ? pack2<F16>(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv) : 0u;
                            *reinterpret_cast<uint4 *>(dst + e) = w;
                        }
                    } else if (!whole) {
                        if constexpr (TREE) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = any ? o[e] : 0u;
                        }
                        // four lanes store 64 bytes of a row together: pieces of 16 bytes are
                        // transposed among them, in two halves of 16 columns
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
#pragma unroll
                            for (int p = 0; p < 8; p += 2) {
                                uint32_t &y = o[p * 4 + e], &z = o[p * 4 + 4 + e];
                                const uint32_t v = __shfl_xor_sync(0xffffffffu, (lane & 1) ? y : z, 1);
                                ((lane & 1) ? y : z) = v;
                            }
#pragma unroll
                            for (int p = 0; p < 8; p += 4) {
#pragma unroll
                                for (int q = p; q < p + 2; ++q) {
                                    uint32_t &y = o[q * 4 + e], &z = o[q * 4 + 8 + e];
                                    const uint32_t v = __shfl_xor_sync(0xffffffffu, (lane & 2) ? y : z, 2);
                                    ((lane & 2) ? y : z) = v;
                                }
                            }
                        }
#pragma unroll
                        for (int p = 0; p < 8; ++p) {
                            const int back = (lane & 3) - (p & 3);  // this lane's row is `back` below the piece's
                            if (r - back < rows)
                                *reinterpret_cast<uint4 *>(o_parts + (part - back) * D + c + (p >> 2) * 16 +
                                                           (lane & 3) * 4) =
                                    make_uint4(o[p * 4], o[p * 4 + 1], o[p * 4 + 2], o[p * 4 + 3]);
                        }
                    }
                    __syncwarp();
                }
                if (live && patch) {
                    // tiles that were cleaned, from the one in which the rows begin to differ: what they
                    // add to the stored row or part (a rare path, kept small)
                    const int from = max(t.tile0, max(0, all_see) / kTile) * kTile;
                    const int to = TREE ? (any ? min(t.len, t.tile1 * kTile) : 0) : min(seen, t.tile1 * kTile);
                    uint16_t *const dst = a.o.p + tok * a.o.ts + (int64_t)hq * a.o.hs;
#pragma unroll 1
                    for (int p = from; p < to; ++p) {
                        if (TREE && !(tree::sees32(mask, p - tree0) & 1u)) continue;
                        const uint32_t pg = (uint32_t)p / (uint32_t)a.cache.page_size;
                        const int page = a.cache.table[(int64_t)t.s * a.cache.table_stride + pg];
                        if (page < 0 || page >= a.cache.n_pages) continue;
                        const uint16_t *const v = a.cache.v + page * a.cache.page_stride +
                                                  (int64_t)(p - (int)pg * a.cache.page_size) * a.cache.token_stride +
                                                  t.h * a.cache.head_stride;
#pragma unroll 1
                        for (int c = 0; c < D; ++c) {
                            const float y = unpack1<F16>(v[c]);
                            if (isfinite(y)) continue;
                            if (whole)
                                dst[c] = (uint16_t)pack2<F16>(unpack1<F16>(dst[c]) + y, 0.f);
                            else
                                o_parts[part * D + c] += y;
                        }
                    }
                }
                if (live && whole && a.lse)
                    a.lse[tok * a.h_q + hq] = kLn2 * (m + log2f(l));
                if (live && !whole) ml_parts[part] = make_float2(m, l);
            } else if (lane == 0) {
                mbar_arrive(bar(kOFree));
            }
            __syncwarp();
        }
    } else if (warp < kMmas) {
        // ---- K and V: a warp's lanes hold the offsets of its rows of a tile
        constexpr int R = Sh::LOAD_ROWS;
        const int w = (warp - kLoads) & (64 / R - 1);
        auto clean = [&](uint32_t st) {  // the values this thread copied, landed
            auto piece = [&](int x) {
                const int row = w * R + x % (R / 4) * 4 + (lane >> 3);
                return reinterpret_cast<uint4 *>(smem + Sh::OFF_RING + st * Sh::STAGE + x / (R / 4) * Sh::BOX + row * 128 +
                                                 (((lane & 7) ^ (row & 7)) << 4));
            };
            bool found = false;
#pragma unroll 8
            for (int x = 0; x < R / 4 * (D / 64); ++x) {
                const uint4 v = *piece(x);
                found = found || any_nonfinite<F16>(v.x, v.y, v.z, v.w);
            }
            if (!found) return;
#pragma unroll 1
            for (int x = 0; x < R / 4 * (D / 64); ++x) {
                const uint4 v = *piece(x);
                *piece(x) = make_uint4(cleaned<F16>(v.x), cleaned<F16>(v.y), cleaned<F16>(v.z), cleaned<F16>(v.w));
            }
            *s_found = 1;
        };
        // A lane's row of a tile: its page id is loaded a tile early and looked at when the tile's
        // turn comes; then its offset in the cache, or -1.
        struct Ahead {
            int page, slot;  // slot -1: no token
        };
        auto look_up = [&](const Triple &u, int tile) {
            Ahead x{0, -1};
            const int p = tile * kTile + w * R + (lane & (R - 1));
            if (p < u.len) {
                const uint32_t pg = (uint32_t)p / (uint32_t)a.cache.page_size;
                x.slot = p - (int)pg * a.cache.page_size;
                x.page = a.cache.table[(int64_t)u.s * a.cache.table_stride + pg];
            }
            return x;
        };
        struct Tiles {  // of K or of V, through all triples
            Walk walk;
            Triple t;
            int tile;
            Ahead next;
            uint32_t g;
        };
        auto begin = [&] {
            Tiles x;
            x.walk = walk;
            x.t.tile1 = x.tile = 0;
            x.next = Ahead{0, -1};
            x.g = 0;
            return x;
        };
        auto load = [&](Tiles &x, bool values) {  // the next tile, if there is one
            if (x.tile == x.t.tile1) {
                if (!x.walk.next(a, sp, L.blocks_of_rows, x.t)) return false;
                x.tile = x.t.tile0;
                x.next = look_up(x.t, x.tile);
            }
            int64_t lane_off = -1;
            if (x.next.slot >= 0) {
                if (x.next.page < 0 || x.next.page >= a.cache.n_pages)
                    record_invalid(a.err);
                else
                    lane_off = x.next.page * a.cache.page_stride + x.next.slot * a.cache.token_stride +
                               x.t.h * a.cache.head_stride;
            }
            if (++x.tile < x.t.tile1) x.next = look_up(x.t, x.tile);
            const uint32_t i = values ? value_stage(x.g) : key_stage(x.g), st = i % N, use = i / N;
            ++x.g;
            if (use > 0 && !wait(kKvEmpty + st, use - 1)) return false;
            const uint16_t *const from = values ? a.cache.v : a.cache.k;
            const uint32_t to = base + Sh::OFF_RING + st * Sh::STAGE;
            // eight lanes copy 128 bytes of a row, then the row's next 128: an offset is passed
            // on once for all of them
#pragma unroll
            for (int y = 0; y < R / 4; ++y) {
                const int lr = y * 4 + (lane >> 3), row = w * R + lr;
                const int64_t off = __shfl_sync(0xffffffffu, lane_off, lr);
                const uint32_t at = to + row * 128 + (((lane & 7) ^ (row & 7)) << 4);
                const uint16_t *const src = from + (off < 0 ? 0 : off) + (lane & 7) * 8;
                // no token (past the end, or its page is out of range): zeros
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    cp_async16(at + c * Sh::BOX, src + c * 64, off < 0 ? 0u : 16u);
            }
            if (values && (TREE || a.n_tok > 1) && x.tile * kTile > x.t.len - a.n_tok + (TREE ? 0 : 1)) {
                cp_async_commit();
                cp_async_wait<0>();
                clean(st);
                mbar_arrive(bar(kKvFull + st));
            } else {
                cp_async_arrive(bar(kKvFull + st));
            }
            return true;
        };
        if constexpr (R == 32) {
            Tiles x = begin();
            while (load(x, warp >= kLoads + 2)) {}
        } else {
            Tiles k = begin(), v = begin();
            load(k, false);
            do
                load(k, false);
            while (load(v, true));
        }
        cp_async_commit();
        cp_async_wait<0>();
    } else if (warp == kMmas) {
        // ---- MMAs: the whole warp walks the tiles, one elected lane issues
        const bool issue = elect_one();
        const uint32_t negate = a.scale < 0.f ? 1u << 13 : 0u;  // x = |sc| (-Q) K^T
        const uint32_t id_s = (F16 ? idesc_f16_f32(128, kTile, 0, 0) : idesc_bf16_f32(128, kTile, 0, 0)) | negate;
        const uint32_t id_o = F16 ? idesc_f16_f32(128, D, 0, 1) : idesc_bf16_f32(128, D, 0, 1);
        const uint64_t q0 = smem_desc_sw128(base, 0, 1024);
        const uint64_t k0 = smem_desc_sw128(base + Sh::OFF_RING, 0, 1024);
        const uint64_t v0 = smem_desc_sw128(base + Sh::OFF_RING, Sh::BOX, 1024);
        uint32_t gs = 0, g = 0;
        Walk k_walk = walk;
        Triple kt;
        kt.tile0 = kt.tile1 = 0;
        int k_tile = 0, k_it = -1;
        bool k_more = true;
        // S of the next tile: whether there is one (Q and its keys are waited for), the product for a
        // block of rows, and the step to the tile after.
        auto keys = [&] {
            if (k_tile == kt.tile1) {
                k_more = k_walk.next(a, sp, L.blocks_of_rows, kt);
                if (!k_more) return false;
                ++k_it;
                if (!wait(kQFull + k_it % Sh::QS, k_it / Sh::QS)) return false;
                k_tile = kt.tile0;
            }
            const uint32_t i = key_stage(gs);
            if (!wait(kKvFull + i % N, i / N)) return false;
            fence_proxy_async_smem();  // copies by other threads, before the MMAs read them
            tc_fence_after_sync();
            return true;
        };
        auto score = [&](int b) {
            const uint32_t st = key_stage(gs) % N;
            const uint64_t qd = q0 + ((k_it % Sh::QS * (B * Sh::Q_BYTES) + b * Sh::Q_BYTES) >> 4);
            const uint64_t kd = k0 + (uint64_t)(st * (Sh::STAGE >> 4));
            const uint32_t d = tmem + kColsS + b * 128 + (gs & 1) * kTile;
            if (issue) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_bf16(d, qd + (((k >> 2) * Sh::Q_BLOCK + (k & 3) * 32) >> 4),
                             kd + (((k >> 2) * Sh::BOX + (k & 3) * 32) >> 4), id_s, k > 0);
                mma_commit(bar(kSFull + 2 * b + (gs & 1)));
                if (b == B - 1) {
                    mma_commit(bar(kKvEmpty + st));
                    if (k_tile == kt.tile1 - 1) mma_commit(bar(kQEmpty + k_it % Sh::QS));
                }
            }
            __syncwarp();
        };
        auto scored = [&] {
            ++k_tile;
            ++gs;
        };
#pragma unroll 1
        for (int x = 0; x < 2 && keys(); ++x) {
#pragma unroll
            for (int b = 0; b < B; ++b) score(b);
            scored();
        }
        for (int it = 0; ok && walk.next(a, sp, L.blocks_of_rows, t); ++it) {
            for (int tile = t.tile0; ok && tile < t.tile1; ++tile) {
                const bool ahead = g > 0 && k_more && keys();
                if (!ok) break;
                const uint32_t i = value_stage(g), st = i % N;
                const uint64_t vd = v0 + (uint64_t)(st * (Sh::STAGE >> 4));
                const uint32_t p = tmem + kColsS + (g & 1) * kTile;
                // block by block, so that one's P is made while the other's products run
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    if (ahead) score(b);  // over P of the tile before, whose P V is issued
                    if (b == 0) {
                        if (tile == t.tile0 && it > 0 && !wait(kOFree, it - 1)) break;
                        if (!wait(kKvFull + st, i / N)) break;
                    }
                    if (!wait(kPFull + 2 * b + (g & 1), g >> 1)) break;
                    fence_proxy_async_smem();
                    tc_fence_after_sync();
                    if (issue) {
#pragma unroll
                        for (int k = 0; k < kTile / 16; ++k)
                            pair::mma_ts_one(tmem + b * 128, p + b * 128 + k * 8, vd + ((k * 16 * 128) >> 4), id_o,
                                             tile > t.tile0 || k > 0);
                        mma_commit(bar(kPvDone + 2 * b + (g & 1)));
                        if (b == B - 1) {
                            mma_commit(bar(kKvEmpty + st));
                            if (tile == t.tile1 - 1) mma_commit(bar(kODone));
                        }
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (ahead) scored();
                ++g;
            }
        }
    } else {
        // ---- Q: row r of the block at its place in the operand tile; rows past the last are left
        const int w = warp - kMmas - 1;
        for (int it = 0; ok && walk.next(a, sp, L.blocks_of_rows, t); ++it) {
            const int z = it % Sh::QS;
            if (it >= Sh::QS && !wait(kQEmpty + z, it / Sh::QS - 1)) break;
            const int live = min(sp.block_rows, rows - t.rb * sp.block_rows);
            constexpr int RPI = 32 / CPR;
            for (int row = w * RPI + lane / CPR; row < live; row += 3 * RPI) {
                const int r = t.rb * sp.block_rows + row, j = r / a.group;
                const int64_t tok = (int64_t)t.s * a.n_tok + j;
                const int chunk = lane % CPR;
                cp_async16(base + (z * B + (row >> 7)) * Sh::Q_BYTES + (chunk >> 3) * Sh::Q_BLOCK + (row & 127) * 128 + (((chunk & 7) ^ (row & 7)) << 4),
                           a.q.p + tok * a.q.ts + (int64_t)(t.h * a.group + r - j * a.group) * a.q.hs + chunk * 8, 16u);
            }
            cp_async_arrive(bar(kQFull + z));
            if (w == 0 && lane == 0 && t.tile0 == 0) leave_parts(a, sp, L, cut, me, t.s, t.h, t.rb, t.seg0, t.tiles);
            __syncwarp();
        }
        cp_async_commit();
        cp_async_wait<0>();
    }
    if (!ok) {
        // a wait gave up: leave the copies and MMAs in flight time to end before shared
        // memory and TMEM go (they wait for nothing themselves)
        atomicCAS(a.err, 0, (int32_t)GDR_ERR_DEVICE_TIMEOUT);
        const long long t_end = clock64() + 4000000;
        while (clock64() < t_end) {}
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kMmas) tmem_dealloc(tmem, 512);
}

template <int D, bool F16, bool TREE, int B>
cudaError_t launch_as(const Args &a, cudaStream_t s) {
    static SmemOptIn opt_in;
    using Sh = Shape<D, B>;
    const cudaError_t e = opt_in.set(reinterpret_cast<const void *>(wide_kernel<D, F16, TREE, B>), (int)Sh::SMEM);
    if (e != cudaSuccess) return e;
    wide_kernel<D, F16, TREE, B><<<kBlocks, Sh::THREADS, Sh::SMEM, s>>>(a);
    return cudaGetLastError();
}

template <int D, bool F16>
cudaError_t launch(const Args &a, cudaStream_t s) {
    if (!a.parents) return launch_as<D, F16, false, 1>(a, s);
    if constexpr (D <= 128) {
        if (kind_of(a.n_tok * a.group, D, true, (int64_t)a.n_seqs * a.h_kv) == kPaired) return launch_as<D, F16, true, 2>(a, s);
    }
    return launch_as<D, F16, true, 1>(a, s);
}

}  // namespace

cudaError_t launch_decode_wide(const Args &a, cudaStream_t s) {
    if (a.d == 64) return a.f16 ? launch<64, true>(a, s) : launch<64, false>(a, s);
    if (a.d == 128) return a.f16 ? launch<128, true>(a, s) : launch<128, false>(a, s);
    return a.f16 ? launch<256, true>(a, s) : launch<256, false>(a, s);
}

}  // namespace attn
}  // namespace gdr
