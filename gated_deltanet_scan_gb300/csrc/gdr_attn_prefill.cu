// Causal attention over whole packed prompts, on tcgen05 tensor cores.
//
// Math.  For one key/value head the queries of the `group` heads that share it are
// rows of one matrix, token by token: row r of a block of 128 is query head
// r % group of its token r / group.  Over tiles of 128 tokens, with the running
// reference m of each row,
//     x = sc Q K^T  (sc = scale log2 e),   p = 2^(x - m),   l += sum p,   O += P V,
// and o = O / l at the end.  m follows the row's maximum only when that is 2^8 above
// it; O and l are then multiplied by 2^(m_old - m).
//
// Bound by the tensor cores: 4 d flops a visible (query, token) pair.  A pair of CTAs
// (a cluster of two SMs) works on 256 rows with cta_group::2 MMAs: each CTA holds its
// 128 rows of Q, S = Q K^T and O, and half of every key tile (64 tokens) and value
// tile (half of the columns), so a tile crosses L2 once for 256 rows (32 bytes a clock
// and SM at full MMA rate, against the 64 a single CTA of 128 rows would need).  O
// (d columns) and two S tiles (128 each) fill TMEM at d = 256; P overwrites its S as
// 16-bit pairs and is the second MMA's A operand from there.
//
// Twelve warps.  One thread loads K and V tiles by TMA into a ring, in the order the
// MMAs take them: K0, K1, V0, K2, V1, ...  One thread of the leading CTA issues
// S_{j+1} before P V_j, so the tensor pipe has work while P_j is made.  Two warpgroups
// make P: one the even tiles, the other the odd ones, one row per thread.  Each hands
// the row's reference m on to the other as soon as it has its tile's maximum, so they
// work on two tiles at the same time; each keeps the sum l of its own tiles.  A
// warpgroup that raises m rescales O itself, between the two MMAs.
//
// A token must not see what later tokens or other sequences hold, even a NaN, and 0
// times NaN is NaN.  In S that is a select.  In the few tiles in which some row of the
// pair does not see every token, two warps replace the value tile's infinities and
// NaNs by zeros before the MMA reads it; where they found any, the rows that do see
// them get them added at the end.
#include "gdr_attn_common.cuh"
#include "gdr_attn_ptx.cuh"
#include "gdr_internal.h"
#include "tc_ptx.cuh"

namespace gdr {
namespace attn {
namespace {

using namespace tc;

constexpr int kThreads = 384;
constexpr int kPairs = 76;   // CTA pairs on 152 SMs
constexpr int kRows = 128;  // rows per CTA
constexpr int kTile = 128;  // tokens per tile
constexpr long long kWaitLimit = 4000000000LL;  // SM clocks (about 2 s)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;

template <int D>
struct Shape {
    static constexpr uint32_t Q_BLOCK = kRows * 128;       // 64 columns of Q
    static constexpr uint32_t Q_BYTES = Q_BLOCK * (D / 64);
    static constexpr int VC = D / 2 < 64 ? D / 2 : 64;     // columns of one value box
    static constexpr int V_BOXES = D / 2 / VC;
    static constexpr uint32_t V_BOX = kTile * VC * 2;
    static constexpr uint32_t K_BOX = 64 * 128;            // 64 tokens, 64 columns
    static constexpr uint32_t STAGE = 128 * D;             // half a key or value tile
    static constexpr int STAGES = D == 256 ? 5 : 8;
    static constexpr uint32_t OFF_RING = Q_BYTES;
    static constexpr uint32_t OFF_M = OFF_RING + STAGES * STAGE;  // float [2][128]: m handed on
    static constexpr uint32_t OFF_L = OFF_M + 1024;               // float [2][128]: the warpgroups' l
    static constexpr uint32_t OFF_BAR = OFF_L + 1024;
    static constexpr uint32_t OFF_WORDS = OFF_BAR + 56 * 8;       // TMEM address, flags
    static constexpr uint32_t BYTES = OFF_WORDS + 128;
    static_assert(BYTES <= 227 * 1024, "shared memory of one CTA");
    // TMEM columns: O at 0, S tiles from here on.  With three of them (d <= 128) the
    // MMAs of two more tiles' S run while a tile's P is made; at d = 256 two fit.
    static constexpr int S_TILES = D == 256 ? 2 : 3;
    static constexpr uint32_t COLS_S = 512 - S_TILES * kTile;
    static constexpr int AHEAD = S_TILES - 1;              // tiles by which S runs ahead of P V
};

// barriers, as 8-byte words from OFF_BAR
enum Bar {
    kQFull = 0,                // on the leading CTA
    kQEmpty = kQFull + 1,
    kKvFull = kQEmpty + 1,     // [stages], on the leading CTA
    kKvEmpty = kKvFull + 8,    // [stages]
    kVLocal = kKvEmpty + 8,    // [stages]: a value tile to be looked through
    kSFull = kVLocal + 8,      // [S tiles]
    kPFull = kSFull + 3,       // [S tiles], on the leading CTA
    kPvDone = kPFull + 3,      // [2]: P V of even and odd tiles
    kODone = kPvDone + 2,      // a block's last P V
    kOFree = kODone + 1,       // O is read, on the leading CTA
    kMReady = kOFree + 1,      // [2][4]: m of a warp's rows
    kPatch = kMReady + 8,      // [8]: a block's flags
    kBars = kPatch + 8,
};
static_assert(kBars <= 56, "barrier words");

struct Maps {
    CUtensorMap q, k, v;
};

// Packed rows: tokens per CTA and per pair.
__host__ __device__ inline int tokens_per_cta(int group) { return kRows / group; }

// One block of work: 2 x 128 rows of one sequence and key/value head.
struct Block {
    int64_t t0;   // the sequence's first token
    int len;      // its tokens
    int h;        // key/value head
    int first;    // the block's first token in the sequence
    int n;        // tiles of tokens its rows see
    int j_clean;  // the first of them that some row sees only in part
};

// A pair's blocks, found by one warp: block number `want` counts from the last block of
// the last sequence, the one whose rows see most.  Numbers only grow, so the sequences
// behind the cursor are not looked at again.
struct Cursor {
    int hi;         // sequences below this one are still to come
    int64_t after;  // blocks (of one head) of the others
    int item;       // round of this pair
    __device__ __forceinline__ bool next(const Args &a, int pair_id, int pairs, int lane, Block &b) {
        // pairs take the blocks of a round in turn, back and forth: the sizes even out
        const int64_t number = (int64_t)item * pairs + ((item & 1) ? pairs - 1 - pair_id : pair_id);
        ++item;
        const int64_t want =
            number >> 31 ? number / a.h_kv : (int64_t)((uint32_t)number / (uint32_t)a.h_kv);
        const int per_pair = 2 * tokens_per_cta(a.group);
        while (hi > 0) {
            const int s = hi - 1 - lane;
            int64_t t0 = 0, t1 = 0;
            if (s >= 0) {
                t0 = a.cu[s];
                t1 = a.cu[s + 1];
                if (t0 < 0 || t1 < t0 || t1 > a.t_total) {
                    record_invalid(a.err);
                    t0 = t1 = 0;
                }
            }
            const int n = (int)((uint32_t)(t1 - t0 + per_pair - 1) / (uint32_t)per_pair);
            int x = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            const int64_t end = after + x;
            const uint32_t hit = __ballot_sync(0xffffffffu, want >= end - n && want < end);
            if (hit) {
                const int src = __ffs(hit) - 1;
                b.t0 = __shfl_sync(0xffffffffu, t0, src);
                b.len = (int)(__shfl_sync(0xffffffffu, t1, src) - b.t0);
                b.h = (int)(number - want * a.h_kv);
                b.first = (int)(__shfl_sync(0xffffffffu, end, src) - 1 - want) * per_pair;
                b.n = (min(b.len, b.first + per_pair) + kTile - 1) / kTile;
                b.j_clean = (b.first + 1) >> 7;
                return true;
            }
            after += __shfl_sync(0xffffffffu, x, 31);
            hi -= 32;
        }
        return false;
    }
};

template <int D, bool F16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ Args a, const __grid_constant__ Maps maps) {
    using Sh = Shape<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    float *const s_m = reinterpret_cast<float *>(smem + Sh::OFF_M);
    float *const s_l = reinterpret_cast<float *>(smem + Sh::OFF_L);
    const uint32_t bars = base + Sh::OFF_BAR;
    uint32_t *const s_tmem = reinterpret_cast<uint32_t *>(smem + Sh::OFF_WORDS);
    uint32_t *const s_flags = s_tmem + 1;  // [8 blocks][2 CTAs]: values to be added at the end
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform for the compiler, too
    const uint32_t rank = pair::cta_rank();
    const int per_cta = tokens_per_cta(a.group);
    const int pair_id = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    auto bar = [&](int i) { return bars + 8u * i; };

    // --- barriers and TMEM
    if (tid == 0) {
        mbar_init(bar(kQFull), 2);
        mbar_init(bar(kQEmpty), 1);
        for (int i = 0; i < Sh::STAGES; ++i) {
            mbar_init(bar(kKvFull + i), 2);
            mbar_init(bar(kKvEmpty + i), 1);
            mbar_init(bar(kVLocal + i), 1);
        }
        for (int i = 0; i < Sh::S_TILES; ++i) {
            mbar_init(bar(kSFull + i), 1);
            mbar_init(bar(kPFull + i), 8);
        }
        mbar_init(bar(kPvDone), 1);
        mbar_init(bar(kPvDone + 1), 1);
        mbar_init(bar(kODone), 1);
        mbar_init(bar(kOFree), 16);
        for (int i = 0; i < 8; ++i) {
            mbar_init(bar(kMReady + i), 1);
            mbar_init(bar(kPatch + i), 2);
        }
        fence_mbar_init();
    }
    if (warp == 9) {
        pair::tmem_alloc(smem_u32(s_tmem), 512);
        pair::tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    pair::cluster_sync();
    tc_fence_after_sync();
    const uint32_t tmem = *s_tmem;
    bool ok = true;
    auto gave_up = [&] {
        // a wait gave up: leave the copies and MMAs in flight time to end before shared
        // memory and TMEM go (they wait for nothing themselves)
        atomicCAS(a.err, 0, (int32_t)GDR_ERR_DEVICE_TIMEOUT);
        const long long t_end = clock64() + 4000000;
        while (clock64() < t_end) {}
    };
    auto all_ok = [&](bool mine_ok) { return __all_sync(0xffffffffu, mine_ok) != 0; };

    // The ring takes a block's tiles in the order K0 .. K_AHEAD, V0, K_{AHEAD + 1}, V1, ...,
    // the last values at the end, and blocks one after the other.  Every role walks the same
    // blocks and counts stages, tiles and blocks through all of them: the counts give stages,
    // S tiles and barrier phases.
    constexpr int A = Sh::AHEAD;
    auto k_index = [](int j) { return j <= A ? j : 2 * j - A; };
    auto v_index = [](int j, int n) { return j <= n - 1 - A ? A + 1 + 2 * j : n + j; };
    Cursor cursor{a.n_seqs, 0, 0};
    Block b;

    // the launch's 384 x 168 registers become 128 x 56 and 256 x 224
    if (warp >= 8) {
        pair::fewer_registers<56>();
        if (warp == 8) {
            // ---- loads (both CTAs: own halves)
            const bool issue = elect_one();
            const uint32_t q_bar = pair::map_to(bar(kQFull), 0), full0 = pair::map_to(bar(kKvFull), 0);
            uint32_t i0 = 0;  // stages before this block's
            for (int it = 0; ok && cursor.next(a, pair_id, pairs, lane, b); ++it) {
                const int t_kv = (int)b.t0;
                auto free_stage = [&](uint32_t i) {
                    const uint32_t use = i / Sh::STAGES;
                    if (use > 0)
                        ok = ok && mbar_wait_bounded(bar(kKvEmpty + i % Sh::STAGES), (use - 1) & 1, kWaitLimit);
                    ok = all_ok(ok);
                    return base + Sh::OFF_RING + (i % Sh::STAGES) * Sh::STAGE;
                };
                auto load_k = [&](int j) {
                    const uint32_t i = i0 + k_index(j), dst = free_stage(i);
                    if (ok && issue) {
                        const uint32_t full = full0 + 8u * (i % Sh::STAGES);
                        pair::arrive_expect_remote(full, Sh::STAGE);
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            pair::tma_load_3d_pair(dst + c * Sh::K_BOX, &maps.k, full, c * 64, b.h,
                                                   t_kv + j * kTile + (int)rank * 64);
                    }
                    __syncwarp();
                };
                load_k(0);
                if (it > 0) ok = all_ok(ok && mbar_wait_bounded(bar(kQEmpty), (it - 1) & 1, kWaitLimit));
                if (ok && issue) {
                    pair::arrive_expect_remote(q_bar, (uint32_t)(D / 64) * 128u * (uint32_t)(per_cta * a.group));
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        pair::tma_load_3d_pair(base + c * Sh::Q_BLOCK, &maps.q, q_bar, c * 64, b.h * a.group,
                                               t_kv + b.first + (int)rank * per_cta);
                }
                __syncwarp();
                for (int j = 1; j <= A && j < b.n; ++j) load_k(j);
                for (int j = 0; j < b.n && ok; ++j) {
                    if (j > 0 && j + A < b.n) load_k(j + A);
                    const uint32_t i = i0 + v_index(j, b.n), st = i % Sh::STAGES, dst = free_stage(i);
                    if (ok && issue) {
                        const int x = (int)rank * (D / 2);
                        if (j >= b.j_clean) {  // looked through by warps 10 and 11, which then report the stage full
                            mbar_arrive_expect_tx(bar(kVLocal + st), Sh::STAGE);
#pragma unroll
                            for (int c = 0; c < Sh::V_BOXES; ++c)
                                tma_load_3d(dst + c * Sh::V_BOX, &maps.v, bar(kVLocal + st), x + c * Sh::VC, b.h,
                                            t_kv + j * kTile);
                        } else {
                            const uint32_t full = full0 + 8u * st;
                            pair::arrive_expect_remote(full, Sh::STAGE);
#pragma unroll
                            for (int c = 0; c < Sh::V_BOXES; ++c)
                                pair::tma_load_3d_pair(dst + c * Sh::V_BOX, &maps.v, full, x + c * Sh::VC, b.h,
                                                       t_kv + j * kTile);
                        }
                    }
                    __syncwarp();
                }
                i0 += 2 * b.n;
            }
        } else if (warp == 9 && rank == 0) {
            // ---- MMAs.  The whole warp walks the tiles and one elected lane issues, so that
            // descriptors are made in uniform registers (one lane in a branch of its own took
            // 1500 clocks a tile, more than the MMAs): a tile's are one base plus constants.
            const bool issue = elect_one();
            const uint32_t negate = a.scale < 0.f ? 1u << 13 : 0u;  // x = |sc| (-Q) K^T
            const uint32_t id_s = (F16 ? idesc_f16_f32(256, kTile, 0, 0) : idesc_bf16_f32(256, kTile, 0, 0)) | negate;
            const uint32_t id_o = F16 ? idesc_f16_f32(256, D, 0, 1) : idesc_bf16_f32(256, D, 0, 1);
            const uint64_t q0 = smem_desc_sw128(base, 0, 1024);
            const uint64_t k0 = smem_desc_sw128(base + Sh::OFF_RING, 0, 1024);
            const uint64_t v0 = Sh::VC == 64 ? smem_desc(base + Sh::OFF_RING, Sh::V_BOX, 1024, kSwizzle128)
                                             : smem_desc(base + Sh::OFF_RING, Sh::V_BOX, 512, kSwizzle64);
            uint32_t i0 = 0, g0 = 0;  // stages and tiles before this block's
            Block ahead;
            bool more = cursor.next(a, pair_id, pairs, lane, ahead);
            for (int it = 0; ok && more; ++it) {
                b = ahead;
                auto score = [&](int j) {
                    const uint32_t i = i0 + k_index(j), st = i % Sh::STAGES, s_tile = (g0 + j) % Sh::S_TILES;
                    ok = all_ok(ok && mbar_wait_bounded(bar(kKvFull + st), (i / Sh::STAGES) & 1, kWaitLimit));
                    if (!ok) return;
                    tc_fence_after_sync();
                    const uint64_t kd = k0 + (uint64_t)(st * (Sh::STAGE >> 4));
                    const uint32_t d = tmem + Sh::COLS_S + s_tile * kTile;
                    if (issue) {
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            pair::mma_ss(d, q0 + (((k >> 2) * Sh::Q_BLOCK + (k & 3) * 32) >> 4),
                                         kd + (((k >> 2) * Sh::K_BOX + (k & 3) * 32) >> 4), id_s, k > 0);
                        pair::commit_both(bar(kKvEmpty + st));
                        pair::commit_both(bar(kSFull + s_tile));
                        if (j == b.n - 1) pair::commit_both(bar(kQEmpty));
                    }
                    __syncwarp();
                };
                ok = all_ok(mbar_wait_bounded(bar(kQFull), it & 1, kWaitLimit));
                // the S tiles are free: the P V that read them are issued
                for (int j = 0; j <= A && j < b.n; ++j) score(j);
                more = cursor.next(a, pair_id, pairs, lane, ahead);  // while P of the first tile is made
                if (it > 0) ok = all_ok(ok && mbar_wait_bounded(bar(kOFree), (it - 1) & 1, kWaitLimit));
                for (int j = 0; j < b.n && ok; ++j) {
                    if (j > 0 && j + A < b.n) score(j + A);  // over P of tile j - 1, whose P V is issued
                    const uint32_t i = i0 + v_index(j, b.n), st = i % Sh::STAGES;
                    const uint32_t g = g0 + j, s_tile = g % Sh::S_TILES;
                    ok = ok && (j < b.j_clean
                                    ? mbar_wait_bounded(bar(kKvFull + st), (i / Sh::STAGES) & 1, kWaitLimit)
                                    : pair::wait_cluster(bar(kKvFull + st), (i / Sh::STAGES) & 1, kWaitLimit));
                    ok = ok && mbar_wait_bounded(bar(kPFull + s_tile), (g / Sh::S_TILES) & 1, kWaitLimit);
                    ok = all_ok(ok);
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint64_t vd = v0 + (uint64_t)(st * (Sh::STAGE >> 4));
                    const uint32_t p = tmem + Sh::COLS_S + s_tile * kTile;
                    if (issue) {
#pragma unroll
                        for (int k = 0; k < kTile / 16; ++k)
                            pair::mma_ts(tmem, p + k * 8, vd + ((k * 16 * (Sh::VC * 2)) >> 4), id_o, j > 0 || k > 0);
                        pair::commit_both(bar(kKvEmpty + st));
                        pair::commit_both(bar(kPvDone + (g & 1)));
                        if (j == b.n - 1) pair::commit_both(bar(kODone));
                    }
                    __syncwarp();
                }
                i0 += 2 * b.n;
                g0 += b.n;
            }
        } else if (warp >= 10) {
            // ---- value tiles that some row sees only in part (both CTAs: own halves)
            uint32_t i0 = 0, turns = 0;  // stages before this block's; per stage, phase of its barrier
            for (int it = 0; cursor.next(a, pair_id, pairs, lane, b); ++it) {
                bool found = false;
                for (int j = b.j_clean; j < b.n; ++j) {  // even after a timeout: the two warps meet in each
                    const uint32_t st = (i0 + v_index(j, b.n)) % Sh::STAGES;
                    ok = ok && mbar_wait_bounded(bar(kVLocal + st), (turns >> st) & 1, kWaitLimit);
                    turns ^= 1u << st;
                    uint4 *const tile = reinterpret_cast<uint4 *>(smem + Sh::OFF_RING + st * Sh::STAGE);
                    constexpr uint32_t e = F16 ? 0x7C007C00u : 0x7F807F80u;
#pragma unroll 4
                    for (int x = tid - 320; ok && x < (int)Sh::STAGE / 16; x += 64) {
                        uint4 w = tile[x];
                        uint32_t *const p = &w.x;
                        bool bad = false;
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const bool lo = (p[y] & e & 0xFFFFu) == (e & 0xFFFFu);
                            const bool hi = (p[y] & e & 0xFFFF0000u) == (e & 0xFFFF0000u);
                            bad = bad || lo || hi;
                            p[y] &= (lo ? 0xFFFF0000u : ~0u) & (hi ? 0xFFFFu : ~0u);
                        }
                        if (bad) {
                            tile[x] = w;
                            found = true;
                        }
                    }
                    fence_proxy_async_smem();
                    named_sync(1, 64);
                    if (tid == 320 && ok) pair::arrive_remote_release(pair::map_to(bar(kKvFull + st), 0));
                }
                // the block's flag, to both CTAs.  Its slot is used again eight blocks on, when this
                // block's last stages have left the ring of at most eight
                const int slot = it & 7;
                found = pair::named_or(2, 64, found);
                if (tid == 320) {
#pragma unroll
                    for (uint32_t r = 0; r < 2; ++r) {
                        pair::store_remote(pair::map_to(smem_u32(s_flags + slot * 2 + rank), r), found);
                        pair::arrive_remote_release(pair::map_to(bar(kPatch + slot), r));
                    }
                }
                i0 += 2 * b.n;
            }
        }
        if (!ok) gave_up();
        __syncwarp();
        pair::cluster_sync();
    } else {
        pair::more_registers<224>();
        // ---- softmax: warpgroup wg takes a block's tiles wg, wg + 2, ...; a thread is a row
        const int wg = warp >> 2, row = tid & 127, wq = warp & 3;
        const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
        // a scale of 0 still has to leave a masked score at minus infinity
        const float sc = fmaxf(fabsf(a.scale), 1e-30f) * kLog2e;
        const int tok = row / a.group, head_in_group = row - tok * a.group;
        const uint32_t p_bars = pair::map_to(bar(kPFull), 0), o_free = pair::map_to(bar(kOFree), 0);
        uint32_t g0 = 0;              // tiles before this block's
        uint32_t turn[2] = {0, 0};    // tiles of either warpgroup before this block's
        Block ahead;
        bool more = cursor.next(a, pair_id, pairs, lane, ahead);
        for (int it = 0; more; ++it) {
            b = ahead;
            const int n = b.n, mine = b.first + (int)rank * per_cta;
            const int token = mine + tok;  // in the sequence
            float m_own = -CUDART_INF_F, l = 0.f;
            for (int j = wg; ok && j < n; j += 2) {
                const uint32_t g = g0 + j, st = g % Sh::S_TILES;
                ok = all_ok(mbar_wait_bounded(bar(kSFull + st), (g / Sh::S_TILES) & 1, kWaitLimit));
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t s_at = lanes + Sh::COLS_S + st * kTile;
                uint32_t r[128];
#pragma unroll
                for (int c = 0; c < 128; c += 32) pair::tmem_load32_start(s_at + c, r + c);
                pair::tmem_load_wait(r);
                if (j * kTile + kTile - 1 > mine) {  // some row of this CTA sees only part of the tile
                    const int seen = token - j * kTile;  // columns 0 .. seen
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (c > seen) r[c] = 0xFF800000u;
                }
                float top[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) top[e] = __uint_as_float(r[e]);
#pragma unroll
                for (int c = 4; c < 124; c += 8) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        top[e] = pair::max3(top[e], __uint_as_float(r[c + e]), __uint_as_float(r[c + 4 + e]));
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) top[e] = fmaxf(top[e], __uint_as_float(r[124 + e]));
                const float x_top = sc * fmaxf(pair::max3(top[0], top[1], top[2]), top[3]);
                // the reference after the tile before, from the other warpgroup
                float m_prev = -CUDART_INF_F;
                if (j > 0) {
                    const uint32_t turn_prev = turn[wg ^ 1] + ((j - 1) >> 1);
                    ok = all_ok(mbar_wait_bounded(bar(kMReady + 4 * (wg ^ 1) + wq), turn_prev & 1, kWaitLimit));
                    if (!ok) break;
                    m_prev = s_m[(wg ^ 1) * 128 + row];
                }
                const bool raise = j == 0 || x_top > m_prev + kSlack;
                const float m = raise ? x_top : m_prev;
                s_m[wg * 128 + row] = m;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kMReady + 4 * wg + wq));

                if (j > 0 && __any_sync(0xffffffffu, raise)) {
                    // O is that of tiles 0 .. j - 1 then: P V of tile j waits for this warp's P.  (S of
                    // tile j is complete, so P V of tile j - 3 is: this barrier's phase is unambiguous.)
                    ok = all_ok(mbar_wait_bounded(bar(kPvDone + ((g - 1) & 1)), ((g - 1) >> 1) & 1, kWaitLimit));
                    if (!ok) break;
                    tc_fence_after_sync();
                    const float f = raise ? fast_exp2(m_prev - m) : 1.f;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        pair::tmem_load32(lanes + c, o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        pair::tmem_store32(lanes + c, o);
                    }
                }
                l *= m_own == m ? 1.f : fast_exp2(m_own - m);
                m_own = m;
                uint64_t sum[2] = {0, 0};
                const uint64_t sc2 = pair::pack_f32x2(sc, sc), m2 = pair::pack_f32x2(-m, -m);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t p[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const int i = half * 64 + 2 * c;
                        float x, y;
                        pair::unpack_f32x2(
                            pair::fma_f32x2(pair::pack_f32x2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), sc2,
                                            m2),
                            x, y);
                        x = fast_exp2(x);
                        y = fast_exp2(y);
                        sum[c & 1] = pair::add_f32x2(sum[c & 1], pair::pack_f32x2(x, y));
                        p[c] = pack2<F16>(x, y);
                    }
                    pair::tmem_store32(s_at + half * 32, p);
                }
                {
                    float x, y;
                    pair::unpack_f32x2(pair::add_f32x2(sum[0], sum[1]), x, y);
                    l += x + y;
                }
                pair::tmem_store_wait();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) pair::arrive_remote(p_bars + 8u * st);
            }
            more = cursor.next(a, pair_id, pairs, lane, ahead);  // while the last P V runs
            s_l[wg * 128 + row] = l;
            if (wg >= n) s_m[wg * 128 + row] = -CUDART_INF_F;  // no tile was this warpgroup's
            named_sync(3, 256);
            const float2 e0 = make_float2(s_m[row], s_l[row]), e1 = make_float2(s_m[128 + row], s_l[128 + row]);
            // read: the next block may write them.  A warp whose wait gave up comes here, too: all leave.
            ok = !pair::named_or(4, 256, !ok);
            if (!ok) break;
            ok = all_ok(mbar_wait_bounded(bar(kODone), it & 1, kWaitLimit) &&
                        pair::wait_cluster(bar(kPatch + (it & 7)), (it >> 3) & 1, kWaitLimit));
            if (ok) {
                // ---- o = O / l: warpgroup wg writes half of the columns
                tc_fence_after_sync();
                const bool live = tok < per_cta && token < b.len;
                const int64_t t = b.t0 + token;
                const int hq = b.h * a.group + head_in_group;
                const float m = ((n - 1) & 1) ? e1.x : e0.x;
                const float l_all = (e0.x == m ? e0.y : e0.y * fast_exp2(e0.x - m)) +
                                    (e1.x == m ? e1.y : e1.y * fast_exp2(e1.x - m));
                const float inv = 1.f / l_all;
                volatile uint32_t *const flags = s_flags + (it & 7) * 2;
                const bool patch = flags[0] | flags[1];
                const int c0 = wg * (D / 2);
                uint16_t *const dst = a.o.p + t * a.o.ts + (int64_t)hq * a.o.hs + c0;
#pragma unroll 1
                for (int c = 0; c < D / 2; c += 32) {
                    uint32_t o[32];
                    pair::tmem_load32(lanes + c0 + c, o);
                    if (c + 32 >= D / 2) {  // this warp has read its part of O
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) pair::arrive_remote(o_free);
                    }
                    if (live && patch) {
                        for (int p = b.j_clean * kTile; p <= token; ++p) {
                            const uint16_t *const v = a.v.p + (b.t0 + p) * a.v.ts + (int64_t)b.h * a.v.hs + c0 + c;
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const float x = unpack1<F16>(v[e]);
                                if (!isfinite(x)) o[e] = __float_as_uint(__uint_as_float(o[e]) + x);
                            }
                        }
                    }
                    if (live) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint4 w;
                            w.x = pack2<F16>(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv);
                            w.y = pack2<F16>(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
                            w.z = pack2<F16>(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv);
                            w.w = pack2<F16>(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv);
                            *reinterpret_cast<uint4 *>(dst + c + e) = w;
                        }
                    }
                    __syncwarp();
                }
                if (wg == 0 && live && a.lse) a.lse[t * a.h_q + hq] = kLn2 * (m + log2f(l_all));
            }
            g0 += n;
            turn[0] += (n + 1) >> 1;
            turn[1] += n >> 1;
        }
        if (!ok) gave_up();
        __syncwarp();
        pair::cluster_sync();
    }
    // both CTAs are done with TMEM and with each other's shared memory
    if (warp == 9) pair::tmem_dealloc(tmem, 512);
}

template <int D>
constexpr uint32_t smem_bytes() {
    // at least 116 KiB, so that one CTA has the SM (and its TMEM) to itself
    return Shape<D>::BYTES < 116u * 1024 ? 116u * 1024 : Shape<D>::BYTES;
}

template <int D, bool F16>
cudaError_t launch(const Args &a, cudaStream_t s) {
    using Sh = Shape<D>;
    Maps m;
    const int per_cta = tokens_per_cta(a.group);
    if (!encode_heads_3d(&m.q, a.q.p, F16, D, a.h_q, a.t_total, a.q.hs, a.q.ts, 64, a.group, per_cta,
                         CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_heads_3d(&m.k, a.k.p, F16, D, a.h_kv, a.t_total, a.k.hs, a.k.ts, 64, 1, 64,
                         CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_heads_3d(&m.v, a.v.p, F16, D, a.h_kv, a.t_total, a.v.hs, a.v.ts, Sh::VC, 1, kTile,
                         Sh::VC == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
        return cudaErrorInvalidValue;
    static SmemOptIn opt_in;
    cudaError_t e = opt_in.set(reinterpret_cast<const void *>(prefill_kernel<D, F16>), (int)smem_bytes<D>());
    if (e != cudaSuccess) return e;
    // one pair per two SMs, or fewer: every sequence has at most one block that is not full
    const int64_t blocks = (a.t_total / (2 * per_cta) + a.n_seqs) * a.h_kv;
    const unsigned pairs = blocks < kPairs ? (unsigned)blocks : kPairs;
    prefill_kernel<D, F16><<<2 * pairs, kThreads, smem_bytes<D>(), s>>>(a, m);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefill(const Args &a, cudaStream_t s) {
    if (a.d == 64) return a.f16 ? launch<64, true>(a, s) : launch<64, false>(a, s);
    if (a.d == 128) return a.f16 ? launch<128, true>(a, s) : launch<128, false>(a, s);
    return a.f16 ? launch<256, true>(a, s) : launch<256, false>(a, s);
}

}  // namespace attn
}  // namespace gdr
