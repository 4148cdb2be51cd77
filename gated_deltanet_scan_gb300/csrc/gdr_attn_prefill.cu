// Causal attention over whole packed prompts, on tcgen05 tensor cores.
//
// Math.  For one key/value head the queries of the `group` heads that share it are
// rows of one matrix, token by token: row r of a block of 128 is query head
// r % group of its token r / group.  Over tiles of 128 tokens, with the running
// reference m of each row,
//     x = sc Q K^T  (sc = scale log2 e),   p = 2^(x - m),   l += sum p,   O += P V,
// and o = O / l at the end.  m lies under the row's maximum as Reference says and follows
// it only when p could grow too large; O and l are then multiplied by 2^(m_old - m).
//
// Bound by the tensor cores: 4 d flops a visible (query, token) pair.  A pair of CTAs
// (a cluster of two SMs) works on 256 rows with cta_group::2 MMAs: each CTA holds its
// 128 rows of Q, S = Q K^T and O, and half of every key tile (64 tokens) and value
// tile (half of the columns), so a tile crosses L2 once for 256 rows (32 bytes a clock
// and SM at full MMA rate, against the 64 a single CTA of 128 rows would need).  O
// (d columns) and two S tiles (128 each) fill TMEM at d = 256; P overwrites its S as
// 16-bit pairs and is the second MMA's A operand from there.
//
// Sixteen warps, persistent: every pair walks its blocks of 256 rows, and all roles run
// over the blocks' ends, so that a block's start and end hide behind its neighbours'.
//   loads   one warp; K and V tiles by TMA into a ring, in the order the MMAs take them:
//           K runs AHEAD tiles ahead of V, over the blocks' ends too.  It also finds the
//           blocks and tells the other roles (entries of four blocks in shared memory).
//   MMAs    one warp of the leading CTA; S of the tile AHEAD comes before P V of this one,
//           so the tensor pipe has work while P is made.
//   P       two warpgroups, one the even tiles, the other the odd ones, one row per thread.
//           Each hands the row's reference m on to the other as soon as it has its tile's
//           maximum, so they work on two tiles at the same time; each keeps the sum l of its
//           own tiles.  A warpgroup that raises m rescales O itself, between the two MMAs.
//   O / l   a warpgroup reads O when a block's last P V is done, and stores the result while
//           the next block's first tiles are already in work.
//
// P is rounded to 16 bits, the second MMA's type: the products bound this kernel, and more
// bits would take a third one.
//
// A token must not see what later tokens or other sequences hold, even a NaN, and 0
// times NaN is NaN.  In S that is a select.  In the few tiles in which some row of the
// pair does not see every token, two warps replace the value tile's infinities and
// NaNs by zeros before the MMA reads it; where they found any, the rows that do see
// them get them added at the end.
#include "gdr_attn_common.cuh"
#include "gdr_attn_mma.cuh"
#include "gdr_attn_ptx.cuh"
#include "gdr_internal.h"
#include "tc_ptx.cuh"

namespace gdr {
namespace attn {
namespace {

using namespace tc;

constexpr int kThreads = 512;
constexpr int kPairs = 76;   // CTA pairs on 152 SMs
constexpr int kRows = 128;  // rows per CTA
constexpr int kTile = 128;  // tokens per tile

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
    static constexpr int Q_TILES = D == 256 ? 1 : 2;       // the next block's Q loads beside this one's
    static constexpr uint32_t OFF_RING = Q_TILES * Q_BYTES;
    static constexpr uint32_t OFF_M = OFF_RING + STAGES * STAGE;  // float [128]: m handed on
    static constexpr uint32_t OFF_L = OFF_M + 512;                // float [2][128]: l of a block's other warpgroup
    static constexpr uint32_t OFF_INV = OFF_L + 1024;             // float [2][128]: a block's 1 / l
    static constexpr uint32_t OFF_ENTRY = OFF_INV + 1024;         // int4 [4]: blocks
    static constexpr uint32_t OFF_WORDS = OFF_ENTRY + 64;         // TMEM address; flags [4][2]
    static constexpr uint32_t OFF_BAR = OFF_WORDS + 48;
    static constexpr int BARS = 3 * STAGES + 2 * (D == 256 ? 2 : 3) + 28;
    static constexpr uint32_t BYTES = OFF_BAR + 8 * BARS;
    static_assert(BYTES <= 227 * 1024, "shared memory of one CTA");
    // TMEM columns: O at 0, S tiles from here on.  With three of them (d <= 128) the
    // MMAs of two more tiles' S run while a tile's P is made; at d = 256 two fit.
    static constexpr int S_TILES = D == 256 ? 2 : 3;
    static constexpr uint32_t COLS_S = 512 - S_TILES * kTile;
    static constexpr int AHEAD = S_TILES - 1;              // tiles by which S runs ahead of P V
};

// barriers, as 8-byte words from OFF_BAR
template <int D>
struct Bar {
    static constexpr int N = Shape<D>::STAGES, S = Shape<D>::S_TILES;
    static constexpr int QFull = 0;              // [Q tiles], on the leading CTA
    static constexpr int QEmpty = QFull + 2;     // [Q tiles]
    static constexpr int KvFull = QEmpty + 2;    // [stages], on the leading CTA
    static constexpr int KvEmpty = KvFull + N;   // [stages]
    static constexpr int VLocal = KvEmpty + N;   // [stages]: a value tile to be looked through
    static constexpr int SFull = VLocal + N;     // [S tiles]
    static constexpr int PFull = SFull + S;      // [S tiles], on the leading CTA
    static constexpr int PvDone = PFull + S;     // [2]: P V of even and odd tiles
    static constexpr int ODone = PvDone + 2;     // a block's last P V
    static constexpr int OFree = ODone + 1;      // O is read, on the leading CTA
    static constexpr int MReady = OFree + 1;     // [4]: m of a warp's rows
    static constexpr int Patch = MReady + 4;     // [4 blocks]: flags
    static constexpr int Block = Patch + 4;      // [4 blocks]: entries
    static constexpr int Read = Block + 4;       // [4 blocks]: entry, flags and 1 / l are read (P: 8 warps, O: 4)
    static constexpr int LOther = Read + 4;      // [2 blocks]: l of the warpgroup that has not the last tile
    static constexpr int Inv = LOther + 2;       // [2 blocks]: 1 / l
    static constexpr int COUNT = Inv + 2;
};

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

// A pair's blocks, found by one warp.  Sequences are taken 32 at a time from the last, and
// the blocks of such a group by their index in the sequence, the largest first: so the
// longest blocks come first, and the pairs, which take a round's blocks in turn, back and
// forth, come out even (8 prompts of 512 to 8192 tokens, sequence by sequence: the last
// pair 6% over the mean).  Numbers only grow, so groups behind the cursor are not looked
// at again.
struct Cursor {
    int hi;         // sequences below this one are still to come
    int64_t after;  // blocks (of one head) of the groups behind
    int item;       // round of this pair
    __device__ __forceinline__ bool next(const Args &a, int pair_id, int pairs, int lane, Block &b) {
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
                // the short kernel's, which is launched beside this one for several sequences
                if (a.n_seqs > 1 && t1 - t0 <= short_tokens(a.group)) t1 = t0;
            }
            const int n = (int)((uint32_t)(t1 - t0 + per_pair - 1) / (uint32_t)per_pair);
            auto from = [&](int level) {  // blocks of this index or above in the group
                return (int64_t)__reduce_add_sync(0xffffffffu, (uint32_t)max(0, n - level));
            };
            const int64_t all = from(0), u = want - after;
            if (u < all) {
                int lo = 0, up = __reduce_max_sync(0xffffffffu, n);  // from(lo) > u >= from(up)
                while (up - lo > 1) {
                    const int mid = (lo + up) >> 1;
                    if (from(mid) > u)
                        lo = mid;
                    else
                        up = mid;
                }
                // the sequences that have a block `lo`, the last one first
                const uint32_t have = __ballot_sync(0xffffffffu, n > lo);
                const int rank = (int)(u - from(up));
                const uint32_t me = __ballot_sync(
                    0xffffffffu, n > lo && __popc(have & ((1u << lane) - 1u)) == rank);
                const int src = __ffs(me) - 1;
                b.t0 = __shfl_sync(0xffffffffu, t0, src);
                b.len = (int)(__shfl_sync(0xffffffffu, t1, src) - b.t0);
                b.h = (int)(number - want * a.h_kv);
                b.first = lo * per_pair;
                b.n = (min(b.len, b.first + per_pair) + kTile - 1) / kTile;
                b.j_clean = (b.first + 1) >> 7;
                return true;
            }
            after += all;
            hi -= 32;
        }
        return false;
    }
};

template <int D, bool F16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ Args a, const __grid_constant__ Maps maps) {
    using Sh = Shape<D>;
    using Bar = Bar<D>;
    static_assert(Bar::COUNT == Sh::BARS, "barrier words");
    constexpr int A = Sh::AHEAD, N = Sh::STAGES, S = Sh::S_TILES, QT = Sh::Q_TILES;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    float *const s_m = reinterpret_cast<float *>(smem + Sh::OFF_M);
    float *const s_l = reinterpret_cast<float *>(smem + Sh::OFF_L);
    float *const s_inv = reinterpret_cast<float *>(smem + Sh::OFF_INV);
    int4 *const s_entry = reinterpret_cast<int4 *>(smem + Sh::OFF_ENTRY);
    uint32_t *const s_tmem = reinterpret_cast<uint32_t *>(smem + Sh::OFF_WORDS);
    uint32_t *const s_flags = s_tmem + 1;  // [4 blocks][2 CTAs]: values to be added at the end
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform for the compiler, too
    const uint32_t rank = pair::cta_rank();
    const int per_cta = tokens_per_cta(a.group);
    auto bar = [&](int i) { return base + Sh::OFF_BAR + 8u * i; };

    // the short kernel may start beside this one: neither reads what the other writes
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 8 && elect_one()) {
        pair::prefetch_map(&maps.q);
        pair::prefetch_map(&maps.k);
        pair::prefetch_map(&maps.v);
    }
    Cursor cursor{a.n_seqs, 0, 0};
    Block kb;  // the loading warp goes on with these
    if (!cursor.next(a, blockIdx.x >> 1, gridDim.x >> 1, lane, kb)) return;  // no block: both CTAs leave

    // --- barriers and TMEM
    if (tid < 8) s_flags[tid] = 0;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(Bar::QFull + i), 2);
            mbar_init(bar(Bar::QEmpty + i), 1);
            mbar_init(bar(Bar::PvDone + i), 1);
            mbar_init(bar(Bar::LOther + i), 4);
            mbar_init(bar(Bar::Inv + i), 4);
        }
        for (int i = 0; i < N; ++i) {
            mbar_init(bar(Bar::KvFull + i), 2);
            mbar_init(bar(Bar::KvEmpty + i), 1);
            mbar_init(bar(Bar::VLocal + i), 1);
        }
        for (int i = 0; i < S; ++i) {
            mbar_init(bar(Bar::SFull + i), 1);
            mbar_init(bar(Bar::PFull + i), 8);
        }
        mbar_init(bar(Bar::ODone), 1);
        mbar_init(bar(Bar::OFree), 8);
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(Bar::MReady + i), 1);
            mbar_init(bar(Bar::Patch + i), 2);
            mbar_init(bar(Bar::Block + i), 1);
            mbar_init(bar(Bar::Read + i), 12);
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
    // every lane of the warp waits, and all of them go on or give up
    auto wait = [&](int i, uint32_t parity) {
        ok = __all_sync(0xffffffffu, ok && pair::wait_bounded(bar(i), parity & 1)) != 0;
        return ok;
    };
    // Block number `it` of this pair, from the entry the loading warp left; n = 0: there is none.
    auto fetch = [&](int it, Block &b) {
        if (!wait(Bar::Block + (it & 3), it >> 2)) return false;
        const int4 e = s_entry[it & 3];
        b.t0 = e.x;
        b.len = e.y;
        b.first = e.z;
        b.h = e.w;
        b.n = (min(b.len, b.first + 2 * per_cta) + kTile - 1) / kTile;
        b.j_clean = (b.first + 1) >> 7;
        return b.n > 0;
    };

    // Roles count stages (i), tiles (g) and blocks (it) through all of a pair's blocks: the
    // counts give stages, S tiles and barrier phases.  Stage order: K of tiles 0 .. A, V of
    // tile 0, K of tile A + 1, V of tile 1, ..., at the very end the last values.

    // the launch's 512 x 128 registers become 128 x 56, 128 x 120 and 256 x 168
    if (warp >= 8 && warp < 12) {
        pair::fewer_registers<56>();
        if (warp == 8) {
            // ---- loads (both CTAs: own halves)
            const bool issue = elect_one();
            const uint32_t q_full = pair::map_to(bar(Bar::QFull), 0), kv_full = pair::map_to(bar(Bar::KvFull), 0);
            uint32_t i = 0;
            // Q of block q_it is still to be loaded, when its place is free
            int q_it = 0, q_token = 0, q_head = 0;
            bool q_waits = false;
            auto load_q = [&](bool block) {
                if (!q_waits) return;
                const int slot = q_it % QT, use = q_it / QT;
                if (use > 0) {
                    if (block)
                        wait(Bar::QEmpty + slot, use - 1);
                    else if (!__all_sync(0xffffffffu, mbar_test_wait(bar(Bar::QEmpty + slot), (use - 1) & 1)))
                        return;
                }
                if (ok && issue) {
                    const uint32_t full = q_full + 8u * slot;
                    pair::arrive_expect_remote(full, (uint32_t)(D / 64) * 128u * (uint32_t)(per_cta * a.group));
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        pair::tma_load_3d_pair(base + slot * Sh::Q_BYTES + c * Sh::Q_BLOCK, &maps.q, full, c * 64,
                                               q_head * a.group, q_token);
                }
                __syncwarp();
                q_waits = false;
            };
            auto free_stage = [&] {  // of the ring; Q's place may become free first
                const int st = i % N, use = i / N;
                if (use > 0 && q_waits) {
                    const long long t_end = clock64() + pair::kWaitLimit;
                    while (ok && q_waits &&
                           !__all_sync(0xffffffffu, mbar_test_wait(bar(Bar::KvEmpty + st), (use - 1) & 1))) {
                        load_q(false);
                        if (clock64() > t_end) ok = false;
                        ok = __all_sync(0xffffffffu, ok);
                    }
                }
                if (use > 0) wait(Bar::KvEmpty + st, use - 1);
                return base + Sh::OFF_RING + st * Sh::STAGE;
            };
            Block vb;
            int k_it = -1, kj = kb.n, v_it = 0, vj = 0;
            bool k_more = true;
            auto load_k = [&] {
                if (kj == kb.n) {  // the next block
                    load_q(true);
                    ++k_it;
                    kj = 0;
                    if (k_it > 0) k_more = cursor.next(a, blockIdx.x >> 1, gridDim.x >> 1, lane, kb);
                    if (!k_more) kb = Block{};
                    if (k_it >= 4) wait(Bar::Read + (k_it & 3), (k_it >> 2) - 1);
                    if (ok && issue) {
                        s_entry[k_it & 3] = make_int4((int)kb.t0, kb.len, kb.first, kb.h);
                        mbar_arrive(bar(Bar::Block + (k_it & 3)));
                    }
                    __syncwarp();
                    if (!k_more || !ok) return;
                    q_it = k_it;
                    q_token = (int)kb.t0 + kb.first + (int)rank * per_cta;
                    q_head = kb.h;
                    q_waits = true;
                    load_q(false);
                }
                const uint32_t dst = free_stage();
                if (ok && issue) {
                    const uint32_t full = kv_full + 8u * (i % N);
                    pair::arrive_expect_remote(full, Sh::STAGE);
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        pair::tma_load_3d_pair(dst + c * Sh::K_BOX, &maps.k, full, c * 64, kb.h,
                                               (int)kb.t0 + kj * kTile + (int)rank * 64);
                }
                __syncwarp();
                ++kj;
                ++i;
            };
            for (int j = 0; j <= A && k_more && ok; ++j) load_k();
            bool more = ok && fetch(0, vb);
            for (bool start = true; more; start = false) {
                if (!start && k_more) load_k();
                const uint32_t dst = free_stage();
                if (ok && issue) {
                    const int x = (int)rank * (D / 2), y = (int)vb.t0 + vj * kTile, st = i % N;
                    if (vj >= vb.j_clean) {  // looked through by warps 10 and 11, which then report the stage full
                        mbar_arrive_expect_tx(bar(Bar::VLocal + st), Sh::STAGE);
#pragma unroll
                        for (int c = 0; c < Sh::V_BOXES; ++c)
                            tma_load_3d(dst + c * Sh::V_BOX, &maps.v, bar(Bar::VLocal + st), x + c * Sh::VC, vb.h, y);
                    } else {
                        const uint32_t full = kv_full + 8u * st;
                        pair::arrive_expect_remote(full, Sh::STAGE);
#pragma unroll
                        for (int c = 0; c < Sh::V_BOXES; ++c)
                            pair::tma_load_3d_pair(dst + c * Sh::V_BOX, &maps.v, full, x + c * Sh::VC, vb.h, y);
                    }
                }
                __syncwarp();
                ++i;
                if (++vj == vb.n) {
                    vj = 0;
                    more = fetch(++v_it, vb);
                }
                load_q(false);
                more = more && ok;
            }
            load_q(true);
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
            uint32_t i = 0, gs = 0, g = 0;  // stage; tiles of S and of P V so far
            int k_it = -1, kj = 0, kn = 0, v_it = 0, vj = 0;
            bool k_more = true;
            Block b;
            auto score = [&] {
                if (kj == kn) {
                    ++k_it;
                    kj = 0;
                    k_more = fetch(k_it, b);
                    kn = b.n;
                    if (!k_more || !wait(Bar::QFull + k_it % QT, k_it / QT)) return;
                }
                const uint32_t st = i % N, s_tile = gs % S;
                if (!wait(Bar::KvFull + st, i / N)) return;
                tc_fence_after_sync();
                const uint64_t qd = q0 + (uint64_t)((k_it % QT) * (Sh::Q_BYTES >> 4));
                const uint64_t kd = k0 + (uint64_t)(st * (Sh::STAGE >> 4));
                const uint32_t d = tmem + Sh::COLS_S + s_tile * kTile;
                if (issue) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        pair::mma_ss(d, qd + (((k >> 2) * Sh::Q_BLOCK + (k & 3) * 32) >> 4),
                                     kd + (((k >> 2) * Sh::K_BOX + (k & 3) * 32) >> 4), id_s, k > 0);
                    pair::commit_both(bar(Bar::KvEmpty + st));
                    pair::commit_both(bar(Bar::SFull + s_tile));
                    if (kj == kn - 1) pair::commit_both(bar(Bar::QEmpty + k_it % QT));
                }
                __syncwarp();
                ++kj;
                ++gs;
                ++i;
            };
            for (int j = 0; j <= A && k_more && ok; ++j) score();
            Block vb;
            bool more = ok && fetch(0, vb);
            while (more && ok) {
                if (g > 0 && k_more) score();  // over P of the tile before, whose P V is issued
                if (!ok) break;
                const uint32_t st = i % N, s_tile = g % S;
                if (vj == 0 && v_it > 0 && !wait(Bar::OFree, v_it - 1)) break;
                // A looked-through tile that was written was released at cluster scope before this barrier
                // was told, and is read by the MMA alone.  Waits acquire at CTA scope here and for the flags
                // (this CTA's own shared memory): at cluster scope each took 2500 clocks a block.
                if (!wait(Bar::KvFull + st, i / N) || !wait(Bar::PFull + s_tile, g / S)) break;
                tc_fence_after_sync();
                const uint64_t vd = v0 + (uint64_t)(st * (Sh::STAGE >> 4));
                const uint32_t p = tmem + Sh::COLS_S + s_tile * kTile;
                if (issue) {
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        pair::mma_ts(tmem, p + k * 8, vd + ((k * 16 * (Sh::VC * 2)) >> 4), id_o, vj > 0 || k > 0);
                    pair::commit_both(bar(Bar::KvEmpty + st));
                    pair::commit_both(bar(Bar::PvDone + (g & 1)));
                    if (vj == vb.n - 1) pair::commit_both(bar(Bar::ODone));
                }
                __syncwarp();
                ++i;
                ++g;
                if (++vj == vb.n) {
                    vj = 0;
                    more = fetch(++v_it, vb);
                }
            }
        } else if (warp >= 10) {
            // ---- value tiles that some row sees only in part (both CTAs: own halves)
            uint32_t g = 0, k_count = 0, turns = 0;  // V tiles so far; K tiles known of; per stage, its barrier's phase
            int k_it = 0;
            bool k_more = true;
            Block b;
            for (int it = 0;; ++it) {
                const bool more = fetch(it, b);
                ok = !pair::named_or(2, 64, !ok);  // the two warps leave together
                if (!more || !ok) break;
                bool found = false;
                for (int j = 0; j < b.n; ++j, ++g) {
                    if (j < b.j_clean) continue;
                    // stages before this one: V of g tiles, and K of those up to A tiles ahead
                    while (ok && k_more && k_count < g + A + 1) {
                        k_more = fetch(k_it++, kb);
                        k_count += kb.n;
                    }
                    const uint32_t st = (g + min(g + A + 1, k_count)) % N;
                    ok = ok && pair::wait_bounded(bar(Bar::VLocal + st), (turns >> st) & 1);
                    turns ^= 1u << st;
                    bool here = false;
                    uint4 *const tile = reinterpret_cast<uint4 *>(smem + Sh::OFF_RING + st * Sh::STAGE);
                    if (ok) {
                        constexpr int PER = Sh::STAGE / 16 / 64;  // 16-byte pieces per thread
#pragma unroll 1
                        for (int x0 = 0; x0 < PER; x0 += 8) {
                            bool bad = false;
#pragma unroll
                            for (int x = 0; x < 8; ++x) {
                                const uint4 w = tile[tid - 320 + (x0 + x) * 64];
                                bad = bad || any_nonfinite<F16>(w.x, w.y, w.z, w.w);
                            }
                            here = here || bad;
                            if (!bad) continue;
#pragma unroll 1
                            for (int x = 0; x < 8; ++x) {
                                uint4 &w = tile[tid - 320 + (x0 + x) * 64];
                                w = make_uint4(cleaned<F16>(w.x), cleaned<F16>(w.y), cleaned<F16>(w.z),
                                               cleaned<F16>(w.w));
                            }
                        }
                    }
                    if (here) fence_proxy_async_smem();
                    here = pair::named_or(1, 64, here);
                    found = found || here;
                    if (tid == 320 && ok) {
                        const uint32_t full = pair::map_to(bar(Bar::KvFull + st), 0);
                        if (here)  // written: a release, which costs a thousand clocks, only then
                            pair::arrive_remote_release(full);
                        else
                            pair::arrive_remote(full);
                    }
                    __syncwarp();
                }
                // both CTAs look for values to add where a flag is set.  Flags are never reset: a later
                // block of the slot looks in vain
                if (tid == 320 && ok) {
#pragma unroll
                    for (uint32_t r = 0; r < 2; ++r) {
                        const uint32_t told = pair::map_to(bar(Bar::Patch + (it & 3)), r);
                        if (found) {
                            pair::store_remote(pair::map_to(smem_u32(s_flags + (it & 3) * 2 + rank), r), 1);
                            pair::arrive_remote_release(told);
                        } else {
                            pair::arrive_remote(told);
                        }
                    }
                }
                __syncwarp();
            }
        }
        if (!ok) gave_up();
        __syncwarp();
        pair::cluster_sync();
    } else if (warp < 8) {
        pair::more_registers<168>();
        // ---- P: warpgroup wg takes the tiles with g % 2 == wg; a thread is a row
        const int wg = warp >> 2, row = tid & 127, wq = warp & 3;
        const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
        const float sc = softmax_scale(a.scale);
        const int tok = row / a.group, head_in_group = row - tok * a.group;
        const uint32_t p_bars = pair::map_to(bar(Bar::PFull), 0);
        uint32_t g0 = 0;              // tiles before this block's
        uint32_t others = 0;          // per block slot, phase of LOther: blocks of two tiles or more
        Block b;
        for (int it = 0; fetch(it, b); ++it) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(Bar::Read + (it & 3)));
            const int n = b.n, mine = b.first + (int)rank * per_cta;
            const int token = mine + tok;  // in the sequence
            float m_own = -CUDART_INF_F, l = 0.f;
            for (int j = (g0 ^ wg) & 1; j < n; j += 2) {
                const uint32_t g = g0 + j, st = g % S;
                if (!wait(Bar::SFull + st, g / S)) break;
                tc_fence_after_sync();
                const uint32_t s_at = lanes + Sh::COLS_S + st * kTile;
                uint32_t r[128];
#pragma unroll
                for (int c = 0; c < 128; c += 32) pair::tmem_load32_start(s_at + c, r + c);
                pair::tmem_load_wait(r);
                if (j * kTile + kTile - 1 > mine) {  // some row of this CTA sees only part of the tile
                    const int seen = token - j * kTile;  // columns 0 .. seen
#pragma unroll
                    for (int c0 = 0; c0 < 128; c0 += 32) {
                        const int last = seen - c0;
                        const uint32_t sees = last < 0 ? 0u : last >= 31 ? ~0u : (2u << last) - 1u;
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (!(sees & (1u << c))) r[c0 + c] = 0xFF800000u;
                    }
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
                // the reference after the tile before, from the other warpgroup; its place is
                // written again only after this wait, also between two blocks' tiles
                if (g > 0 && !wait(Bar::MReady + wq, g - 1)) break;
                const float m_prev = j > 0 ? s_m[row] : -CUDART_INF_F;
                const bool raise = j == 0 || x_top > m_prev + Reference<F16>::TOP;
                const float m = raise ? x_top - Reference<F16>::LEAD : m_prev;
                s_m[row] = m;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(Bar::MReady + wq));

                if (j > 0 && __any_sync(0xffffffffu, raise)) {
                    // O is that of tiles 0 .. j - 1 then: P V of tile j waits for this warp's P.  (S of
                    // tile g is complete, so P V of tile g - 3 is: this barrier's phase is unambiguous.)
                    if (!wait(Bar::PvDone + ((g - 1) & 1), (g - 1) >> 1)) break;
                    tc_fence_after_sync();
                    const float f = raise ? fast_exp2(m_prev - m) : 1.f;
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t o[16];
                        pair::tmem_load16(lanes + c, o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        pair::tmem_store16(lanes + c, o);
                    }
                }
                l *= m_own == m ? 1.f : fast_exp2(m_own - m);
                m_own = m;
                uint64_t sum[2] = {0, 0};
                const float ref = m == -CUDART_INF_F ? 0.f : m;  // no finite score yet: p = 2^-inf
                const uint64_t sc2 = pair::pack_f32x2(sc, sc), m2 = pair::pack_f32x2(-ref, -ref);
#pragma unroll
                for (int quarter = 0; quarter < 4; ++quarter) {
                    uint32_t p[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const int i = quarter * 32 + 2 * c;
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
                    pair::tmem_store16(s_at + quarter * 16, p);
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

                const int slot = it & 1;
                if (j == n - 2) {  // the other warpgroup has the last tile
                    s_l[slot * 128 + row] = l;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(Bar::LOther + slot));
                } else if (j == n - 1) {
                    if (n > 1) {  // the other sum is relative to its last tile's m, handed on to this one
                        if (!wait(Bar::LOther + slot, others >> slot)) break;
                        l += s_l[slot * 128 + row] * (m_prev == m ? 1.f : fast_exp2(m_prev - m));
                    }
                    // the place of 1 / l: read for the block before last
                    if (it >= 2 && !wait(Bar::Read + ((it - 2) & 3), (it - 2) >> 2)) break;
                    s_inv[slot * 128 + row] = inverse_sum(l);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(Bar::Inv + slot));
                    if (a.lse && tok < per_cta && token < b.len)
                        a.lse[(b.t0 + token) * a.h_q + b.h * a.group + head_in_group] = kLn2 * (m + log2f(l));
                }
            }
            if (!ok) break;
            g0 += n;
            if (n > 1) others ^= 1u << (it & 1);
        }
        if (!ok) gave_up();
        __syncwarp();
        pair::cluster_sync();
    } else {
        pair::fewer_registers<120>();
        // ---- o = O / l; a thread is a row
        const int row = tid & 127;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const int tok = row / a.group, head_in_group = row - tok * a.group;
        const uint32_t o_free = pair::map_to(bar(Bar::OFree), 0);
        Block b;
        for (int it = 0; fetch(it, b); ++it) {
            const int token = b.first + (int)rank * per_cta + tok;
            const bool live = tok < per_cta && token < b.len;
            uint16_t *dst = live ? a.o.p + (b.t0 + token) * a.o.ts + (int64_t)(b.h * a.group + head_in_group) * a.o.hs
                                 : nullptr;
            if (!wait(Bar::Inv + (it & 1), it >> 1)) break;
            const float inv = s_inv[(it & 1) * 128 + row];
            if (!wait(Bar::Patch + (it & 3), it >> 2)) break;
            volatile uint32_t *const flags = s_flags + (it & 3) * 2;
            const bool patch = flags[0] | flags[1];
            __syncwarp();
            if (!wait(Bar::ODone, it)) break;
            tc_fence_after_sync();
            // Four lanes write a row's 64 bytes together, eight rows an instruction: a lane storing
            // its own row touches 32 lines an instruction, which held O for 4400 clocks a block.
            uint16_t *quad[4];  // rows of this lane's four, at this lane's 8 columns
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                quad[e] = reinterpret_cast<uint16_t *>(
                    __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(dst), (lane & ~3) | e));
                if (quad[e]) quad[e] += (lane & 3) * 8;
            }
            // 32 columns at a time: 128 of a row in registers hold O for less long, but their code crowds the
            // instruction cache (20 prompts of 500 tokens, d = 128: 54 against 51 us; 8 of 3600: 583 against 590).
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t w[16];
                {
                    uint32_t o[32];
                    pair::tmem_load32(lanes + c, o);
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        w[e / 2] = pack2<F16>(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv);
                }
                if (c + 32 == D) {  // this warp has read its part of O
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        pair::arrive_remote(o_free);
                        mbar_arrive(bar(Bar::Read + (it & 3)));
                    }
                    __syncwarp();
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {  // 16-byte pieces transposed among four lanes
#pragma unroll
                    for (int p = 0; p < 4; p += 2) {
                        uint32_t &x = w[p * 4 + e], &y = w[p * 4 + 4 + e];
                        const uint32_t z = __shfl_xor_sync(0xffffffffu, (lane & 1) ? x : y, 1);
                        ((lane & 1) ? x : y) = z;
                    }
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        uint32_t &x = w[p * 4 + e], &y = w[p * 4 + 8 + e];
                        const uint32_t z = __shfl_xor_sync(0xffffffffu, (lane & 2) ? x : y, 2);
                        ((lane & 2) ? x : y) = z;
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (quad[e])
                        *reinterpret_cast<uint4 *>(quad[e] + c) =
                            make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
            }
            __syncwarp();
            // what the looked-through tiles' infinities and NaNs add to the rows that see them, in the
            // stored row: a rare path, kept small (the roles' code has to fit the instruction cache)
            if (live && patch) {
#pragma unroll 1
                for (int p = b.j_clean * kTile; p <= token; ++p) {
                    const uint16_t *const v = a.v.p + (b.t0 + p) * a.v.ts + (int64_t)b.h * a.v.hs;
#pragma unroll 1
                    for (int c = 0; c < D; ++c) {
                        const float x = unpack1<F16>(v[c]);
                        if (!isfinite(x)) dst[c] = (uint16_t)pack2<F16>(unpack1<F16>(dst[c]) + x, 0.f);
                    }
                }
            }
            __syncwarp();
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

static cudaError_t launch_long(const Args &a, cudaStream_t s) {
    if (a.d == 64) return a.f16 ? launch<64, true>(a, s) : launch<64, false>(a, s);
    if (a.d == 128) return a.f16 ? launch<128, true>(a, s) : launch<128, false>(a, s);
    return a.f16 ? launch<256, true>(a, s) : launch<256, false>(a, s);
}

cudaError_t launch_prefill(const Args &a, cudaStream_t s) {
    // The lengths are on the device; the totals say when one of the kernels has nothing to do.
    const bool some_long = a.t_total > short_tokens(a.group), some_short = !some_long || a.n_seqs > 1;
    if (some_long) {
        const cudaError_t e = launch_long(a, s);
        if (e != cudaSuccess) return e;
    }
    return some_short ? launch_prefill_short(a, some_long, s) : cudaSuccess;
}

}  // namespace attn
}  // namespace gdr
