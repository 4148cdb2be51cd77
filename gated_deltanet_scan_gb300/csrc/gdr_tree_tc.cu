// The gated delta rule over trees of drafted tokens, bf16 inputs, on tcgen05 tensor cores.
//
// Formulas: gdr_tree_rule.cuh, with the corrections solved for: the unit triangular I + N, whose
// row j has entries at j's ancestors only, has an inverse T with entries at the same places, so
//     u_j = sum_{i in A_j} T_ji R_i,   o_j = e^{G_j} S_0^T q_j + sum_{i in A_j} W_ji R_i,   W = P T,
// R_j = beta_j (v_j - e^{G_j} S_0^T k_j).  T and W need no state; the rest is two products that
// a state's columns enter, both on the tensor cores.
//
// One block of 1024 threads an SM walks consecutive (sequence, V head) pairs:
//
//   gates    (warp 31) the tree, and the sums of the gates along its paths, a pair or two ahead of
//   factors  (warps 24 .. 29) K and Q of a QK head by cp.async into the operand layout; the Gram
//            products [K; Q] K^T, of which the paths' are kept; N and P of every ancestor; T and W, for
//            two V heads of a QK head at once (where they fit), since the steps are chains of loads; then,
//            pair by pair, the bf16 parts of T - I and W into an operand tile.  T comes by doubling: blocks
//            of b = 1, 2, 4, ... levels of the paths are inverted; joining an even block and the odd one
//            under it, T_ti = -sum_s T_ts Y_si with Y_si = sum_j N_sj T_ji, s in the odd block and j in the
//            even one, so a path of 64 takes six rounds of two steps (level by level it takes 63).
//   states   (warps 16 .. 23) a thread has half a column of the state, from a ring of 16 rows a stage that
//            bulk copies fill (loads into registers held 4,000 clocks up at 64 nodes: an SM has some
//            32 KB of them on their way); it splits each value exactly into three bf16 parts and stores
//            them at its lane of TMEM: X^T = S_0^T [K; Q]^T has M = d columns, N = 2 n nodes and inner
//            size d, and the state is the operand that lives in TMEM
//   rows     (warps 0 .. 15) R and e^G S_0^T q are made from X in place, and [U; O]^T is what they are
//            plus R^T [T - I; W]^T, inner size n, R's parts in TMEM too.  Neither the state nor R passes
//            through shared memory.  Of the nine products of parts six are made, smallest first: cutting leaves
//            a middle part under 2^-7 and a low one under 2^-15 of the value, so the three that are left out are
//            together under 2^-21 of a product.  What the accumulators cut after every 16 products weighs more:
//            o and u are 1.5 to 3.9 * 10^-7 of their norm off 64 bits.
//   MMAs     (warp 30) both products: an issuing thread stands still while the tensor pipe is full.
//
// Bound by the chain X, R, U and O of a pair, 9,500 clocks at 64 nodes, and as long by the factors' of two
// heads (18,000); everything else is done while the pairs before go through it, and HBM would need 5,600. 64
// trees of 64 nodes with 32 heads: 96 us; their 336 MB (294 of it DRAM traffic, the rest is still in L2 when
// the kernel ends) would take 49.6, so 52% of the measured bandwidth (an fp32 kernel level by level took 2,222).
// 8 of 41 nodes 20.8 us (4.6), one of 24 12.4 (0.5): there the first
// pair of a block takes 15,000 to 25,000 clocks, a quarter of them instructions that come from memory.
//
// A node's rows of T and W are zero but at its ancestors, and zero times an infinity or NaN would
// reach it: such values of R (rare) enter the product as zeros and are added afterwards to the
// nodes whose path they are on.
//
// Every role's code runs once a pair or two, and the first pair waits for all of it to come from
// memory: it is kept small, in loops where registers allow.
//
// Deep paths cost more: the joins and W are sums over lists in shared memory, cubic in a path's length, and a
// pair of more than half of all possible entries goes through them alone. 64 chains of 64: 438 us, 16 of them 133,
// one 44; 64 chains of 32 105, of 24 87.
//
// d < 128 leaves lanes (and warps) idle, and the factors, which then bound it, as they are: 64 trees of 64 nodes
// take 87 us at d = 64 (floor 20), 82 at d = 32 (8.8), one of 24 12.3 at either.
#include "gdr_attn.h"
#include "gdr_attn_mma.cuh"
#include "gdr_attn_ptx.cuh"
#include "gdr_tree_rule.cuh"
#include "tc_ptx.cuh"

namespace gdr {
namespace {

using namespace tc;

constexpr int NT = 1024;
constexpr int kRows = 512, kStates = 256, kFactors = 192;  // threads of these roles, in this order
constexpr int kShares = kRows / 128;                       // threads of a column
constexpr int kNodes = tree::kMaxNodes;
constexpr int kEntries = kNodes * (kNodes + 1) / 2;  // of the paths' lists: ancestors, and the node itself last
constexpr int kSecondHead = kEntries / 2;            // where a second V head's are, if it fits
constexpr int kStageRows = 16;  // of the state's rings, one for either half of its warps
__host__ __device__ constexpr int ring_slots(int half) { return half == 0 ? 3 : 2; }
constexpr int kSlots = ring_slots(0) + ring_slots(1);
constexpr int kJoins = 6;  // of blocks of 1, 2, ..., 32 levels
constexpr int kGrid = 152;

struct Shape {
    static constexpr uint32_t BLOCK = 128 * 128;          // 128 rows of 64 values
    static constexpr uint32_t KQ = 2 * BLOCK;             // rows [0, r) K, [r, 2 r) Q, r = n rounded up to 16; two of them
    static constexpr uint32_t OFF_B = 2 * KQ;             // three parts of [T; W], rows likewise
    static constexpr uint32_t OFF_NP = OFF_B + 3 * BLOCK;       // N and P, float2 an entry
    static constexpr uint32_t OFF_T = OFF_NP + kEntries * 8;     // T
    static constexpr uint32_t OFF_W = OFF_T + kEntries * 4;      // W
    static constexpr uint32_t OFF_ITEM = OFF_W + kEntries * 4;   // entries join by join, the nodes themselves last: struct Entry
    static constexpr uint32_t OFF_UP = OFF_ITEM + kEntries * 4;  // where the ancestor's own list starts, 16 bits an entry
    static constexpr uint32_t OFF_ANC = OFF_UP + kEntries * 2;   // the ancestor, 8 bits an entry
    static constexpr uint32_t OFF_V = OFF_ANC + kEntries;        // [n][d]
    static constexpr uint32_t STAGE = kStageRows * 128 * 4;
    static constexpr uint32_t OFF_S = OFF_V + kNodes * 128 * 2;
    static constexpr uint32_t BYTES = OFF_S + kSlots * STAGE;
    static_assert(OFF_V % 16 == 0 && OFF_S % 16 == 0, "bulk copies");
    // TMEM columns: the state's parts, X (then U and O), the Gram products, R's parts
    static constexpr uint32_t A = 0, X = 192, GRAM = 320, RP = 384;
};
// What a role reports without waiting for who waits for it has a barrier for each of some buffers, so that
// no phase is passed over.
enum Bar {
    kTables = 0,    // [2] gates -> factors
    kKqFull = 2,    // [2] factors -> MMAs
    kGateFull = 4,  // [4] factors -> rows
    kTabFree = 8,   // [2] factors -> gates
    kBFull = 10,    // factors -> MMAs
    kBFree,         // MMAs (or rows) -> factors
    kGram,          // a commit -> factors
    kParts,         // states -> MMAs
    kFirst,         // a commit -> rows, states
    kRParts,        // rows -> MMAs, states
    kSecond,        // a commit -> rows
    kXFree,         // rows -> MMAs
    kVFull,         // states (their copies) -> rows
    kSFull,         // [kSlots] copies -> states
    kBars = kSFull + kSlots
};

// The gates run ahead of the factors, these of the rows: trees and gates have four buffers.
struct Tables {
    uint64_t mask[4][kNodes];
    uint64_t real[4];          // the rows that are nodes
    uint64_t plane[4][kJoins];  // those whose level (number of ancestors) has bit k
    uint16_t start[4][kNodes];  // where a node's list starts
    int entries[4], deepest[4];  // of all lists; ancestors of the deepest node
    float2 sum[2][kNodes];  // G as two floats
    float grown[2][kNodes], beta[2][kNodes], rk[kNodes], rq[kNodes];  // 1 / |k|, 1 / |q|
    float4 gate[4][kNodes];  // beta, e^G / |k|, e^G / |q|, P_jj
    uint32_t tmem, odd;
    uint64_t bar[kBars];
};

// Columns of this thread's lane loaded (complete after pair::tmem_load_wait) and stored (after
// pair::tmem_store_wait).
__device__ __forceinline__ void tmem_load16_start(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_load1_start(uint32_t taddr, uint32_t &r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_store1(uint32_t taddr, uint32_t r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(r) : "memory");
}
__device__ __forceinline__ void tmem_store8(uint32_t taddr, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
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
__device__ __forceinline__ bool is_odd(uint32_t x) { return (x & 0x7F800000u) == 0x7F800000u; }  // infinite or NaN

// An entry of a path's list, packed: its place, the node, the ancestor's level and the node's.
struct Entry {
    int e, t, r, d;
    __device__ __forceinline__ explicit Entry(uint32_t p) : e(p & 4095), t(p >> 12 & 63), r(p >> 18 & 63), d(p >> 24) {}
    static __device__ __forceinline__ uint32_t pack(int e, int t, int r, int d) {
        return (uint32_t)(e | t << 12 | r << 18 | d << 24);
    }
};

// A pair, and what the factors share with the pair before.
struct Item {
    int seq, h, hq;
    bool new_tree, new_kq;
};
struct Items {
    int at, end, seq, hq;
    __device__ __forceinline__ explicit Items(const Args &a) : seq(-1), hq(-1) {
        const int total = a.n_seqs * a.h_v, each = total / gridDim.x, rest = total % gridDim.x;
        at = blockIdx.x * each + min((int)blockIdx.x, rest);
        end = at + each + ((int)blockIdx.x < rest ? 1 : 0);
    }
    __device__ __forceinline__ Item next(const Args &a) {
        Item it;
        it.seq = at / a.h_v;
        it.h = at - it.seq * a.h_v;
        it.hq = it.h / (a.h_v / a.h_qk);
        it.new_tree = it.seq != seq;
        it.new_kq = it.new_tree || it.hq != hq;
        seq = it.seq;
        hq = it.hq;
        ++at;
        return it;
    }
};

__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, pair::wait_bounded(bar, parity & 1));
}

// ---- the gates' warp -----------------------------------------------------------------------------
__device__ __forceinline__ bool gates(const Args &a, int32_t *err, Tables &s) {
    const int lane = threadIdx.x & 31, n = a.fixed_len;
    auto bar = [&](int i) { return smem_u32(s.bar + i); };
    int trees = -1;
    Items items(a);
    int2 parents;
    float g[2], b[2];
    auto load = [&](const Item &it) {
        const int64_t row0 = (int64_t)it.seq * n;
        parents = tree::load_parents(a.parents + row0, n, lane);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int j = lane + 32 * x;
            g[x] = j < n ? a.g[(row0 + j) * a.h_v + it.h] : 0.f;
            b[x] = j < n ? a.beta[(row0 + j) * a.h_v + it.h] : 0.f;
        }
    };
    Item it = items.next(a);
    load(it);  // before anything else of the block
    __syncthreads();
#pragma unroll 1
    for (int i = 0;; ++i) {
        // the buffers are free once the factors have used them two pairs ago
        if (i >= 2 && !wait_warp(bar(kTabFree + (i & 1)), i - 2 >> 1)) return false;
        // masks and sums of the gates along the paths; sums in doubles, since their differences enter exponentials
        double sum[2] = {tree::gate(g[0]), tree::gate(g[1])};
        const tree::Masks m = tree::masks<true>(parents, n, lane, sum);
        if (it.new_tree) {
            const int z = ++trees & 3;
            if (m.bad) atomicCAS(err, 0, (int32_t)GDR_ERR_INVALID_ARG);
            const uint32_t real[2] = {__ballot_sync(0xffffffffu, m.a[0] != 0), __ballot_sync(0xffffffffu, m.a[1] != 0)};
            int length[2], at = 0;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                s.mask[z][lane + 32 * x] = m.a[x];
                length[x] = __popcll(m.a[x]);
                int upto = length[x];
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, upto, d);
                    if (lane >= d) upto += y;
                }
                s.start[z][lane + 32 * x] = (uint16_t)(at + upto - length[x]);
                at += __shfl_sync(0xffffffffu, upto, 31);
            }
            const int longest = __reduce_max_sync(0xffffffffu, max(length[0], length[1]));
#pragma unroll 1
            for (int k = 0; k < kJoins; ++k) {
                const uint32_t p0 = __ballot_sync(0xffffffffu, length[0] > 0 && (length[0] - 1 >> k & 1));
                const uint32_t p1 = __ballot_sync(0xffffffffu, length[1] > 0 && (length[1] - 1 >> k & 1));
                if (lane == 0) s.plane[z][k] = (uint64_t)p1 << 32 | p0;
            }
            if (lane == 0) {
                s.entries[z] = at;
                s.deepest[z] = longest - 1;
                s.real[z] = (uint64_t)real[1] << 32 | real[0];
            }
        }
#pragma unroll 1
        for (int x = 0; 32 * x < n; ++x) {
            const int j = lane + 32 * x;
            const double y = x ? sum[1] : sum[0];
            const float hi = (float)y, lo = (float)(y - (double)hi), logit = x ? b[1] : b[0];
            s.sum[i & 1][j] = make_float2(hi, lo);
            s.grown[i & 1][j] = expf(hi) * (1.f + lo);
            s.beta[i & 1][j] = a.beta_logits ? 1.f / (1.f + expf(-logit)) : logit;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kTables + (i & 1)));
        if (items.at == items.end) return true;
        it = items.next(a);
        load(it);
    }
}

// ---- the factors' warps --------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ bool factors(const Args &a, uint8_t *smem, Tables &s) {
    using Sh = Shape;
    constexpr uint32_t ID = 2;
    constexpr int N = kFactors;
    float2 *const s_np = reinterpret_cast<float2 *>(smem + Sh::OFF_NP);
    float *const s_t = reinterpret_cast<float *>(smem + Sh::OFF_T), *const s_w = reinterpret_cast<float *>(smem + Sh::OFF_W);
    uint32_t *const s_item = reinterpret_cast<uint32_t *>(smem + Sh::OFF_ITEM);
    uint16_t *const s_up = reinterpret_cast<uint16_t *>(smem + Sh::OFF_UP);
    uint8_t *const s_anc = smem + Sh::OFF_ANC;
    uint8_t *const parts = smem + Sh::OFF_B;
    const uint32_t base = smem_u32(smem);
    const int tid = threadIdx.x - kRows - kStates;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int n = a.fixed_len, nr = (n + 15) & ~15;
    auto bar = [&](int i) { return smem_u32(s.bar + i); };
    auto wait_all = [&](int i, uint32_t parity) { return !pair::named_or(ID, N, !pair::wait_bounded(bar(i), parity & 1)); };
    auto load_kq = [&](const Item &it, int kq) {
        constexpr int CPR = D / 8, RPI = N / CPR;  // 16-byte chunks of a row, rows at a time
        const int c = tid % CPR;
        const int64_t row0 = (int64_t)it.seq * n, step = (int64_t)a.h_qk * D, first = (row0 * a.h_qk + it.hq) * D + c * 8;
        const uint32_t dst = base + kq * Sh::KQ + (c >> 3) * Sh::BLOCK;
#pragma unroll 1
        for (int t = tid / CPR; t < n; t += RPI) {
            attn::cp_async16(dst + sw128_offset(t, c & 7), static_cast<const uint16_t *>(a.k) + first + t * step, 16u);
            attn::cp_async16(dst + sw128_offset(nr + t, c & 7), static_cast<const uint16_t *>(a.q) + first + t * step, 16u);
        }
        attn::cp_async_commit();
    };
    int kq = 0, trees = -1, grams = -1, entries = 0, deepest = 0;
    Items items(a);
    Item next = items.next(a);
    load_kq(next, 0);
    __syncthreads();
    tc_fence_after_sync();
#pragma unroll 1
    for (int i = 0;;) {
        const Item it = next;
        bool more = items.at < items.end;
        if (more) next = items.next(a);
        if (it.new_tree) ++trees;
        const int z = trees & 3;
        uint8_t *const tile = smem + kq * Sh::KQ;
        if (it.new_kq) {
            attn::cp_async_wait<0>();
            fence_proxy_async_smem();
            tc_fence_before_sync();
            named_sync(ID, N);
        }
        // -- the Gram products, before what the MMAs' warp makes of K and Q; then |q| and the paths' lists
        ++grams;
        if (warp == 4) {
            tc_fence_after_sync();
            if (elect_one()) {
                const uint64_t at = smem_desc_sw128(base + kq * Sh::KQ, 0, 1024);
                const uint32_t id = idesc_bf16_f32(128, nr, 0, 0);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t x = at + (((k >> 2) * Sh::BLOCK + (k & 3) * 32) >> 4);
                    mma_bf16(s.tmem + Sh::GRAM, x, x, id, k > 0);
                }
                mma_commit(bar(kGram));
                if (it.new_kq) mbar_arrive(bar(kKqFull + kq));
            }
            __syncwarp();
        }
        if (!wait_all(kTables + (i & 1), i >> 1)) return false;
        if (it.new_tree) {
            entries = s.entries[z];
            deepest = s.deepest[z];
        }
        const bool two = more && !next.new_kq && entries <= kSecondHead;  // another V head of the QK head
        if (two) {
            if (!wait_all(kTables + (i + 1 & 1), i + 1 >> 1)) return false;
            more = items.at < items.end;
            if (more) next = items.next(a);
        }
        {
            if (it.new_tree && tid < n && s.mask[z][tid]) {
                const uint64_t mask = s.mask[z][tid], below = (1ull << tid) - 1;
                const int d = __popcll(mask) - 1, at = s.start[z][tid];
                int r = 0, from = 0;
#pragma unroll 1
                for (uint64_t up = mask; up; ++r, up &= up - 1) {
                    const int j = __ffsll((long long)up) - 1;
                    s_up[at + r] = s.start[z][j];
                    s_anc[at + r] = (uint8_t)j;
                }
                // a node of level d has b entries in the join of blocks of b levels where d has bit b
#pragma unroll 1
                for (int k = 0; k < kJoins; ++k) {
                    const uint64_t plane = s.plane[z][k];
                    const int b = 1 << k, to = from + __popcll(plane & below) * b, r0 = d & -2 * b;
                    if (d & b) {
#pragma unroll 1
                        for (int x = 0; x < b; ++x) s_item[to + x] = Entry::pack(at + r0 + x, tid, r0 + x, d);
                    }
                    from += __popcll(plane) * b;
                }
                s_item[from + __popcll(s.real[z] & below)] = Entry::pack(at + d, tid, d, d);
            }
            if (a.qk_norm && it.new_kq) {  // four lanes a row
#pragma unroll 1
                for (int r = tid >> 2; r < ((n + 7) & ~7); r += N / 4) {  // whole warps
                    float sq = 0.f;
#pragma unroll
                    for (int c0 = 0; c0 < D / 8; c0 += 4) {
                        const int c = c0 + (tid & 3);
                        const uint4 w = *reinterpret_cast<const uint4 *>(tile + (c >> 3) * Sh::BLOCK +
                                                                         sw128_offset(nr + r, c & 7));
                        const uint32_t y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const float lo = __uint_as_float(y[x] << 16), hi = __uint_as_float(y[x] & 0xFFFF0000u);
                            sq = fmaf(lo, lo, fmaf(hi, hi, sq));
                        }
                    }
                    sq += __shfl_xor_sync(0xffffffffu, sq, 1);
                    sq += __shfl_xor_sync(0xffffffffu, sq, 2);
                    if ((tid & 3) == 0 && r < n) s.rq[r] = l2norm_scale(sq);
                }
            } else if (!a.qk_norm && tid < n) {
                s.rq[tid] = 1.f;
            }
            if (!wait_all(kGram, grams)) return false;
            tc_fence_after_sync();
            if (warp < 4) {  // a row of K or Q per lane: what is on its node's path
                const int row = tid < nr ? tid : tid - nr;
                const bool is_k = tid < nr;
                const uint64_t mask = row < n && tid < 2 * nr ? s.mask[z][row] : 0;
                float *to = reinterpret_cast<float *>(s_np + (mask ? s.start[z][row] : 0)) + (is_k ? 0 : 1);
#pragma unroll 1
                for (int c = 0; c < nr; c += 16) {
                    uint32_t y[16];
                    pair::tmem_load16(s.tmem + ((uint32_t)(warp * 32) << 16) + Sh::GRAM + c, y);
                    const uint32_t bits = (uint32_t)(mask >> c);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        if (bits >> k & 1) {
                            *to = __uint_as_float(y[k]);
                            to += 2;
                        }
                    }
                }
                tc_fence_before_sync();
            }
            named_sync(ID, N);
        }
        // -- N and P, and the nodes' own factors
        const int i1 = i + 1;
        if (tid < 2 * kNodes) {
            const int j = tid & 63, x = tid >> 6, b = i + x & 1;
            float4 gate = make_float4(0.f, 0.f, 0.f, 0.f);
            if (s.real[z] >> j & 1) {
                const float2 own = s_np[s.start[z][j] + __popcll(s.mask[z][j]) - 1];
                const float rk = a.qk_norm ? l2norm_scale(own.x) : 1.f, grown = s.grown[b][j];
                gate = make_float4(s.beta[b][j], grown * rk, grown * s.rq[j], s.rq[j] * rk * own.y);
                if (x == 0) s.rk[j] = rk;
            }
            if (x == 0 || two) s.gate[i + x & 3][j] = gate;
        }
        named_sync(ID, N);
        if (tid == 0) {
            mbar_arrive(bar(kGateFull + (i & 3)));
            if (two) mbar_arrive(bar(kGateFull + (i1 & 3)));
        }
#pragma unroll 1
        for (int x = tid; x < entries; x += N) {
            const Entry it(s_item[x]);
            const int e = it.e, t = it.t, j = s_anc[e];
            const float2 raw = s_np[e];
            const float kk = s.rk[t] * s.rk[j] * raw.x, qk = s.rq[t] * s.rk[j] * raw.y;
            {
                const float y = tree::decay(s.sum[i & 1][t], s.sum[i & 1][j]), nji = s.beta[i & 1][t] * y * kk;
                s_np[e] = make_float2(nji, y * qk);
                s_t[e] = -nji;  // T of blocks of two levels
            }
            if (two) {
                const float y = tree::decay(s.sum[i1 & 1][t], s.sum[i1 & 1][j]), nji = s.beta[i1 & 1][t] * y * kk;
                s_np[e + kSecondHead] = make_float2(nji, y * qk);
                s_t[e + kSecondHead] = -nji;
            }
        }
        named_sync(ID, N);
        if (tid == 0) {
            mbar_arrive(bar(kTabFree + (i & 1)));
            if (two) mbar_arrive(bar(kTabFree + (i1 & 1)));
        }
        // -- T, joining blocks of b levels: entry (t, j), t in an odd block and j in the even one above it
#pragma unroll 1
        for (int k = 1, x0 = __popcll(s.plane[z][0]), x1; 1 << k <= deepest; ++k, x0 = x1) {
            const int b = 1 << k;
            x1 = x0 + __popcll(s.plane[z][k]) * b;
            // Y = N + N T, over the rest of the even block; it lies where W will
#pragma unroll 1
            for (int x = x0 + tid; x < x1; x += N) {
                const Entry it(s_item[x]);
                const int at = it.e - it.r, end = (it.r | b - 1) + 1;
                float m0 = s_np[it.e].x, m1 = two ? s_np[it.e + kSecondHead].x : 0.f;
#pragma unroll 4
                for (int y = it.r + 1; y < end; ++y) {
                    const int up = s_up[at + y] + it.r;
                    m0 = fmaf(s_np[at + y].x, s_t[up], m0);
                    if (two) m1 = fmaf(s_np[at + y + kSecondHead].x, s_t[up + kSecondHead], m1);
                }
                s_w[it.e] = m0;
                if (two) s_w[it.e + kSecondHead] = m1;
            }
            named_sync(ID, N);
            // T = -(Y + T Y), over the odd block's levels before
#pragma unroll 1
            for (int x = x0 + tid; x < x1; x += N) {
                const Entry it(s_item[x]);
                const int at = it.e - it.r;
                float m0 = s_w[it.e], m1 = two ? s_w[it.e + kSecondHead] : 0.f;
#pragma unroll 4
                for (int y = it.d & -b; y < it.d; ++y) {
                    const int up = s_up[at + y] + it.r;
                    m0 = fmaf(s_t[at + y], s_w[up], m0);
                    if (two) m1 = fmaf(s_t[at + y + kSecondHead], s_w[up + kSecondHead], m1);
                }
                s_t[it.e] = -m0;
                if (two) s_t[it.e + kSecondHead] = -m1;
            }
            named_sync(ID, N);
        }
        // -- W = P T; at the node itself, where T - I is 0, its P
#pragma unroll 1
        for (int x = tid; x < entries; x += N) {
            const Entry it(s_item[x]);
            const int at = it.e - it.r;
            const float p0 = s.gate[i & 3][it.t].w, p1 = s.gate[i1 & 3][it.t].w;
            float w0 = p0, w1 = p1, y0 = 0.f, y1 = 0.f;
            if (it.r < it.d) {
                y0 = s_t[it.e];
                w0 = fmaf(p0, y0, s_np[it.e].y);
                if (two) {
                    y1 = s_t[it.e + kSecondHead];
                    w1 = fmaf(p1, y1, s_np[it.e + kSecondHead].y);
                }
#pragma unroll 4
                for (int y = it.r + 1; y < it.d; ++y) {
                    const int up = s_up[at + y] + it.r;
                    w0 = fmaf(s_np[at + y].y, s_t[up], w0);
                    if (two) w1 = fmaf(s_np[at + y + kSecondHead].y, s_t[up + kSecondHead], w1);
                }
            }
            s_w[it.e] = w0;
            s_t[it.e] = y0;
            if (two) {
                s_w[it.e + kSecondHead] = w1;
                s_t[it.e + kSecondHead] = y1;
            }
        }
        named_sync(ID, N);
        // -- pair by pair, their parts, once the pair before is done with its own (and so with K and Q before
        // this one's)
#pragma unroll 1
        for (const int last = i + (two ? 1 : 0); i <= last; ++i) {
            const bool first = i < last || !two;
            const int from = first ? 0 : kSecondHead;
            if (i > 0 && !wait_all(kBFree, i - 1)) return false;
            if (first && more && next.new_kq) load_kq(next, kq ^ 1);
            if (first && it.new_tree) {  // the places of another tree's entries
#pragma unroll 1
                for (int x = tid; x < 3 * (int)Sh::BLOCK / 16; x += N)
                    reinterpret_cast<uint4 *>(parts)[x] = make_uint4(0u, 0u, 0u, 0u);
                named_sync(ID, N);
            }
#pragma unroll 1
            for (int x = tid; x < entries; x += N) {  // T and W at the ancestors, W at the node itself
                const Entry it(s_item[x]);
                const int t = it.t, j = s_anc[it.e];
                const float2 f = make_float2(s_t[it.e + from], s_w[it.e + from]);
                uint32_t part[3];
                split3(f.x, f.y, part[0], part[1], part[2]);
                uint8_t *const at = parts + sw128_offset(t, j >> 3) + (j & 7) * 2;
                uint8_t *const aw = parts + sw128_offset(nr + t, j >> 3) + (j & 7) * 2;
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    *reinterpret_cast<uint16_t *>(at + p * Sh::BLOCK) = (uint16_t)part[p];
                    *reinterpret_cast<uint16_t *>(aw + p * Sh::BLOCK) = (uint16_t)(part[p] >> 16);
                }
            }
            fence_proxy_async_smem();
            named_sync(ID, N);
            if (tid == 0) mbar_arrive(bar(kBFull));
        }
        if (!more) break;
        if (next.new_kq) kq ^= 1;
    }
    return true;
}

// ---- the MMAs' warp --------------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ bool products(const Args &a, uint8_t *smem, Tables &s) {
    using Sh = Shape;
    const bool issue = elect_one();
    const int nr = (a.fixed_len + 15) & ~15;
    const uint32_t base = smem_u32(smem);
    auto bar = [&](int i) { return smem_u32(s.bar + i); };
    const uint32_t id = idesc_bf16_f32(128, 2 * nr, 0, 0);
    const uint64_t d_b = smem_desc_sw128(base + Sh::OFF_B, 0, 1024);
    int loads = -1;
    Items items(a);
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = s.tmem;
#pragma unroll 1
    for (int i = 0; items.at < items.end; ++i) {
        const Item it = items.next(a);
        if (it.new_kq) {
            ++loads;
            if (!wait_warp(bar(kKqFull + (loads & 1)), loads >> 1)) return false;
        }
        if (!wait_warp(bar(kParts), i) || (i > 0 && !wait_warp(bar(kXFree), i - 1))) return false;
        tc_fence_after_sync();
        if (issue) {
            const uint64_t d_kq = smem_desc_sw128(base + (loads & 1) * Sh::KQ, 0, 1024);
#pragma unroll 1
            for (int p = 0; p < 3; ++p) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    pair::mma_ts_one(tmem + Sh::X, tmem + Sh::A + p * (D / 2) + k * 8,
                                     d_kq + (((k >> 2) * Sh::BLOCK + (k & 3) * 32) >> 4), id, p > 0 || k > 0);
            }
            mma_commit(bar(kFirst));
        }
        __syncwarp();
        if (!wait_warp(bar(kBFull), i) || !wait_warp(bar(kRParts), i)) return false;
        tc_fence_after_sync();
        if (issue) {
#pragma unroll 1
            for (int p = 0; p < 6; ++p) {
                // parts of R and of T, W: 2 0, 1 1, 0 2, 1 0, 0 1, 0 0
                const int r_part = 0x001012 >> (4 * p) & 15, t_part = 0x010210 >> (4 * p) & 15;
#pragma unroll
                for (int k = 0; k < kNodes / 16; ++k) {
                    if (k * 16 >= nr) break;
                    pair::mma_ts_one(tmem + Sh::X, tmem + Sh::RP + r_part * 32 + k * 8,
                                     d_b + ((t_part * Sh::BLOCK + k * 32) >> 4), id, 1);
                }
            }
            if (!*reinterpret_cast<volatile uint32_t *>(&s.odd)) mma_commit(bar(kBFree));
            mma_commit(bar(kSecond));
        }
        __syncwarp();
    }
    return true;
}

// ---- the states' warps -----------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ bool states(const Args &a, uint8_t *smem, Tables &s) {
    using Sh = Shape;
    constexpr int PER = D / kStageRows / 2;  // stages of a pair for each half of the warps: every other one
    constexpr uint32_t BYTES = kStageRows * D * 4;
    const int tid = threadIdx.x - kRows, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int col = tid & 127, half = warp >> 2;
    const bool work = col - lane < D;
    auto bar = [&](int i) { return smem_u32(s.bar + i); };
    const int first_slot = half * ring_slots(0), slots = half ? ring_slots(1) : ring_slots(0);
    uint8_t *const ring = smem + Sh::OFF_S + first_slot * Sh::STAGE;
    Items items(a);
    const int pairs = items.end - items.at, stages = pairs * PER;
    const float *const state = a.state + (int64_t)items.at * D * D;
    auto load = [&](int q) {  // this half's stage q of all
        if (q >= stages) return;
        const int slot = q % slots;
        mbar_arrive_expect_tx(bar(kSFull + first_slot + slot), BYTES);
        bulk_load(smem_u32(ring + slot * Sh::STAGE), state + ((int64_t)q * 2 + half) * kStageRows * D, BYTES,
                  bar(kSFull + first_slot + slot));
    };
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t lanes = s.tmem + ((uint32_t)((warp & 3) * 32) << 16);
    auto load_values = [&](int64_t pair) {
        constexpr int CPR = D / 8, RPI = kStates / CPR;  // 16-byte chunks of a row, rows at a time
        const int n = a.fixed_len, c = tid % CPR;
        const int64_t seq = pair / a.h_v, row = seq * n * a.h_v + (pair - seq * a.h_v);
        for (int t = tid / CPR; t < n; t += RPI)
            attn::cp_async16(smem_u32(smem + Sh::OFF_V) + (t * D + c * 8) * 2,
                             static_cast<const uint16_t *>(a.v) + (row + (int64_t)t * a.h_v) * D + c * 8, 16u);
        attn::cp_async_arrive(bar(kVFull));
    };
    if (col == 0) {
        for (int q = 0; q < slots; ++q) load(q);
    }
    __syncwarp();
    load_values(items.at);
    // A wait may give up for one warp and not for another: they leave at a vote, never between two.
    bool ok = true;
#pragma unroll 1
    for (int i = 0, q = 0; i < pairs; ++i) {
        ok = (i == 0 || wait_warp(bar(kFirst), i - 1)) && ok;
        tc_fence_after_sync();
#pragma unroll 1
        for (int k = 0; k < PER; ++k, ++q) {
            ok = ok && wait_warp(bar(kSFull + first_slot + q % slots), q / slots);
            const float *const x = reinterpret_cast<const float *>(ring + q % slots * Sh::STAGE) + col;
            float y[kStageRows];
            if (work) {
#pragma unroll
                for (int r = 0; r < kStageRows; ++r) y[r] = x[r * D];
            }
            if (pair::named_or(3 + half, kStates / 2, !ok)) return false;  // the stage is read
            if (col == 0) load(q + slots);
            __syncwarp();
            if (work) {
                uint32_t part[3][kStageRows / 2];
#pragma unroll
                for (int r = 0; r < kStageRows / 2; ++r) split3(y[2 * r], y[2 * r + 1], part[2][r], part[1][r], part[0][r]);
#pragma unroll
                for (int p = 0; p < 3; ++p)  // low first
                    tmem_store8(lanes + Sh::A + p * (D / 2) + (2 * k + half) * (kStageRows / 2), part[p]);
            }
        }
        pair::tmem_store_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kParts));
        // its values, once the rows are done with those of the pair before
        if (i > 0) {
            ok = wait_warp(bar(kRParts), i - 1) && ok;
            if (ok) load_values(items.at + i);
        }
    }
    attn::cp_async_wait<0>();
    return ok;
}

// ---- the rows' warps -------------------------------------------------------------------------------
template <int D, typename Out>
__device__ __forceinline__ bool rows(const Args &a, uint8_t *smem, Tables &s) {
    using Sh = Shape;
    constexpr uint32_t ID = 1;
    constexpr int KN = kNodes / kShares;  // a thread's nodes
    static_assert(KN == 16, "a thread's nodes are one TMEM load");
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int n = a.fixed_len, nr = (n + 15) & ~15;
    const int col = tid & 127, share = warp >> 2, t0 = share * KN;
    const bool work = col - lane < D;
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t lanes = s.tmem + ((uint32_t)((warp & 3) * 32) << 16);
    auto bar = [&](int i) { return smem_u32(s.bar + i); };
    const int64_t step = (int64_t)a.h_v * D;
    const uint16_t *const s_v = reinterpret_cast<const uint16_t *>(smem + Sh::OFF_V) + t0 * D + col;
    int trees = -1;
    bool ok = true;
    Items items(a);
    Item next = items.next(a);
#pragma unroll 1
    for (int i = 0;; ++i) {
        const Item it = next;
        const bool more = items.at < items.end;
        if (more) next = items.next(a);
        if (it.new_tree) ++trees;
        const int64_t out0 = ((int64_t)it.seq * n * a.h_v + it.h) * D + col;
        // -- R and its parts, and what they are added to
        ok = wait_warp(bar(kGateFull + (i & 3)), i >> 2) && ok;
        ok = wait_warp(bar(kVFull), i) && ok;
        ok = wait_warp(bar(kFirst), i) && ok;
        if (pair::named_or(ID, kRows, !ok)) return false;
        tc_fence_after_sync();
        float most = 0.f;
        if (work && t0 < nr) {
            const float4 *const s_gate = s.gate[i & 3] + t0;
            const uint32_t real = (uint32_t)(s.real[trees & 3] >> t0);
            uint32_t y[32], part[3][8];
            tmem_load16_start(lanes + Sh::X + t0, y);
            tmem_load16_start(lanes + Sh::X + nr + t0, y + 16);
            pair::tmem_load_wait(y);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float4 gate = s_gate[k];
                const float r = gate.x * (__uint_as_float((uint32_t)s_v[k * D] << 16) - gate.y * __uint_as_float(y[k]));
                const bool node = real >> k & 1;
                y[k] = node ? __float_as_uint(r) : 0u;
                y[16 + k] = node ? __float_as_uint(gate.z * __uint_as_float(y[16 + k])) : 0u;
                most = fmaf(__uint_as_float(y[k]), 0.f, most);  // NaN from the first infinity or NaN on
            }
            pair::tmem_store16(lanes + Sh::X + t0, y);
            pair::tmem_store16(lanes + Sh::X + nr + t0, y + 16);
            if (most != 0.f) {
#pragma unroll
                for (int k = 0; k < 16; ++k) y[k] = is_odd(y[k]) ? 0u : y[k];
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
                split3(__uint_as_float(y[2 * k]), __uint_as_float(y[2 * k + 1]), part[0][k], part[1][k], part[2][k]);
#pragma unroll
            for (int p = 0; p < 3; ++p) tmem_store8(lanes + Sh::RP + p * 32 + t0 / 2, part[p]);
            pair::tmem_store_wait();
        }
        tc_fence_before_sync();
        const bool odd = pair::named_or(ID, kRows, most != 0.f);
        if (tid == 0) {
            s.odd = odd;
            mbar_arrive(bar(kRParts));
        }
        // -- U and O
        ok = wait_warp(bar(kSecond), i) && ok;
        tc_fence_after_sync();
        if (odd) {  // infinities and NaNs of R to the nodes whose path they are on: rare, and small
            if (work && share == 0) {
                // R_j is one where U_j is, as long as nothing is added to it: from the last node down
#pragma unroll 1
                for (int t = n - 1; t >= 0; --t) {
                    uint32_t y[2];
                    tmem_load1_start(lanes + Sh::X + t, y[0]);
                    tmem_load1_start(lanes + Sh::X + nr + t, y[1]);
                    pair::tmem_load_wait(y);
#pragma unroll 1
                    for (uint64_t up = s.mask[trees & 3][t]; up; up &= up - 1) {
                        const int j = __ffsll((long long)up) - 1;
                        uint32_t w[1];
                        tmem_load1_start(lanes + Sh::X + j, w[0]);
                        pair::tmem_load_wait(w);
                        float f[2] = {0.f, 0.f};  // T and W, the sums of their parts
#pragma unroll 1
                        for (int p = 2; p >= 0; --p) {
                            const uint8_t *const at = smem + Sh::OFF_B + p * Sh::BLOCK + (j & 7) * 2;
                            f[0] += __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(at + sw128_offset(t, j >> 3)) << 16);
                            f[1] += __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(at + sw128_offset(nr + t, j >> 3)) << 16);
                        }
                        const float u = fmaf(f[0], __uint_as_float(w[0]), __uint_as_float(y[0]));
                        const float o = fmaf(f[1], __uint_as_float(w[0]), __uint_as_float(y[1]));
                        if (is_odd(w[0]) && j != t) y[0] = __float_as_uint(u);
                        if (is_odd(w[0])) y[1] = __float_as_uint(o);
                        __syncwarp();  // the next load is the whole warp's
                    }
                    tmem_store1(lanes + Sh::X + t, y[0]);
                    tmem_store1(lanes + Sh::X + nr + t, y[1]);
                    pair::tmem_store_wait();
                }
            }
            tc_fence_before_sync();
            named_sync(ID, kRows);
            tc_fence_after_sync();
            if (tid == 0) mbar_arrive(bar(kBFree));
        }
        if (work && ok && t0 < n) {
            Out *to_o = static_cast<Out *>(a.o) + out0 + t0 * step;
            float *to_u = a.deltas + out0 + t0 * step;
            uint32_t y[32];
            tmem_load16_start(lanes + Sh::X + t0, y);
            tmem_load16_start(lanes + Sh::X + nr + t0, y + 16);
            pair::tmem_load_wait(y);
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kXFree));
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                if (t0 + k >= n) break;
                const float o = a.scale * __uint_as_float(y[16 + k]);
                if constexpr (sizeof(Out) == 2)
                    *to_o = __float2bfloat16_rn(o);
                else
                    *to_o = o;
                to_o += step;
            }
            if (a.deltas) {
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    if (t0 + k >= n) break;
                    *to_u = __uint_as_float(y[k]);
                    to_u += step;
                }
            }
        } else if (lane == 0) {
            mbar_arrive(bar(kXFree));
        }
        if (!more) return ok;
    }
}

template <int D, typename Out>
__global__ void __launch_bounds__(NT, 1) tree_tc_kernel(const __grid_constant__ Args a, int32_t *err) {
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ Tables s;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    if (warp == 0) {
        tmem_alloc(smem_u32(&s.tmem), 512);
        tmem_relinquish();
    } else if (threadIdx.x == 32) {
        for (int i = 0; i < kBars; ++i)
            mbar_init(smem_u32(s.bar + i), i == kParts    ? kStates / 32
                                           : i == kXFree  ? kRows / 32
                                           : i == kVFull  ? kStates
                                                          : 1);
        fence_mbar_init();
    }
    tc_fence_before_sync();
    // every role begins with a __syncthreads(), before which it may issue loads of its own
    bool ok;
    if (warp < kRows / 32)
        ok = rows<D, Out>(a, smem, s);
    else if (warp < (kRows + kStates) / 32)
        ok = states<D>(a, smem, s);
    else if (warp < (kRows + kStates + kFactors) / 32)
        ok = factors<D>(a, smem, s);
    else if (warp == NT / 32 - 2)
        ok = products<D>(a, smem, s);
    else
        ok = gates(a, err, s);
    if (!ok) {
        // a wait gave up: leave the MMAs and copies in flight time to end before their memory goes
        atomicCAS(err, 0, (int32_t)GDR_ERR_DEVICE_TIMEOUT);
        const long long t_end = clock64() + 4000000;
        while (clock64() < t_end) {}
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 0) tmem_dealloc(s.tmem, 512);
}

template <int D, typename Out>
cudaError_t launch_as(const Args &a, int32_t *err, cudaStream_t s) {
    static attn::SmemOptIn opt_in;
    const cudaError_t e = opt_in.set(reinterpret_cast<const void *>(tree_tc_kernel<D, Out>), (int)Shape::BYTES);
    if (e != cudaSuccess) return e;
    const int64_t pairs = (int64_t)a.n_seqs * a.h_v;
    tree_tc_kernel<D, Out><<<(unsigned)(pairs < kGrid ? pairs : kGrid), NT, Shape::BYTES, s>>>(a, err);
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
