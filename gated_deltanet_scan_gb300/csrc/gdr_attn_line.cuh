// The line that decode's work lies on, shared by its kernels and their join.
//
// A triple is a (sequence, key/value head, block of rows).  The tiles of all triples lie
// on one line, sequence by sequence, which is cut into equal parts, one per worker.  A
// triple takes its tiles and, before them, `lead` places for what starting and ending it
// costs a worker, so that a batch of many short sequences is cut evenly too.
#pragma once

#include "gdr_attn_common.cuh"

namespace gdr {
namespace attn {

constexpr int kBlocks = 152;  // one resident block per SM
constexpr int kWarpRows = 16;  // rows the warp kernel takes; more go to the wide kernel

struct Spec {
    int block_rows;  // rows of a key/value head per block of rows
    int tile;        // tokens
    int workers;     // per block of threads
    int lead;        // places
};
// The warp kernel: workers of one warp and 16 rows, a tile 32 d bytes of keys and as many of
// values at a 1216th of the bandwidth (d = 256: 3 us).  The wide kernel: one worker of 128
// rows per SM, tiles of 64 tokens.  Leads measured: 512 / d, 1024 / d and 1536 / d places for
// the first (25 sequences of d = 256 42.3, 39.4, 37.3 us; 64 sequences 120.8, 120.8, 121.6; 96 of
// d = 128 119.5, 119.7, 121.5); 3, 4 and 6 for the second (16 draft tokens 39.8, 38.5, 38.6; 50
// sequences of d = 128 47.2, 47.6, 47.8; 52 of d = 64 30.3, 29.9, 30.5).
enum Kind { kFew = 0, kWide = 1, kPaired = 2 };
__host__ __device__ constexpr Spec spec(Kind kind, int d) {
    return kind == kFew ? Spec{kWarpRows, 16, 8, 1024 / d} : Spec{kind == kPaired ? 256 : 128, 64, 1, 4};
}
// Of the rows of a key/value head, of so many heads of all sequences.  Trees of more than 128 rows of up to 128
// values, more blocks of rows than workers: two of them read the keys and values together.  (The O of two
// blocks of d = 256 would leave no TMEM for their S.)  Fewer have more to lose by parts of twice the rows.
// fp16, us apart / together, every sequence of 1,000, 2,000 and 8,000 tokens (lengths are not known on the host):
//   256 rows, d = 128: 80 heads 39.0 / 41.2, 53.3 / 53.3, 136.8 / 115.5; 96 43.1 / 44.7, 61.4 / 59.4, 159.9 / 133.2;
//     128 51.4 / 51.2, 75.8 / 69.7, 206.6 / 169.3; 512 151 / 135, 242 / 204, 765 / 595
//   256 rows, d = 64: 80 heads 30.0 / 30.5, 43.1 / 39.1, 114.7 / 89.6; 512 117 / 94, 193 / 150, 643 / 467
//   160 rows, d = 128: 80 heads 34.9 / 35.0, 49.5 / 47.0, 133.2 / 110.0; 512 139 / 118, 235 / 189, 757 / 580
// With fewer heads than that: 64 heads of 1,000 28.9 / 34.9, of up to 8,000 53.1 / 50.8; 32 of 4,000 28.9 / 32.9, of
// 16,000 45.9 / 45.1; 4 of 1,500 16.4 / 20.5.
inline Kind kind_of(int rows, int d, bool tree, int64_t heads) {
    return rows <= kWarpRows                                                                ? kFew
           : tree && rows > 128 && d <= 128 && (int64_t)((rows + 127) / 128) * heads > kBlocks ? kPaired
                                                                                              : kWide;
}

// Where the parts of a triple's rows are, for the join.
struct __align__(16) Parts {
    int w0, w1;     // first and last worker
    int count;      // parts to join; 1: the worker wrote the rows themselves
    int packed;     // whether the first part is its worker's second; w0 in its block; workers of a block
    __device__ __forceinline__ int64_t row(int i, int part_rows) const {  // of part i's first row
        const int wk = i == 0 ? w0 : i == count - 1 ? w1 : w0 - (packed >> 1 & 15) + i * (packed >> 5);
        return (int64_t)(2 * wk + (i == 0 ? packed & 1 : 0)) * part_rows;
    }
};

// Workspace: per triple its parts' places, then per worker two parts (its first and its last, cut,
// triple): per row m and l, then O.
struct Layout {
    int blocks_of_rows, part_rows, workers;
    size_t ml, o, total;
};
__host__ __device__ inline Layout layout(int rows, const Spec &sp, int d, int64_t heads) {  // of all sequences
    Layout L;
    L.blocks_of_rows = (rows + sp.block_rows - 1) / sp.block_rows;
    L.part_rows = rows < sp.block_rows ? rows : sp.block_rows;
    L.workers = kBlocks * sp.workers;
    const size_t parts = (size_t)L.workers * 2 * L.part_rows;
    L.ml = (size_t)heads * L.blocks_of_rows * sizeof(Parts);
    L.o = L.ml + (parts * 8 + 15) / 16 * 16;
    L.total = L.o + parts * d * 4;
    return L;
}

// Tokens of sequence s; outside [0, limit], or fewer than a tree's nodes, counts as none.
__device__ __forceinline__ int64_t length_of(const Args &a, int s) {
    const int64_t n = a.kv_lens[s];
    return n < a.least || n > (int64_t)a.cache.max_pages * a.cache.page_size ? 0 : n;
}
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {  // a, b >= 0; mostly 32-bit values
    return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}
// The line of `total` places in equal parts, the first `rest` one longer; never more
// parts than places.
struct Cut {
    int64_t each, rest;
    int parts, per_block;  // workers in use, and of each block: few places spread over many blocks
    __device__ __forceinline__ Cut(int64_t total, int workers_per_block) {
        per_block = total >= (int64_t)kBlocks * workers_per_block ? workers_per_block
                                                                  : max(1, (int)((uint32_t)total / kBlocks));
        parts = total < kBlocks * per_block ? (int)total : kBlocks * per_block;
        each = parts > 0 ? quotient(total, parts) : 0;
        rest = total - each * parts;
    }
    __device__ __forceinline__ int64_t start(int w) const { return each * w + (w < rest ? w : rest); }
    __device__ __forceinline__ int part_of(int64_t place) const {
        const int64_t longer = rest * (each + 1);
        return (int)(place < longer ? quotient(place, each + 1) : rest + quotient(place - longer, each));
    }
};

// Left by one thread of the worker of a triple's first tiles.  A worker's part is its first where its own
// start is not before the triple's: so all parts but perhaps the first one's.  All but the last worker's
// part are joined within their blocks: the parts are those of the first such worker of every block, and
// the last worker's.  (Found by the join's threads, each for its row, it took them 500 instructions.)
__device__ __forceinline__ void leave_parts(const Args &a, const Spec &sp, const Layout &L, const Cut &cut, int me, int s,
                                            int h, int rb, int64_t seg0, int64_t tiles) {
    Parts p;
    p.w0 = me;
    p.w1 = cut.part_of(seg0 + sp.lead + tiles - 1);
    p.count = p.w1 == me ? 1 : (p.w1 - 1) / cut.per_block - me / cut.per_block + 2;
    p.packed = (cut.start(me) >= seg0 ? 0 : 1) | me % cut.per_block << 1 | cut.per_block << 5;
    static_cast<Parts *>(a.ws)[((int64_t)s * a.h_kv + h) * L.blocks_of_rows + rb] = p;
}

// The part of one triple that falls to a worker.
struct Triple {
    int s, h, rb;
    int len, tiles;       // of the sequence
    int tile0, tile1;     // the worker's
    int64_t seg0;         // where the triple starts on the line
};
// A worker's way along its part of the line, from sequence s, which starts at `base`.
struct Walk {
    int64_t at, end, base;
    int s;
    __device__ __forceinline__ bool next(const Args &a, const Spec &sp, int blocks_of_rows, Triple &t) {
        const int64_t per_seq = (int64_t)a.h_kv * blocks_of_rows;
        while (at < end) {
            int64_t len, tiles, places;
            for (;;) {
                len = length_of(a, s);
                tiles = (len + sp.tile - 1) / sp.tile;
                places = len > 0 ? tiles + sp.lead : 0;
                if (at < base + places * per_seq) break;
                base += places * per_seq;
                ++s;
            }
            const int hr = (int)quotient(at - base, places);
            t.s = s;
            t.h = hr / blocks_of_rows;
            t.rb = hr - t.h * blocks_of_rows;
            t.len = (int)len;
            t.tiles = (int)tiles;
            t.seg0 = base + hr * places;
            t.tile0 = (int)max((int64_t)0, at - t.seg0 - sp.lead);
            t.tile1 = (int)min(tiles, end - t.seg0 - sp.lead);
            at = t.seg0 + places;
            if (t.tile1 > t.tile0) return true;  // else only lead places: the next worker has the tiles
        }
        return false;
    }
};

// The line's scan by a whole block of THREADS: THREADS sequences at a time, an exclusive
// sum of their places; the first pass finds the total, the second where each of the
// block's WORKERS starts (one pass of sums does both where there are up to THREADS
// sequences).
template <int THREADS, int WORKERS>
struct Line {
    int64_t scan[THREADS + 1];
    int64_t warp_sum[THREADS / 32];
    int64_t base[WORKERS];
    int seq[WORKERS];

    __device__ __forceinline__ int64_t place(const Args &a, const Spec &sp, int blocks_of_rows) {
        const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
        const int64_t per_seq = (int64_t)a.h_kv * blocks_of_rows;
        int64_t total = 0;
        const int chunks = (a.n_seqs + THREADS - 1) / THREADS;
        if (tid < WORKERS) seq[tid] = -1;
        for (int pass = 0; pass < 2; ++pass) {
            int64_t sum = 0;
            for (int c = 0; c < chunks; ++c) {
                if (pass == 0 || chunks > 1) {
                    const int s = c * THREADS + tid;
                    int64_t n = 0;
                    if (s < a.n_seqs) {
                        n = length_of(a, s);
                        if (pass == 0 && blockIdx.x == 0 && n != a.kv_lens[s]) record_invalid(a.err);
                        if (n > 0) n = ((n + sp.tile - 1) / sp.tile + sp.lead) * per_seq;
                    }
                    int64_t x = n;
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
                        if (lane >= d) x += y;
                    }
                    __syncthreads();
                    if (lane == 31) warp_sum[warp] = x;
                    __syncthreads();
                    int64_t before = 0;
#pragma unroll
                    for (int i = 0; i < THREADS / 32; ++i)
                        if (i < warp) before += warp_sum[i];
                    scan[tid] = sum + before + x - n;
                    if (tid == THREADS - 1) scan[THREADS] = sum + before + x;
                    __syncthreads();
                }
                sum = scan[THREADS];
                if (pass == 1) {
                    const int s0 = c * THREADS, m = min(THREADS, a.n_seqs - s0);
                    if (tid < WORKERS) {  // the last sequence that starts at or before the worker's part
                        const Cut cut(total, WORKERS);
                        const int64_t at = cut.start(min((int)blockIdx.x * cut.per_block + tid, cut.parts));
                        if (tid < cut.per_block && seq[tid] < 0 && at < sum) {
                            int lo = 0, hi = m - 1;
                            while (lo < hi) {
                                const int mid = (lo + hi + 1) >> 1;
                                if (scan[mid] <= at)
                                    lo = mid;
                                else
                                    hi = mid - 1;
                            }
                            seq[tid] = s0 + lo;
                            base[tid] = scan[lo];
                        }
                    }
                }
            }
            total = sum;
        }
        __syncthreads();
        return total;
    }
    // Worker `wk` of this block, number `me` on the line.
    __device__ __forceinline__ Walk walk(const Cut &cut, int wk, int &me) const {
        me = blockIdx.x * cut.per_block + wk;
        Walk w;
        w.at = cut.start(min(me, cut.parts));  // beyond the parts: nothing to do
        w.end = wk < cut.per_block ? cut.start(min(me + 1, cut.parts)) : w.at;
        w.base = base[wk];
        w.s = seq[wk];
        return w;
    }
};

cudaError_t launch_decode_wide(const Args &a, cudaStream_t s);

}  // namespace attn
}  // namespace gdr
