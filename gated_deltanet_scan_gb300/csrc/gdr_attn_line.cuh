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
__host__ __device__ constexpr Spec spec(bool wide, int d) {
    return wide ? Spec{128, 64, 1, 4} : Spec{kWarpRows, 16, 8, 1024 / d};
}
inline bool is_wide(int rows) { return rows > kWarpRows; }

// Workspace: place of every sequence's first triple on the line ([n_seqs + 1], the last
// one the total), then per worker two parts (its first and its last, cut, triple): per
// row m and l, then O.
struct Layout {
    int blocks_of_rows, part_rows, workers;
    size_t ml, o, total;
};
__host__ __device__ inline Layout layout(int rows, const Spec &sp, int d, int n_seqs) {
    Layout L;
    L.blocks_of_rows = (rows + sp.block_rows - 1) / sp.block_rows;
    L.part_rows = rows < sp.block_rows ? rows : sp.block_rows;
    L.workers = kBlocks * sp.workers;
    const size_t parts = (size_t)L.workers * 2 * L.part_rows;
    L.ml = ((size_t)(n_seqs + 1) * 8 + 15) / 16 * 16;
    L.o = L.ml + (parts * 8 + 15) / 16 * 16;
    L.total = L.o + parts * d * 4;
    return L;
}

// Tokens of sequence s; outside [0, limit] counts as none.
__device__ __forceinline__ int64_t length_of(const Args &a, int s) {
    const int64_t n = a.kv_lens[s];
    return n < 0 || n > (int64_t)a.cache.max_pages * a.cache.page_size ? 0 : n;
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
// sequences).  Block 0 leaves the sequences' places in the workspace for the join.
template <int THREADS, int WORKERS>
struct Line {
    int64_t scan[THREADS + 1];
    int64_t warp_sum[THREADS / 32];
    int64_t base[WORKERS];
    int seq[WORKERS];

    __device__ __forceinline__ int64_t place(const Args &a, const Spec &sp, int blocks_of_rows) {
        const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
        const int64_t per_seq = (int64_t)a.h_kv * blocks_of_rows;
        int64_t *const line = reinterpret_cast<int64_t *>(a.ws);
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
                    if (blockIdx.x == 0) {
                        if (tid < m) line[s0 + tid] = scan[tid];
                        if (tid == 0 && c == chunks - 1) line[a.n_seqs] = sum;
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
