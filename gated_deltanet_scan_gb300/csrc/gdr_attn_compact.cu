// The accepted path of a tree of drafted tokens, moved to the front of the tree's slots in
// every layer's cache, and the sequences' new lengths.
//
// The path's nodes in rising order, i = 0, 1, ..., are rows r_0 < r_1 < ... of the tree, so
// r_i >= i: row base + r_i goes to slot base + i, for keys and values of every head and layer.
// Slot i may be an earlier node's row (r_k = i, k < i) and is never a later one's (r_k > i for
// k > i), so whoever moves a vector of all rows in rising order may write row i once rows
// 0 .. i are read: a thread owns one 16-byte vector position (layer, K or V, head, place in the
// head) and reads kBatch rows of it before it writes them.  Nothing waits for another thread.
//
// Bound by latency: a path is a few rows (2 KB per row, layer and K or V at 4 heads of 256),
// behind the loads of the tree, the length and the page table.  All layers are one launch: 8 layers of 4
// heads of 256, one tree of 24 nodes 6.2 us, 64 of 64 8.2 us (their bytes would take 1.5).
#include "gdr_attn_common.cuh"
#include "gdr_internal.h"
#include "gdr_tree.cuh"

namespace gdr {
namespace attn {
namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 8;

__global__ void __launch_bounds__(kThreads) compact_kernel(const __grid_constant__ Args a) {
    __shared__ int64_t s_from[tree::kMaxNodes], s_to[tree::kMaxNodes];  // offsets in a layer, -1: not moved
    __shared__ int s_count;
    const int s = blockIdx.x, lane = threadIdx.x & 31;
    if (threadIdx.x < 32) {
        const int last = a.last[s];
        const int64_t len = a.kv_lens[s], base = len - a.n_tok;
        const tree::Masks nodes = tree::masks(a.parents + (int64_t)s * a.n_tok, a.n_tok, lane);
        const bool inside = base >= 0 && len <= (int64_t)a.cache.max_pages * a.cache.page_size;
        uint64_t path = tree::mask_of(nodes, last & 63);
        if (last < 0 || last >= a.n_tok || !inside) path = 0;
        const int count = __popcll(path);
        // a sequence of no tokens is not in the batch, whatever its tree and last node hold
        const bool bad = len != 0 && (nodes.bad || last < -1 || (last >= 0 && count == 0) || !inside);
        if (bad && blockIdx.y == 0) record_invalid(a.err);
        auto offset = [&](int64_t p) -> int64_t {
            const int pg = (int)((uint32_t)p / (uint32_t)a.cache.page_size);
            const int page = a.cache.table[(int64_t)s * a.cache.table_stride + pg];
            if (page < 0 || page >= a.cache.n_pages) {
                record_invalid(a.err);
                return -1;
            }
            return page * a.cache.page_stride + (p - (int64_t)pg * a.cache.page_size) * a.cache.token_stride;
        };
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int j = lane + 32 * x;
            if (!(path >> j & 1)) continue;
            const int i = __popcll(path & ((1ull << j) - 1));
            int64_t from = -1, to = -1;
            if (i != j) {
                from = offset(base + j);
                to = offset(base + i);
            }
            s_from[i] = to < 0 ? -1 : from;
            s_to[i] = to;
        }
        if (lane == 0) {
            s_count = count;
            if (a.lens_out && blockIdx.y == 0) a.lens_out[s] = inside ? (int32_t)(base + count) : (int32_t)len;
        }
    }
    __syncthreads();
    const int count = s_count, per_row = a.h_kv * (a.d / 8);
    const int64_t vec = (int64_t)blockIdx.y * kThreads + threadIdx.x;
    const int64_t plane = vec / per_row;  // 2 layer + (K or V)
    if (plane >= 2 * (int64_t)a.n_layers) return;
    const int x = (int)(vec - plane * per_row), h = x / (a.d / 8);
    uint16_t *const at = ((plane & 1) ? a.cache.v : a.cache.k) + (plane >> 1) * a.layer_stride + h * a.cache.head_stride +
                         (x - h * (a.d / 8)) * 8;
    for (int i0 = 0; i0 < count; i0 += kBatch) {
        uint4 w[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (i0 + u < count && s_from[i0 + u] >= 0) w[u] = *reinterpret_cast<const uint4 *>(at + s_from[i0 + u]);
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (i0 + u < count && s_from[i0 + u] >= 0) *reinterpret_cast<uint4 *>(at + s_to[i0 + u]) = w[u];
    }
}

}  // namespace

cudaError_t launch_compact(const Args &a, cudaStream_t s) {
    const int64_t vectors = 2 * (int64_t)a.n_layers * a.h_kv * (a.d / 8);
    const dim3 grid((unsigned)a.n_seqs, (unsigned)((vectors + kThreads - 1) / kThreads));
    compact_kernel<<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace attn
}  // namespace gdr
