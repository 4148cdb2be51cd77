// Internal launch interface of the attention operators.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/gdr.h"

namespace gdr {
namespace attn {

// A kernel's opt-in to more than 48 KiB of dynamic shared memory, set once per
// device (one bit each; setting it twice from two threads is harmless).
struct SmemOptIn {
    std::atomic<uint64_t> done{0};
    cudaError_t set(const void *kernel, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = dev < 64 ? 1ull << dev : 0;
        if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
        return e;
    }
};

// Strided rows of heads: value x of head h of token t at p[t * ts + h * hs + x].
struct Rows {
    uint16_t *p;
    int64_t ts, hs;
};

struct Cache {
    uint16_t *k, *v;
    int64_t page_stride, token_stride, head_stride;
    const int32_t *table;
    int64_t table_stride;
    int32_t n_pages, page_size, max_pages;
};

// Everything one launch needs, already validated on the host.
struct Args {
    int h_q, h_kv, group, d;
    int f16;  // 1: fp16, 0: bf16
    float scale;
    int n_seqs, n_tok;  // n_tok: decode's tokens per sequence
    const int32_t *cu;  // packed sequences' starts; nullptr (append): t_total / n_seqs tokens each
    int64_t t_total;
    Rows q, k, v, o;
    Rows q_out, k_out;  // append: p is nullptr where not wanted
    Cache cache;
    const int32_t *kv_lens;
    int least;               // smallest length but 0 that a sequence may have
    const int32_t *parents;  // a tree's, [n_seqs][n_tok]; nullptr: the last tokens are a chain
    float *lse;
    const float *inv_freq;
    int rot, interleaved;
    // compaction: the caches of n_layers layers, layer_stride elements apart
    const int32_t *last;  // each tree's last accepted node, or -1
    int32_t *lens_out;    // nullptr where not wanted
    int n_layers;
    int64_t layer_stride;
    void *ws;
    int32_t *err;
};

cudaError_t launch_append(const Args &a, cudaStream_t s);
// Prompts: a short sequence goes to the short kernel, a longer one to the two-SM kernel;
// each skips the other's.  Short is what fills at most one of the two-SM kernel's blocks
// (256 rows), up to 128 tokens.  Measured with all sequences in one kernel, short against
// two-SM: 16 heads of 256 in groups of 4, 64 tokens x 8 8.0 / 11.0 us, x 32 20.9 / 18.7,
// 128 tokens x 8 13.7 / 12.1, x 32 44.0 / 27.0; 16 heads of 128 in groups of 1, 128 tokens
// x 8 9.9 / 12.7, x 32 25.3 / 27.1, 256 tokens x 8 21.4 / 16.4, x 32 67.7 / 36.0; of 64,
// 128 tokens x 32 16.5 / 24.3.
__host__ __device__ constexpr int short_tokens(int group) { return 256 / group < 128 ? 256 / group : 128; }
cudaError_t launch_prefill(const Args &a, cudaStream_t s);
// `after`: launched as a programmatic dependent of the two-SM kernel just before it.
cudaError_t launch_prefill_short(const Args &a, bool after, cudaStream_t s);
cudaError_t launch_decode(const Args &a, cudaStream_t s);
cudaError_t launch_compact(const Args &a, cudaStream_t s);
size_t decode_workspace_bytes(int h_q, int h_kv, int d, int n_seqs, int n_tok, bool tree);

}  // namespace attn
}  // namespace gdr
