// C-ABI entry points of the attention operators: argument checks on the host,
// then the launches.
#include <climits>
#include <cmath>

#include "gdr_attn.h"
#include "gdr_internal.h"
#include "gdr_overlap.h"

namespace gdr {
namespace attn {
namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 38;

bool aligned(const void *p, uintptr_t bytes) { return p && (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
bool stride_ok(int64_t s) { return s >= 0 && s < kMaxStride && (s & 7) == 0; }
bool rows_ok(const gdr_rows *r) {
    return r && aligned(r->ptr, 16) && stride_ok(r->token_stride) && stride_ok(r->head_stride);
}
// Rows that a kernel writes.
bool out_rows_ok(const gdr_rows *r, int64_t tokens, int heads, int d) {
    return rows_ok(r) && !overlap(tokens, r->token_stride, heads, r->head_stride, d);
}
bool out_cache_ok(const gdr_kv_cache *c, int heads, int d) {  // any two of its three dimensions
    return !overlap(c->n_pages, c->page_stride, c->page_size, c->token_stride, d) &&
           !overlap(c->page_size, c->token_stride, heads, c->head_stride, d) &&
           !overlap(c->n_pages, c->page_stride, heads, c->head_stride, d);
}
Rows to_rows(const gdr_rows *r) {
    if (!r) return Rows{nullptr, 0, 0};
    return Rows{static_cast<uint16_t *>(r->ptr), r->token_stride, r->head_stride};
}

gdr_status check_dims(const gdr_attn_dims *d) {
    if (!d || d->h_q <= 0 || d->h_kv <= 0 || d->h_q % d->h_kv != 0 || d->d <= 0) return GDR_ERR_INVALID_ARG;
    if (d->dtype != GDR_F32 && d->dtype != GDR_BF16 && d->dtype != GDR_F16) return GDR_ERR_INVALID_ARG;
    if (!std::isfinite(d->scale)) return GDR_ERR_INVALID_ARG;
    if (d->dtype == GDR_F32) return GDR_ERR_UNSUPPORTED;
    if (d->d != 64 && d->d != 128 && d->d != 256) return GDR_ERR_UNSUPPORTED;
    if (d->h_q / d->h_kv > 128 || d->h_kv > 65535) return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

gdr_status check_cache(const gdr_kv_cache *c) {
    if (!c || !aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->page_table, 4)) return GDR_ERR_INVALID_ARG;
    if (!stride_ok(c->page_stride) || !stride_ok(c->token_stride) || !stride_ok(c->head_stride))
        return GDR_ERR_INVALID_ARG;
    if (c->n_pages < 1 || c->page_size < 1 || c->max_pages < 1 || c->table_stride < 0) return GDR_ERR_INVALID_ARG;
    // positions and the ends of tiles past them are 32-bit
    if ((int64_t)c->page_size * c->max_pages > INT_MAX - 1023) return GDR_ERR_INVALID_ARG;
    return GDR_OK;
}

Args make_args(const gdr_attn_dims *d) {
    Args a{};
    a.h_q = d->h_q;
    a.h_kv = d->h_kv;
    a.group = d->h_q / d->h_kv;
    a.d = d->d;
    a.f16 = d->dtype == GDR_F16;
    a.scale = d->scale;
    return a;
}

Cache to_cache(const gdr_kv_cache *c) {
    return Cache{static_cast<uint16_t *>(c->k), static_cast<uint16_t *>(c->v), c->page_stride, c->token_stride,
                 c->head_stride, c->page_table, c->table_stride, c->n_pages, c->page_size, c->max_pages};
}

gdr_status from_cuda(cudaError_t e) { return e == cudaSuccess ? GDR_OK : GDR_ERR_CUDA; }

bool nodes_ok(int32_t n_tok) { return n_tok >= 1 && n_tok <= 64; }

// `parents`: of trees of t_total / n_seqs rows each, or nullptr.
gdr_status append(const gdr_attn_dims *dims, int32_t n_seqs, const int32_t *cu_seqlens, const int32_t *parents,
                  int64_t t_total, const gdr_rows *q, const gdr_rows *k, const gdr_rows *v, const gdr_rows *q_out,
                  const gdr_rows *k_out, const gdr_kv_cache *cache, const int32_t *kv_lens, const float *inv_freq,
                  int32_t rot_dim, int32_t interleaved, gdr_stream_t stream) {
    gdr_status st = check_dims(dims);
    if (st != GDR_OK) return st;
    if (n_seqs < 0 || t_total < 0 || (n_seqs == 0 && t_total > 0)) return GDR_ERR_INVALID_ARG;
    if (rot_dim < 0 || rot_dim > dims->d || (rot_dim & 1)) return GDR_ERR_INVALID_ARG;
    if (t_total == 0) return GDR_OK;  // an empty batch's tensors may have no address
    if (rot_dim > 0 && !aligned(inv_freq, 4)) return GDR_ERR_INVALID_ARG;
    st = check_cache(cache);
    if (st != GDR_OK) return st;
    if (t_total > INT_MAX) return GDR_ERR_UNSUPPORTED;
    if (cu_seqlens ? !aligned(cu_seqlens, 4) : t_total % n_seqs != 0) return GDR_ERR_INVALID_ARG;
    if (!aligned(kv_lens, 4) || !rows_ok(k) || !rows_ok(v)) return GDR_ERR_INVALID_ARG;
    if (!q != !q_out || (q && (!rows_ok(q) || !out_rows_ok(q_out, t_total, dims->h_q, dims->d))))
        return GDR_ERR_INVALID_ARG;
    if (k_out && !out_rows_ok(k_out, t_total, dims->h_kv, dims->d)) return GDR_ERR_INVALID_ARG;
    if (!out_cache_ok(cache, dims->h_kv, dims->d)) return GDR_ERR_INVALID_ARG;
    // in place: the same rows (a row is read whole before it is written)
    if (q && q->ptr == q_out->ptr &&
        (q->token_stride != q_out->token_stride || q->head_stride != q_out->head_stride))
        return GDR_ERR_INVALID_ARG;
    if (k_out && k->ptr == k_out->ptr &&
        (k->token_stride != k_out->token_stride || k->head_stride != k_out->head_stride))
        return GDR_ERR_INVALID_ARG;
    Args a = make_args(dims);
    a.n_seqs = n_seqs;
    a.cu = cu_seqlens;
    a.parents = parents;
    a.t_total = t_total;
    a.q = to_rows(q);
    a.k = to_rows(k);
    a.v = to_rows(v);
    a.q_out = to_rows(q_out);
    a.k_out = to_rows(k_out);
    a.cache = to_cache(cache);
    a.kv_lens = kv_lens;
    a.inv_freq = inv_freq;
    a.rot = rot_dim;
    a.interleaved = interleaved != 0;
    a.err = gdr::device_error_word();
    if (!a.err) return GDR_ERR_CUDA;
    return from_cuda(launch_append(a, reinterpret_cast<cudaStream_t>(stream)));
}

// `parents`: of trees of n_tok rows each, or nullptr.
gdr_status decode(const gdr_attn_dims *dims, int32_t n_seqs, int32_t n_tok, const int32_t *parents, const gdr_rows *q,
                  const gdr_kv_cache *cache, const int32_t *kv_lens, const gdr_rows *o, float *lse, void *workspace,
                  size_t workspace_bytes, gdr_stream_t stream) {
    gdr_status st = check_dims(dims);
    if (st != GDR_OK) return st;
    if (n_seqs < 0) return GDR_ERR_INVALID_ARG;
    if (n_seqs == 0) return GDR_OK;
    st = check_cache(cache);
    if (st != GDR_OK) return st;
    if (!rows_ok(q) || !out_rows_ok(o, (int64_t)n_seqs * n_tok, dims->h_q, dims->d) || !aligned(kv_lens, 4) ||
        (lse && !aligned(lse, 4)))
        return GDR_ERR_INVALID_ARG;
    if ((int64_t)n_seqs * n_tok > INT_MAX / dims->h_q) return GDR_ERR_UNSUPPORTED;
    const size_t need = decode_workspace_bytes(dims->h_q, dims->h_kv, dims->d, n_seqs, n_tok, parents != nullptr);
    if (need > 0 && (!aligned(workspace, 16) || workspace_bytes < need)) return GDR_ERR_INVALID_ARG;
    Args a = make_args(dims);
    a.n_seqs = n_seqs;
    a.n_tok = n_tok;
    a.t_total = (int64_t)n_seqs * n_tok;
    a.q = to_rows(q);
    a.o = to_rows(o);
    a.cache = to_cache(cache);
    a.kv_lens = kv_lens;
    a.parents = parents;
    a.least = parents ? n_tok : 0;
    a.lse = lse;
    a.ws = workspace;
    a.err = gdr::device_error_word();
    if (!a.err) return GDR_ERR_CUDA;
    return from_cuda(launch_decode(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace
}  // namespace attn
}  // namespace gdr

using namespace gdr::attn;

extern "C" {

gdr_status gdr_attn_append(const gdr_attn_dims *dims, int32_t n_seqs, const int32_t *cu_seqlens, int64_t t_total,
                           const gdr_rows *q, const gdr_rows *k, const gdr_rows *v, const gdr_rows *q_out,
                           const gdr_rows *k_out, const gdr_kv_cache *cache, const int32_t *kv_lens,
                           const float *inv_freq, int32_t rot_dim, int32_t interleaved, gdr_stream_t stream) {
    return append(dims, n_seqs, cu_seqlens, nullptr, t_total, q, k, v, q_out, k_out, cache, kv_lens, inv_freq, rot_dim,
                  interleaved, stream);
}

gdr_status gdr_attn_append_tree(const gdr_attn_dims *dims, int32_t n_seqs, int32_t n_tok, const int32_t *parents,
                                const gdr_rows *q, const gdr_rows *k, const gdr_rows *v, const gdr_rows *q_out,
                                const gdr_rows *k_out, const gdr_kv_cache *cache, const int32_t *kv_lens,
                                const float *inv_freq, int32_t rot_dim, int32_t interleaved, gdr_stream_t stream) {
    if (n_seqs < 0 || !nodes_ok(n_tok) || (n_seqs > 0 && !aligned(parents, 4))) return GDR_ERR_INVALID_ARG;
    return append(dims, n_seqs, nullptr, parents, (int64_t)n_seqs * n_tok, q, k, v, q_out, k_out, cache, kv_lens,
                  inv_freq, rot_dim, interleaved, stream);
}

gdr_status gdr_attn_prefill(const gdr_attn_dims *dims, int32_t n_seqs, const int32_t *cu_seqlens, int64_t t_total,
                            const gdr_rows *q, const gdr_rows *k, const gdr_rows *v, const gdr_rows *o, float *lse,
                            gdr_stream_t stream) {
    gdr_status st = check_dims(dims);
    if (st != GDR_OK) return st;
    if (n_seqs < 0 || t_total < 0 || (n_seqs == 0 && t_total > 0)) return GDR_ERR_INVALID_ARG;
    if (t_total == 0) return GDR_OK;
    if (t_total > INT_MAX) return GDR_ERR_UNSUPPORTED;
    if (!aligned(cu_seqlens, 4) || !rows_ok(q) || !rows_ok(k) || !rows_ok(v) ||
        !out_rows_ok(o, t_total, dims->h_q, dims->d))
        return GDR_ERR_INVALID_ARG;
    if (lse && !aligned(lse, 4)) return GDR_ERR_INVALID_ARG;
    Args a = make_args(dims);
    a.n_seqs = n_seqs;
    a.cu = cu_seqlens;
    a.t_total = t_total;
    a.q = to_rows(q);
    a.k = to_rows(k);
    a.v = to_rows(v);
    a.o = to_rows(o);
    a.lse = lse;
    a.err = gdr::device_error_word();
    if (!a.err) return GDR_ERR_CUDA;
    return from_cuda(launch_prefill(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t gdr_attn_decode_workspace_bytes(const gdr_attn_dims *dims, int32_t n_seqs, int32_t n_tok) {
    if (check_dims(dims) != GDR_OK || n_seqs <= 0 || n_tok < 1 || n_tok > 16) return 0;
    return decode_workspace_bytes(dims->h_q, dims->h_kv, dims->d, n_seqs, n_tok, false);
}

gdr_status gdr_attn_decode(const gdr_attn_dims *dims, int32_t n_seqs, int32_t n_tok, const gdr_rows *q,
                           const gdr_kv_cache *cache, const int32_t *kv_lens, const gdr_rows *o, float *lse,
                           void *workspace, size_t workspace_bytes, gdr_stream_t stream) {
    const gdr_status st = check_dims(dims);
    if (st != GDR_OK) return st;
    if (n_tok < 1 || n_tok > 16) return GDR_ERR_INVALID_ARG;
    return decode(dims, n_seqs, n_tok, nullptr, q, cache, kv_lens, o, lse, workspace, workspace_bytes, stream);
}

size_t gdr_attn_decode_tree_workspace_bytes(const gdr_attn_dims *dims, int32_t n_seqs, int32_t n_tok) {
    if (check_dims(dims) != GDR_OK || n_seqs <= 0 || !nodes_ok(n_tok)) return 0;
    return decode_workspace_bytes(dims->h_q, dims->h_kv, dims->d, n_seqs, n_tok, true);
}

gdr_status gdr_attn_decode_tree(const gdr_attn_dims *dims, int32_t n_seqs, int32_t n_tok, const int32_t *parents,
                                const gdr_rows *q, const gdr_kv_cache *cache, const int32_t *kv_lens, const gdr_rows *o,
                                float *lse, void *workspace, size_t workspace_bytes, gdr_stream_t stream) {
    const gdr_status st = check_dims(dims);
    if (st != GDR_OK) return st;
    if (!nodes_ok(n_tok) || (n_seqs > 0 && !aligned(parents, 4))) return GDR_ERR_INVALID_ARG;
    return decode(dims, n_seqs, n_tok, parents, q, cache, kv_lens, o, lse, workspace, workspace_bytes, stream);
}

gdr_status gdr_attn_commit_tree(const gdr_attn_dims *dims, int32_t n_seqs, int32_t n_tok, const int32_t *parents,
                                const int32_t *last, int32_t n_layers, int64_t layer_stride, const gdr_kv_cache *cache,
                                const int32_t *kv_lens, int32_t *lens_out, gdr_stream_t stream) {
    gdr_status st = check_dims(dims);
    if (st != GDR_OK) return st;
    if (n_seqs < 0 || !nodes_ok(n_tok) || n_layers < 1) return GDR_ERR_INVALID_ARG;
    if (n_seqs == 0) return GDR_OK;
    if (!aligned(parents, 4) || !aligned(last, 4) || !aligned(kv_lens, 4) || (lens_out && !aligned(lens_out, 4)))
        return GDR_ERR_INVALID_ARG;
    // other blocks read a sequence's length, last node and parents while one writes its new length
    auto over = [&](const int32_t *x, int64_t n) { return lens_out < x + n && x < lens_out + n_seqs; };
    if (lens_out && (over(kv_lens, n_seqs) || over(last, n_seqs) || over(parents, (int64_t)n_seqs * n_tok)))
        return GDR_ERR_INVALID_ARG;
    st = check_cache(cache);
    if (st != GDR_OK) return st;
    if (!stride_ok(layer_stride) || !out_cache_ok(cache, dims->h_kv, dims->d)) return GDR_ERR_INVALID_ARG;
    if (overlap(n_layers, layer_stride, cache->n_pages, cache->page_stride, dims->d) ||
        overlap(n_layers, layer_stride, cache->page_size, cache->token_stride, dims->d) ||
        overlap(n_layers, layer_stride, dims->h_kv, cache->head_stride, dims->d))
        return GDR_ERR_INVALID_ARG;
    // a block per 128 16-byte vectors of a row in all layers, in a grid dimension of 65535
    if ((int64_t)n_layers * dims->h_kv * (dims->d / 4) > 65535 * (int64_t)128) return GDR_ERR_UNSUPPORTED;
    Args a = make_args(dims);
    a.n_seqs = n_seqs;
    a.n_tok = n_tok;
    a.parents = parents;
    a.last = last;
    a.n_layers = n_layers;
    a.layer_stride = layer_stride;
    a.cache = to_cache(cache);
    a.kv_lens = kv_lens;
    a.lens_out = lens_out;
    a.err = gdr::device_error_word();
    if (!a.err) return GDR_ERR_CUDA;
    return from_cuda(launch_compact(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
