// Causal attention over whole packed prompts.
//
// One warp per query row: the running maximum m and sum l of the softmax and the
// row's output in fp32, one token at a time.
#include "gdr_attn_common.cuh"
#include "gdr_internal.h"

namespace gdr {
namespace attn {
namespace {

template <int D, bool F16>
__global__ void __launch_bounds__(128) prefill_rows_kernel(const __grid_constant__ Args a) {
    constexpr int W = D / 64;  // 32-bit words per lane
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= a.t_total * a.h_q) return;
    const int64_t t = row / a.h_q;
    const int h = (int)(row - t * a.h_q);
    const int s = find_seq(a.cu, a.n_seqs, t);
    const int64_t t0 = a.cu[s], t1 = a.cu[s + 1];
    if (t0 < 0 || t < t0 || t1 <= t || t1 > a.t_total) {
        record_invalid(a.err);
        return;
    }
    float2 q[W], o[W];
    const uint32_t *qp = reinterpret_cast<const uint32_t *>(a.q.p + t * a.q.ts + h * a.q.hs);
#pragma unroll
    for (int i = 0; i < W; ++i) {
        q[i] = unpack2<F16>(qp[lane + 32 * i]);
        o[i] = make_float2(0.f, 0.f);
    }
    float m = -CUDART_INF_F, l = 0.f;
    for (int64_t p = t0; p <= t; ++p) {
        const uint32_t *kp = reinterpret_cast<const uint32_t *>(a.k.p + p * a.k.ts + (h / a.group) * a.k.hs);
        const uint32_t *vp = reinterpret_cast<const uint32_t *>(a.v.p + p * a.v.ts + (h / a.group) * a.v.hs);
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float2 k = unpack2<F16>(kp[lane + 32 * i]);
            x += q[i].x * k.x + q[i].y * k.y;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        x *= a.scale;
        const float mn = fmaxf(m, x);
        const float c = m == mn ? 1.f : __expf(m - mn), w = __expf(x - mn);
        l = l * c + w;
        m = mn;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float2 v = unpack2<F16>(vp[lane + 32 * i]);
            o[i].x = o[i].x * c + w * v.x;
            o[i].y = o[i].y * c + w * v.y;
        }
    }
    uint32_t *op = reinterpret_cast<uint32_t *>(a.o.p + t * a.o.ts + h * a.o.hs);
    const float r = 1.f / l;
#pragma unroll
    for (int i = 0; i < W; ++i) op[lane + 32 * i] = pack2<F16>(o[i].x * r, o[i].y * r);
    if (a.lse && lane == 0) a.lse[row] = m + logf(l);
}

template <int D>
void launch(const Args &a, cudaStream_t s) {
    const unsigned blocks = (unsigned)((a.t_total * a.h_q + 3) / 4);
    if (a.f16)
        prefill_rows_kernel<D, true><<<blocks, 128, 0, s>>>(a);
    else
        prefill_rows_kernel<D, false><<<blocks, 128, 0, s>>>(a);
}

}  // namespace

cudaError_t launch_prefill(const Args &a, cudaStream_t s) {
    if (a.d == 64)
        launch<64>(a, s);
    else if (a.d == 128)
        launch<128>(a, s);
    else
        launch<256>(a, s);
    return cudaGetLastError();
}

}  // namespace attn
}  // namespace gdr
