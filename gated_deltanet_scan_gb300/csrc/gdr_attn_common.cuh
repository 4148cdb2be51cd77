// Device helpers shared by the attention kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "gdr_attn.h"

namespace gdr {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void record_invalid(int32_t *err) { atomicCAS(err, 0, (int32_t)GDR_ERR_INVALID_ARG); }

// Two 16-bit values of a word as floats, and back (round to nearest even).
template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (F16) {
        return __half22float2(*reinterpret_cast<__half2 *>(&w));
    } else {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (F16) {
        __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    } else {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    }
}
template <bool F16>
__device__ __forceinline__ float unpack1(uint16_t w) {
    if constexpr (F16)
        return __half2float(*reinterpret_cast<__half *>(&w));
    else
        return __uint_as_float((uint32_t)w << 16);
}

// Two weights p >= 0 as bf16 pairs whose sum holds 16 bits of them: cut to bf16, and the rest
// rounded to it.  The rest is taken of p (1 + 2^-23), so that neither part is 0 (from 2^-103
// up) and an infinite value times either is that infinity.
__device__ __forceinline__ void split2(float a, float b, uint32_t &cut, uint32_t &rest) {
    constexpr float kOver = 1.00000011920928955f;  // 1 + 2^-23
    cut = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
    rest = pack2<false>(fmaf(a, kOver, -__uint_as_float(cut << 16)), fmaf(b, kOver, -__uint_as_float(cut & 0xFFFF0000u)));
}

// The reference m of a row's weights p = 2^(x - m), which enter P V in 16 bits.  Sums are
// rescaled when m moves, so it follows the row's maximum only when that is TOP above it,
// and is then LEAD under it.  bf16 rounds weights of any size relative to themselves.  fp16
// does so from 2^-14 up, and its largest value is just under 2^16: with weights of up to
// 2^TOP = 2^15, those of a row's other tokens keep their accuracy down to 2^-22 of the
// largest one and are lost below 2^-33, at no cost (a reference at the maximum itself:
// 2^-14 and 2^-25, which many tokens of little weight add up to).
template <bool F16>
struct Reference {
    static constexpr float LEAD = F16 ? 8.f : 0.f, TOP = F16 ? 15.f : 8.f;
};
template <bool F16>
__device__ __forceinline__ float next_reference(float m, float top) {
    using R = Reference<F16>;
    return top > m + R::TOP || m == -CUDART_INF_F ? fmaxf(m, top - R::LEAD) : m;
}

// Factor of scores that are masked before it is applied: scale log2(e) without its sign.  A
// scale of 0 still has to leave a masked score at minus infinity, so the smallest float
// stands in for it: times any finite score that stays under 2^-21, a weight of 1.
__device__ __forceinline__ float softmax_scale(float scale) {
    return fmaxf(fabsf(scale) * kLog2e, __uint_as_float(1u));
}

// 1 / l for the output o = O / l; a row without a finite score (it sees no token, or its
// scores are all minus infinity) has l = 0 and O = 0, and gives o = 0 and lse = ln 0.
__device__ __forceinline__ float inverse_sum(float l) { return 1.f / (l == 0.f ? 1.f : l); }

// Sequence of token t among packed starts cu[0 .. n]: the last s < n with cu[s] <= t (or
// 0).  The whole warp looks, 32 places at a time: two rounds of loads for a thousand.
__device__ __forceinline__ int find_seq_warp(const int32_t *cu, int n, int64_t t, int lane) {
    int lo = 0, hi = n;  // the answer is in [lo, hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;
        const uint32_t below = __ballot_sync(0xffffffffu, at < hi && cu[at] <= t);
        const int k = below ? 31 - __clz(below) : 0;
        lo += k * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

}  // namespace attn
}  // namespace gdr
