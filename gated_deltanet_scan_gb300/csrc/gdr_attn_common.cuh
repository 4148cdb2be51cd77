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

// Sequence of token t among packed starts cu[0 .. n]: the last s with cu[s] <= t.
__device__ __forceinline__ int find_seq(const int32_t *cu, int n, int64_t t) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

}  // namespace attn
}  // namespace gdr
