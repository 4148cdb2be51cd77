// Asynchronous 16-byte copies and warp-level MMAs of the attention kernels that work on
// few rows (decode, short prompts).
#pragma once

#include <stdint.h>

namespace gdr {
namespace attn {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// One of the barrier's arrivals, when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// True where a 16-bit value is an infinity or NaN.
template <bool F16>
__device__ __forceinline__ bool nonfinite(uint32_t half_word) {
    constexpr uint32_t e = F16 ? 0x7C00u : 0x7F80u;
    return (half_word & e) == e;
}
// True if any of eight is: only an exponent of ones carries into its value's top bit.
template <bool F16>
__device__ __forceinline__ bool any_nonfinite(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    constexpr uint32_t e = F16 ? 0x7C007C00u : 0x7F807F80u, one = F16 ? 0x04000400u : 0x00800080u;
    return ((((a & e) + one) | ((b & e) + one) | ((c & e) + one) | ((d & e) + one)) & 0x80008000u) != 0;
}
// The word with infinities and NaNs replaced by zeros.
template <bool F16>
__device__ __forceinline__ uint32_t cleaned(uint32_t w) {
    return w & (nonfinite<F16>(w) ? 0xFFFF0000u : ~0u) & (nonfinite<F16>(w >> 16) ? 0xFFFFu : ~0u);
}

}  // namespace attn
}  // namespace gdr
