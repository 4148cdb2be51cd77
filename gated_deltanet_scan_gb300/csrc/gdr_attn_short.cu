// Causal attention of short prompts (short_tokens).
//
// The two-SM tcgen05 kernel works on blocks of 256 rows with a start of microseconds; a
// batch of prompts of a few dozen tokens leaves it mostly waiting (32 prompts of 64 tokens,
// 16 heads of 128: 36 us, here 13).  Here a block of four warps takes 64 rows of one
// sequence and key/value head (rows token by token, the group's heads within a token),
// several blocks an SM, with warp-level m16n8k16 MMAs and the formulas of
// gdr_attn_prefill.cu: x = sc Q K^T, p = 2^(x - m), l += sum p, O += P V over tiles of 32
// tokens.  Tiles come in by 16-byte asynchronous copies, one tile ahead.  Bound by
// latency: at these lengths a block sees a few tiles.
#include "gdr_attn_common.cuh"
#include "gdr_attn_mma.cuh"
#include "gdr_internal.h"
#include "tc_ptx.cuh"

namespace gdr {
namespace attn {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 64;  // rows per block
constexpr int kTile = 32;  // tokens per tile

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads) short_kernel(const __grid_constant__ Args a) {
    constexpr int KS = D / 16, NT = D / 8, CPR = D / 8;
    constexpr uint32_t TILE = kTile * D * 2;  // bytes of a key or value tile
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = tc::smem_u32(smem);
    const float sc = a.scale * kLog2e;
    const int r0 = lane >> 2, cq = lane & 3;

    int lo = 0;          // sequences before this one are behind
    int64_t before = 0;  // and their blocks (of one head)
    for (int64_t number = blockIdx.x;; number += gridDim.x) {
        // --- the block: every warp looks for itself, 32 sequences at a time
        const int64_t want = number >> 31 ? number / a.h_kv : (int64_t)((uint32_t)number / (uint32_t)a.h_kv);
        const int h = (int)(number - want * a.h_kv);
        int64_t t0 = 0;
        int len = 0, block = -1;
        while (lo < a.n_seqs) {
            const int s = lo + lane;
            int64_t b = 0, e = 0;
            if (s < a.n_seqs) {
                b = a.cu[s];
                e = a.cu[s + 1];
                if (b < 0 || e < b || e > a.t_total) {
                    record_invalid(a.err);
                    b = e = 0;
                }
            }
            const int n = e - b <= short_tokens(a.group) ? ((int)(e - b) * a.group + kRows - 1) / kRows : 0;
            int x = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            const int64_t end = before + x;
            const uint32_t hit = __ballot_sync(0xffffffffu, want >= end - n && want < end);
            if (hit) {
                const int src = __ffs(hit) - 1;
                t0 = __shfl_sync(0xffffffffu, b, src);
                len = (int)(__shfl_sync(0xffffffffu, e, src) - t0);
                block = (int)(want - __shfl_sync(0xffffffffu, end - n, src));
                break;
            }
            before += __shfl_sync(0xffffffffu, x, 31);
            lo += 32;
        }
        if (block < 0) break;  // the same in every warp

        const int last_token = min(len - 1, (block * kRows + kRows - 1) / a.group);
        const int tiles = last_token / kTile + 1;
        auto load = [&](int tile) {
            if (tile < tiles) {
                const uint32_t kb = base + (tile & 1) * 2 * TILE;
#pragma unroll
                for (int i = 0; i < kTile * CPR / kThreads; ++i) {
                    const int x = i * kThreads + tid, row = x / CPR, chunk = x % CPR;
                    const int p = tile * kTile + row;
                    const bool there = p < len;
                    const int64_t t = t0 + (there ? p : 0);
                    const uint32_t to = row * (D * 2) + ((chunk ^ (row & 7)) << 4);
                    cp_async16(kb + to, a.k.p + t * a.k.ts + h * a.k.hs + chunk * 8, there ? 16u : 0u);
                    cp_async16(kb + TILE + to, a.v.p + t * a.v.ts + h * a.v.hs + chunk * 8, there ? 16u : 0u);
                }
            }
            cp_async_commit();
        };
        load(0);

        uint32_t qf[KS][4];
        int64_t out_row[2];
        int token[2];  // of the row, or -1
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = block * kRows + warp * 16 + r0 + 8 * i;
            const int t = r / a.group, g = r - t * a.group;
            const bool live = t < len;
            token[i] = live ? t : -1;
            out_row[i] = (t0 + t) * a.h_q + h * a.group + g;
            const uint16_t *const src = a.q.p + (t0 + (live ? t : 0)) * a.q.ts + (int64_t)(h * a.group + g) * a.q.hs;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qf[k][i] = live ? *reinterpret_cast<const uint32_t *>(src + k * 16 + cq * 2) : 0u;
                qf[k][2 + i] = live ? *reinterpret_cast<const uint32_t *>(src + k * 16 + 8 + cq * 2) : 0u;
            }
        }
        const int warp_first = (block * kRows + warp * 16) / a.group;  // tokens of this warp's rows
        const int warp_last = min(len - 1, (block * kRows + warp * 16 + 15) / a.group);
        const int block_first = block * kRows / a.group;

        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
        float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};

        for (int tile = 0; tile < tiles; ++tile) {
            const int p0 = tile * kTile;
            load(tile + 1);
            cp_async_wait<1>();
            __syncthreads();
            const uint32_t kb = base + (tile & 1) * 2 * TILE, vb = kb + TILE;

            // Rows that do not see a token have p = 0 for it, and 0 times an infinity or NaN would reach
            // them: in a tile that some row sees only in part such values are added to the rows that see
            // them (p > 0 leaves them as they are) and replaced by zeros.
            bool found = false;
            if (p0 + kTile - 1 > block_first) {
                for (int i = tid; i < kTile * D / 8; i += kThreads) {
                    uint32_t w[4];
                    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                 : "r"(vb + 16 * i)
                                 : "memory");
                    found = found || any_nonfinite<F16>(w[0], w[1], w[2], w[3]);
                }
                found = __syncthreads_or(found);
                if (found) {
#pragma unroll 1
                    for (int t = 0; t < kTile && p0 + t < len; ++t) {
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            uint32_t w;
                            asm volatile("ld.shared.b32 %0, [%1];"
                                         : "=r"(w)
                                         : "r"(vb + t * (D * 2) + ((n ^ (t & 7)) << 4) + cq * 4)
                                         : "memory");
                            if (!nonfinite<F16>(w) && !nonfinite<F16>(w >> 16)) continue;
                            const float2 v = unpack2<F16>(w);
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                if (p0 + t > token[i]) continue;
                                if (nonfinite<F16>(w)) acc[n][2 * i] += v.x;
                                if (nonfinite<F16>(w >> 16)) acc[n][2 * i + 1] += v.y;
                            }
                        }
                    }
                    __syncthreads();
                    for (int i = tid; i < kTile * D / 2; i += kThreads) {
                        uint32_t w;
                        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(vb + 4 * i) : "memory");
                        const uint32_t z = cleaned<F16>(w);
                        if (z != w) asm volatile("st.shared.b32 [%0], %1;" ::"r"(vb + 4 * i), "r"(z) : "memory");
                    }
                    __syncthreads();
                }
            }

            if (p0 <= warp_last) {  // some row of the warp sees some token of the tile
                float x[4][4];
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i >> 2][i & 3] = 0.f;
                {
                    const int row = (lane & 7) + ((lane >> 4) << 3);
                    uint32_t at[4];  // chunk (2 k + b) ^ (row & 7), b = (lane >> 3) & 1
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        at[i] = kb + row * (D * 2) + (((2 * i) ^ ((lane >> 3) & 1) ^ (row & 7)) << 4);
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
#pragma unroll
                        for (int t = 0; t < 4; t += 2) {
                            uint32_t b[4];
                            ldsm4(at[k & 3] + t * 8 * D * 2 + (k >> 2) * 128, b);
                            mma16816<F16>(x[t], qf[k], b[0], b[1]);
                            mma16816<F16>(x[t + 1], qf[k], b[2], b[3]);
                        }
                    }
                }
                const bool masked = p0 + kTile - 1 > warp_first;
                uint32_t pf[2][4];
                float c[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        v[e] = sc * x[e >> 1][2 * i + (e & 1)];
                        if (masked && p0 + (e >> 1) * 8 + cq * 2 + (e & 1) > token[i]) v[e] = -CUDART_INF_F;
                    }
                    float top = v[0];
#pragma unroll
                    for (int e = 1; e < 8; ++e) top = fmaxf(top, v[e]);
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const float mn = next_reference<F16>(m[i], top);
                    const float ref = mn == -CUDART_INF_F ? 0.f : mn;
                    // the first tile's factor is 1, not 2^-inf = 0: the sums may hold added infinities
                    c[i] = m[i] == mn || m[i] == -CUDART_INF_F ? 1.f : tc::fast_exp2(m[i] - ref);
                    m[i] = mn;
                    l[i] *= c[i];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p = tc::fast_exp2(v[2 * e] - ref), q = tc::fast_exp2(v[2 * e + 1] - ref);
                        l[i] += p + q;
                        pf[e >> 1][(e & 1) * 2 + i] = pack2<F16>(p, q);
                    }
                }
                if (__any_sync(0xffffffffu, c[0] != 1.f || c[1] != 1.f)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        acc[n][0] *= c[0];
                        acc[n][1] *= c[0];
                        acc[n][2] *= c[1];
                        acc[n][3] *= c[1];
                    }
                }
                {
                    const int row = lane & 15;
                    uint32_t at[4];  // chunk (n + (lane >> 4)) ^ (row & 7)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        at[i] = vb + row * (D * 2) + (((2 * i) ^ (lane >> 4) ^ (row & 7)) << 4);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
#pragma unroll
                        for (int n = 0; n < NT; n += 2) {
                            uint32_t b[4];
                            ldsm4t(at[(n >> 1) & 3] + t * 16 * D * 2 + (n >> 3) * 128, b);
                            mma16816<F16>(acc[n], pf[t], b[0], b[1]);
                            mma16816<F16>(acc[n + 1], pf[t], b[2], b[3]);
                        }
                    }
                }
            }
            __syncthreads();  // the tile's place is loaded again two tiles on
        }
        cp_async_wait<0>();  // only empty groups are left

#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            if (token[i] < 0) continue;
            const float inv = inverse_sum(l[i]);
            const int64_t t = t0 + token[i];
            uint16_t *const dst = a.o.p + t * a.o.ts + (out_row[i] - t * a.h_q) * a.o.hs;
#pragma unroll
            for (int n = 0; n < NT; ++n)
                *reinterpret_cast<uint32_t *>(dst + n * 8 + cq * 2) =
                    pack2<F16>(acc[n][2 * i] * inv, acc[n][2 * i + 1] * inv);
            if (a.lse && cq == 0) a.lse[out_row[i]] = kLn2 * (m[i] + log2f(l[i]));
        }
        __syncwarp();
    }
    // nothing here reads what the kernel before writes, but work after this waits for both
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int D, bool F16>
cudaError_t launch(const Args &a, bool after, cudaStream_t s) {
    constexpr int bytes = 4 * kTile * D * 2;
    static SmemOptIn opt_in;
    cudaError_t e = opt_in.set(reinterpret_cast<const void *>(short_kernel<D, F16>), bytes);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (a.t_total * a.group / kRows + a.n_seqs) * a.h_kv;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks < 152 * 4 ? blocks : 152 * 4));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = after ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, short_kernel<D, F16>, a);
}

}  // namespace

cudaError_t launch_prefill_short(const Args &a, bool after, cudaStream_t s) {
    if (a.d == 64) return a.f16 ? launch<64, true>(a, after, s) : launch<64, false>(a, after, s);
    if (a.d == 128) return a.f16 ? launch<128, true>(a, after, s) : launch<128, false>(a, after, s);
    return a.f16 ? launch<256, true>(a, after, s) : launch<256, false>(a, after, s);
}

}  // namespace attn
}  // namespace gdr
