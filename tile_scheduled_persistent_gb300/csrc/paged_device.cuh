// Device helpers shared by the two attention kernels over a paged KV cache.
#pragma once

#include "megakernel.cuh"
#include "paged_internal.h"

namespace tiles {
namespace paged {

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t cvt_bf2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Row r of (s, h) again, with nothing but what it sees: for rows whose matrix product
// met an infinity or NaN in a value row that only other rows of the tile see (0 * inf).
// One warp, in two passes (maximum; weights and values): a position a lane for the
// scores, D / 32 dimensions a lane for the values: 24 ms over 32,768 positions (D 128).
template <int D, bool I8>
__device__ __noinline__ void row_again(const AttnParams &p, int s, int h, int t0, int n, int len, int r) {
    constexpr int E = D / 32;
    const View &c = p.c;
    const int lane = threadIdx.x & 31, tok = r / p.G, pos = len - n + tok, hq = h * p.G + r % p.G;
    const int end = min(pos + 1, len), lo = p.window > 0 ? pos - p.window + 1 : 0;  // [lo, end) and the sinks
    const uint16_t *q = p.q + (t0 + tok) * p.q_t + hq * p.q_h;
    float o[E], m = -INFINITY, base = 0.f, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int pass = 0; pass < 2; ++pass) {
        for (int tb = 0; tb < end; tb += 32) {
            if (tb >= p.sinks && tb + 32 <= lo) {
                tb = (lo & ~31) - 32;
                continue;
            }
            const int t = tb + lane;
            int page = -1;
            if (t < end && (t >= lo || t < p.sinks)) page = c.tables[(size_t)s * c.width + (t >> c.psl)];
            const bool see = page >= 0 && page < c.n_pages;
            const size_t at = see ? ((size_t)page * c.nkv + h) * c.ps + (t & (c.ps - 1)) : 0;
            float x = -INFINITY;
            if (see) {
                x = 0.f;
#pragma unroll 4
                for (int d = 0; d < D; d += 8) {
                    float qf[8], kf[8];
                    unpack8(*reinterpret_cast<const uint4 *>(q + d), qf);
                    if (I8) {
                        const uint2 k = *reinterpret_cast<const uint2 *>(c.k + at * D + d);
#pragma unroll
                        for (int i = 0; i < 8; ++i) kf[i] = (float)(int8_t)((i < 4 ? k.x : k.y) >> (8 * (i % 4)));
                    } else {
                        unpack8(*reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(c.k) + at * D + d), kf);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) x = fmaf(qf[i], kf[i], x);
                }
                x *= p.scale_log2;
                if (I8) x *= c.ks[at];
            }
            if (pass == 0) {
                m = x > m || x != x ? x : m;
                continue;
            }
            float w = see ? exp2f(x - base) : 0.f;
            l += w;
            if (I8 && see) w *= c.vs[at];
            const uint32_t seen = __ballot_sync(0xFFFFFFFFu, see);
#pragma unroll 8
            for (int j = 0; j < 32; ++j) {  // (a position that is not seen reads the pool's first row)
                const float wj = __shfl_sync(0xFFFFFFFFu, w, j);
                const size_t i = __shfl_sync(0xFFFFFFFFu, (unsigned long long)at, j) * D + lane * E;
                uint32_t v[E / 2];
#pragma unroll
                for (int e = 0; e < E / 2; ++e)
                    v[e] = I8 ? (uint32_t)*reinterpret_cast<const uint16_t *>(c.v + i + 2 * e)
                              : *reinterpret_cast<const uint32_t *>(c.v + 2 * i + 4 * e);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const uint32_t x2 = (seen >> j) & 1u ? v[e / 2] : 0u;
                    const float ve = I8 ? (float)(int8_t)(x2 >> (8 * (e & 1))) : e & 1 ? bf_hi(x2) : bf_lo(x2);
                    o[e] = fmaf(wj, ve, o[e]);
                }
            }
        }
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) {
            const float y = __shfl_xor_sync(0xFFFFFFFFu, m, k);
            m = y > m || y != y ? y : m;
        }
        base = m == -INFINITY ? 0.f : m;
    }
    l = warp_sum(l);
    uint16_t *out = p.out + (t0 + tok) * p.o_t + hq * p.o_h;
#pragma unroll
    for (int e = 0; e < E; ++e)
        out[lane * E + e] = l == 0.f ? 0 : f2bf(o[e] / l);
}

}  // namespace paged
}  // namespace tiles
