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

// Row r of (s, h) again, position by position with nothing but what it sees:
// for rows whose matrix product met an infinity or NaN in a value row that only
// other rows of the tile see (0 * inf). One warp; D / 32 dimensions a lane;
// writes dimensions [d0, d1).
template <int D, bool I8>
__device__ __noinline__ void row_again(const AttnParams &p, int s, int h, int t0, int n, int len, int r, int d0 = 0, int d1 = D) {
    constexpr int E = D / 32;
    const View &c = p.c;
    const int lane = threadIdx.x & 31, tok = r / p.G, pos = len - n + tok, hq = h * p.G + r % p.G;
    const uint16_t *q = p.q + (t0 + tok) * p.q_t + hq * p.q_h;
    float qf[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        qf[e] = bf2f(q[lane * E + e]);
        o[e] = 0.f;
    }
    for (int pass = 0; pass < 2; ++pass)
        for (int t = 0; t <= pos && t < len; ++t) {
            if (p.window > 0 && t <= pos - p.window && t >= p.sinks) continue;
            const int page = c.tables[(size_t)s * c.width + (t >> c.psl)];
            if (page < 0 || page >= c.n_pages) continue;
            const size_t at = ((size_t)page * c.nkv + h) * c.ps + (t & (c.ps - 1));
            float x = 0.f, v[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const size_t i = at * D + lane * E + e;
                const float kf = I8 ? (float)reinterpret_cast<const int8_t *>(c.k)[i]
                                    : bf2f(reinterpret_cast<const uint16_t *>(c.k)[i]);
                v[e] = I8 ? (float)reinterpret_cast<const int8_t *>(c.v)[i] * c.vs[at]
                          : bf2f(reinterpret_cast<const uint16_t *>(c.v)[i]);
                x = fmaf(qf[e], kf, x);
            }
            x = warp_sum(x) * p.scale_log2;
            if (I8) x *= c.ks[at];
            if (pass == 0) {
                m = x > m || x != x ? x : m;
            } else {
                const float w = exp2f(x - (m == -INFINITY ? 0.f : m));
                l += w;
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = fmaf(w, v[e], o[e]);
            }
        }
    uint16_t *out = p.out + (t0 + tok) * p.o_t + hq * p.o_h;
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (lane * E + e >= d0 && lane * E + e < d1) out[lane * E + e] = l == 0.f ? 0 : f2bf(o[e] / l);
}

}  // namespace paged
}  // namespace tiles
