// Attention of a few query rows per (sequence, KV head) over a paged KV cache:
// one token a sequence, or a few draft tokens.
//
//   out_r = sum_t softmax_t(scale q_r . K_t) V_t   over the positions t row r sees
//
// With at most 16 query rows every K and V byte is used at most 16 times, so
// the kernel is bound by reading the cache once. What it does about it:
//   - K and V go from memory straight to registers in the layout the MMA wants,
//     without shared memory: a dot product does not care about the order of its
//     dimensions, so lane (g, t) of a warp takes 16 consecutive bytes of key row
//     g (and of query row g) as its part of the k index; for P V it takes the
//     same 16 bytes of four value rows and pairs the rows with byte permutes.
//     Each load instruction covers whole 64- or 128-byte runs, a warp has 8 KB
//     in flight, and no barrier stands between a load and its use.
//   - The work is cut evenly: the units (8 KB of K and V) of all (row, head)
//     items form one line, and each CTA takes an equal piece of it, whatever the
//     lengths are. A CTA's four warps take its units in turn and merge their
//     softmax states (m, l, o) in shared memory at the end of an item. An item
//     that several CTAs share leaves partial states in the workspace (at most
//     two a CTA), which the join kernel adds up in order.
// The softmax runs on powers of two with a running maximum; the accumulators are
// rescaled only when a maximum rises. Weights enter the P V product as a BF16
// high part plus a BF16 remainder (2^-17 relative), so the result is FP32-exact
// up to the output's rounding; the extra MMAs are free in a memory-bound kernel.
#include <cuda_runtime.h>

#include <algorithm>

#include "paged_device.cuh"

namespace tiles {
namespace paged {

constexpr int kWarps = 4;
constexpr int kThr = kWarps * 32;
constexpr int kCtasPerSm = 3;
constexpr int kMinUnits = kWarps;  // a CTA's piece is at least one unit a warp

// What a CTA leaves about the item that it began and others finish: the number
// of partial states (0: none), the item, the slot of its own one.
struct JoinRec {
    int parts, s, tile, h, slot, pad[3];
};

__device__ __forceinline__ uint4 ld_stream16(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ld_stream8(const uint8_t *p) {
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
// The INT8 codes in bytes 0 and 2 of y (bytes 1 and 3: anything) as a BF16
// pair, exactly: (0x43, c & 127) - (0x43, c & 128) as BF16 numbers is c.
__device__ __forceinline__ uint32_t pair_codes(uint32_t y) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;"
        : "=r"(r)
        : "r"((y & 0x007F007Fu) | 0x43004300u), "r"((y & 0x00800080u) | 0x43004300u));
    return r;
}

// One (row, KV head, query tile) item's geometry.
struct Item {
    int t0, n, len;       // first token, tokens, length
    int head, lo;         // positions seen by some token: [0, head) and [lo, len)
    int nhu, wu0, nb;     // units of the head part, first unit of the rest, units in all
};
template <int UP>
__device__ __forceinline__ Item item_of(const AttnParams &p, int s, bool *bad) {
    const RowSpan r = row_span(p, s, bad);
    Item it;
    it.t0 = r.t0;
    it.n = r.n;
    it.len = r.len;
    visible_span(p, r.len, r.len - r.n, &it.head, &it.lo);
    it.nhu = (it.head + UP - 1) / UP;
    it.wu0 = it.lo / UP;
    if (it.nhu > it.wu0) it.nhu = it.wu0;
    it.nb = r.n > 0 ? it.nhu + (r.len + UP - 1) / UP - it.wu0 : 0;
    return it;
}

template <int D, bool I8, int RT>
struct Shape {
    static constexpr int EB = I8 ? 1 : 2;
    static constexpr int NB = I8 ? 256 / D : 128 / D;  // 16-position blocks a unit
    static constexpr int UP = 16 * NB;                 // positions a unit
    static constexpr int KC = D * EB / 64;             // 64-byte groups of a key row
    static constexpr int VW = I8 && D == 128 ? 16 : 8; // dimensions a lane takes of a value row and chunk
    static constexpr int VC = D / (8 * VW);            // chunks of a value row
    static constexpr int NS = D / 16;                  // k steps of Q K^T
    static constexpr int RH = RT / 8;                  // rows a lane holds
    static constexpr int LD = D + 4;                   // floats a row in the merge buffer (m, l behind o)
};

template <int D, bool I8, int RT>
__global__ void __launch_bounds__(kThr, kCtasPerSm) stream_kernel(const __grid_constant__ AttnParams p) {
    using S = Shape<D, I8, RT>;
    constexpr int NB = S::NB, UP = S::UP, RH = S::RH, LD = S::LD;
    __shared__ long long wsum[kWarps];
    __shared__ int found[2];
    __shared__ long long found_at;
    __shared__ __align__(16) float mg[kWarps][RT][LD];
    __shared__ int again[RT];
    const View &c = p.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    const int cta = blockIdx.x;
    JoinRec *recs = reinterpret_cast<JoinRec *>(p.ws);
    float *parts = p.ws + (size_t)p.ctas * (sizeof(JoinRec) / 4);
    if (tid == 0) recs[cta].parts = 0;

    // ---- where this CTA's piece of the line begins
    auto tiles_of = [&](const Item &it) { return (it.n * p.G + RT - 1) / RT; };
    const int per = (c.n_seqs + kThr - 1) / kThr, sa = tid * per, sb = min(c.n_seqs, sa + per);
    long long mine = 0;
    for (int s = sa; s < sb; ++s) {
        bool bad = false;
        const Item it = item_of<UP>(p, s, &bad);
        mine += (long long)it.nb * tiles_of(it) * c.nkv;
    }
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    long long before = x - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += wsum[w];
        total += wsum[w];
    }
    // pieces: as many as there are CTAs, but of no fewer than kMinUnits units
    const long long nc = min((long long)p.ctas, max(1ll, total / kMinUnits));
    const bool works = cta < nc && total > 0;
    const long long begin = works ? cta * total / nc : 0, end = works ? (cta + 1) * total / nc : 0;
    if (begin < end) {
        if (begin >= before && begin < before + mine) {  // one thread's rows hold the beginning
            long long at = before;
            int s = sa;
            for (; s < sb; ++s) {
                bool bad = false;
                const Item it = item_of<UP>(p, s, &bad);
                const long long u = (long long)it.nb * tiles_of(it) * c.nkv;
                if (begin < at + u) break;
                at += u;
            }
            found[0] = s;
            found_at = at;
        }
        __syncthreads();
        int s = found[0];
        long long at = found_at;  // line position of row s's first unit
        long long pos = begin;
        while (pos < end) {
            bool bad = false;
            const Item it = item_of<UP>(p, s, &bad);
            const int nt = tiles_of(it);
            const long long row_units = (long long)it.nb * nt * c.nkv;
            if (pos >= at + row_units) {
                at += row_units;
                ++s;
                continue;
            }
            const int idx = (int)((pos - at) / it.nb), h = idx / nt, tile = idx - h * nt;
            const long long item_at = at + (long long)idx * it.nb;
            const int b0 = (int)(pos - item_at), b1 = (int)min((long long)it.nb, end - item_at);
            const int r0 = tile * RT, rows = min(RT, it.n * p.G - r0);
            const int32_t *table = c.tables + (size_t)s * c.width;

            // ---- queries of rows g (and g + 8) in the MMA's k order
            uint32_t qf[RH][S::NS][2];
            int lim[RH];
#pragma unroll
            for (int rr = 0; rr < RH; ++rr) {
                const int r = r0 + g + 8 * rr;
                lim[rr] = -1;
#pragma unroll
                for (int i = 0; i < S::NS; ++i) qf[rr][i][0] = qf[rr][i][1] = 0u;
                if (g + 8 * rr < rows) {
                    const int tok = r / p.G;
                    lim[rr] = it.len - it.n + tok;
                    const uint16_t *q = p.q + (it.t0 + tok) * p.q_t + (long long)(h * p.G + r % p.G) * p.q_h;
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        const int dim = I8 ? 64 * (i / 2) + 16 * t4 + 8 * (i % 2) : 32 * i + 8 * t4;
                        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(q + dim));
                        qf[rr][2 * i][0] = w.x;
                        qf[rr][2 * i][1] = w.y;
                        qf[rr][2 * i + 1][0] = w.z;
                        qf[rr][2 * i + 1][1] = w.w;
                    }
                }
            }
            // positions every row sees: up to the first row's limit, from the last row's window on
            const int p_first = it.len - it.n + r0 / p.G, p_last = it.len - it.n + (r0 + rows - 1) / p.G;
            const int all_hi = p_first, all_lo = p.window > 0 ? p_last - p.window + 1 : 0;

            float o[S::VC * S::VW][2 * RH], m[RH], l[RH];
#pragma unroll
            for (int j = 0; j < S::VC * S::VW; ++j)
#pragma unroll
                for (int e = 0; e < 2 * RH; ++e) o[j][e] = 0.f;
#pragma unroll
            for (int rr = 0; rr < RH; ++rr) {
                m[rr] = -INFINITY;
                l[rr] = 0.f;
            }

            uint4 kr[NB][2][S::KC], vr[NB][4][S::VC];
            float2 ksc[I8 ? NB : 1][2], vsc[I8 ? NB : 1][2];
            auto unit_t0 = [&](int b) { return (b < it.nhu ? b : b - it.nhu + it.wu0) * UP; };
            // pool row of position tb (a multiple of 16), or -1: outside the length, or no page
            auto pool_row = [&](int tb) -> long long {
                if (tb >= it.len) return -1;
                const int page = __ldg(table + (tb >> c.psl));
                if (page < 0 || page >= c.n_pages) return -2;
                return ((long long)page * c.nkv + h) * c.ps + (tb & (c.ps - 1));
            };
            long long krow[NB], nrow[NB];
            auto load_k = [&](const long long (&row)[NB]) {
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
#pragma unroll
                        for (int cc = 0; cc < S::KC; ++cc) {
                            kr[i][a][cc] = make_uint4(0u, 0u, 0u, 0u);
                            if (row[i] >= 0)
                                kr[i][a][cc] =
                                    ld_stream16(c.k + (row[i] + 8 * a + g) * (D * S::EB) + 64 * cc + 16 * t4);
                        }
                        if constexpr (I8) {
                            ksc[i][a] = make_float2(0.f, 0.f);
                            if (row[i] >= 0)
                                ksc[i][a] = __ldg(reinterpret_cast<const float2 *>(c.ks + row[i] + 8 * a + 2 * t4));
                        }
                    }
            };
            auto load_v = [&](const long long (&row)[NB]) {
#pragma unroll
                for (int i = 0; i < NB; ++i) {
#pragma unroll
                    for (int a = 0; a < 4; ++a)
#pragma unroll
                        for (int cc = 0; cc < S::VC; ++cc) {
                            vr[i][a][cc] = make_uint4(0u, 0u, 0u, 0u);
                            if (row[i] >= 0) {
                                const uint8_t *v = c.v + (row[i] + 2 * t4 + (a & 1) + 8 * (a >> 1)) * (D * S::EB);
                                if constexpr (I8 && D == 64) {
                                    const uint2 w = ld_stream8(v + 8 * g);
                                    vr[i][a][cc].x = w.x;
                                    vr[i][a][cc].y = w.y;
                                } else {
                                    vr[i][a][cc] = ld_stream16(v + 128 * cc + 16 * g);
                                }
                            }
                        }
                    if constexpr (I8) {
#pragma unroll
                        for (int a = 0; a < 2; ++a) {
                            vsc[i][a] = make_float2(0.f, 0.f);
                            if (row[i] >= 0)
                                vsc[i][a] = __ldg(reinterpret_cast<const float2 *>(c.vs + row[i] + 8 * a + 2 * t4));
                        }
                    }
                }
            };

            if (b0 + warp < b1) {
#pragma unroll
                for (int i = 0; i < NB; ++i) krow[i] = pool_row(unit_t0(b0 + warp) + 16 * i);
                load_k(krow);
            }
            for (int b = b0 + warp; b < b1; b += kWarps) {
                const int t0 = unit_t0(b);
                load_v(krow);
                const bool more = b + kWarps < b1;
                if (more) {
#pragma unroll
                    for (int i = 0; i < NB; ++i) nrow[i] = pool_row(unit_t0(b + kWarps) + 16 * i);
                }
                // ---- scores
                float sc[NB][2][2 * RH];
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int cc = 0; cc < S::KC; ++cc) {
                            const uint32_t w[4] = {kr[i][a][cc].x, kr[i][a][cc].y, kr[i][a][cc].z, kr[i][a][cc].w};
#pragma unroll
                            for (int st = 0; st < (I8 ? 4 : 2); ++st) {
                                uint32_t k0, k1;
                                const int q = cc * (I8 ? 4 : 2) + st;
                                if constexpr (I8) {
                                    codes_bf16x2(w[st], k0, k1);
                                } else {
                                    k0 = w[2 * st];
                                    k1 = w[2 * st + 1];
                                }
                                if constexpr (RH == 1)
                                    mma_rows8(acc[0], acc[1], qf[0][q][0], qf[0][q][1], k0, k1);
                                else
                                    mma_m16n8k16(acc, qf[0][q][0], qf[RH - 1][q][0], qf[0][q][1], qf[RH - 1][q][1], k0,
                                                 k1);
                            }
                        }
                        float f0 = p.scale_log2, f1 = f0;
                        if constexpr (I8) {
                            f0 *= ksc[i][a].x;
                            f1 *= ksc[i][a].y;
                        }
#pragma unroll
                        for (int e = 0; e < 2 * RH; ++e) sc[i][a][e] = acc[e] * (e & 1 ? f1 : f0);
                    }
                if (more) load_k(nrow);
                // ---- mask, where some row does not see all of the unit
                bool holes = false;
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    holes |= krow[i] < 0;
                    if (krow[i] == -2 && lane == 0) atomicOr(reinterpret_cast<uint32_t *>(c.state), kDevBounds);
                }
                if (holes || t0 + UP - 1 > all_hi || t0 < all_lo) {
#pragma unroll
                    for (int i = 0; i < NB; ++i)
#pragma unroll
                        for (int a = 0; a < 2; ++a)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int t = t0 + 16 * i + 8 * a + 2 * t4 + e;
                                const bool any = krow[i] >= 0 && t < it.len && (t >= it.lo || t < it.head);
#pragma unroll
                                for (int rr = 0; rr < RH; ++rr) {
                                    const bool see = any && t <= lim[rr] &&
                                                     (p.window == 0 || t > lim[rr] - p.window || t < p.sinks);
                                    if (!see) sc[i][a][2 * rr + e] = -INFINITY;
                                }
                                // a value row that no row sees counts as zeros, whatever it holds
                                if (!any) {
#pragma unroll
                                    for (int cc = 0; cc < S::VC; ++cc) vr[i][2 * a + e][cc] = make_uint4(0u, 0u, 0u, 0u);
                                    if constexpr (I8) (e ? vsc[i][a].y : vsc[i][a].x) = 0.f;
                                }
                            }
                }
                // ---- running maximum, weights
                bool rise = false;
                float mn[RH];
#pragma unroll
                for (int rr = 0; rr < RH; ++rr) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int i = 0; i < NB; ++i)
#pragma unroll
                        for (int a = 0; a < 2; ++a) mx = fmaxf(mx, fmaxf(sc[i][a][2 * rr], sc[i][a][2 * rr + 1]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
                    mn[rr] = fmaxf(m[rr], mx);
                    rise |= mn[rr] > m[rr];
                }
                if (__any_sync(0xFFFFFFFFu, rise)) {
#pragma unroll
                    for (int rr = 0; rr < RH; ++rr) {
                        const float corr = mn[rr] > m[rr] ? ex2(m[rr] - mn[rr]) : 1.f;
                        m[rr] = mn[rr];
                        l[rr] *= corr;
#pragma unroll
                        for (int j = 0; j < S::VC * S::VW; ++j) {
                            o[j][2 * rr] *= corr;
                            o[j][2 * rr + 1] *= corr;
                        }
                    }
                }
                float base[RH];
#pragma unroll
                for (int rr = 0; rr < RH; ++rr) base[rr] = m[rr] == -INFINITY ? 0.f : m[rr];
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    uint32_t ph[RH][2], pl[RH][2];
#pragma unroll
                    for (int a = 0; a < 2; ++a)
#pragma unroll
                        for (int rr = 0; rr < RH; ++rr) {
                            float w0 = ex2(sc[i][a][2 * rr] - base[rr]), w1 = ex2(sc[i][a][2 * rr + 1] - base[rr]);
                            l[rr] += w0 + w1;
                            if constexpr (I8) {
                                w0 *= vsc[i][a].x;
                                w1 *= vsc[i][a].y;
                            }
                            const uint32_t hi = cvt_bf2(w0, w1);
                            ph[rr][a] = hi;
                            pl[rr][a] = cvt_bf2(w0 - bf_lo(hi), w1 - bf_hi(hi));
                        }
                    // ---- o += P V, one 8-column tile per dimension a lane holds
#pragma unroll
                    for (int cc = 0; cc < S::VC; ++cc) {
                        const uint32_t w[4][4] = {{vr[i][0][cc].x, vr[i][0][cc].y, vr[i][0][cc].z, vr[i][0][cc].w},
                                                  {vr[i][1][cc].x, vr[i][1][cc].y, vr[i][1][cc].z, vr[i][1][cc].w},
                                                  {vr[i][2][cc].x, vr[i][2][cc].y, vr[i][2][cc].z, vr[i][2][cc].w},
                                                  {vr[i][3][cc].x, vr[i][3][cc].y, vr[i][3][cc].z, vr[i][3][cc].w}};
#pragma unroll
                        for (int j = 0; j < S::VW; ++j) {
                            uint32_t v0, v1;
                            if constexpr (I8) {
                                // the codes of rows a and b in the low bytes of two halves, then to
                                // BF16 as codes_bf16x2 does
                                const uint32_t sel = 0x0400u + 0x0101u * (j % 4);
                                v0 = pair_codes(__byte_perm(w[0][j / 4], w[1][j / 4], sel));
                                v1 = pair_codes(__byte_perm(w[2][j / 4], w[3][j / 4], sel));
                            } else {
                                const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
                                v0 = __byte_perm(w[0][j / 2], w[1][j / 2], sel);
                                v1 = __byte_perm(w[2][j / 2], w[3][j / 2], sel);
                            }
                            float(&oj)[2 * RH] = o[cc * S::VW + j];
                            if constexpr (RH == 1) {
                                mma_rows8(oj[0], oj[1], ph[0][0], ph[0][1], v0, v1);
                                mma_rows8(oj[0], oj[1], pl[0][0], pl[0][1], v0, v1);
                            } else {
                                mma_m16n8k16(oj, ph[0][0], ph[1][0], ph[0][1], ph[1][1], v0, v1);
                                mma_m16n8k16(oj, pl[0][0], pl[1][0], pl[0][1], pl[1][1], v0, v1);
                            }
                        }
                    }
                }
                if (more) {
#pragma unroll
                    for (int i = 0; i < NB; ++i) krow[i] = nrow[i];
                }
            }

            // ---- merge the warps' states
#pragma unroll
            for (int rr = 0; rr < RH; ++rr) {
                l[rr] += __shfl_xor_sync(0xFFFFFFFFu, l[rr], 1);
                l[rr] += __shfl_xor_sync(0xFFFFFFFFu, l[rr], 2);
                float *dst = mg[warp][g + 8 * rr];
                if (t4 == 0) {
                    dst[D] = m[rr];
                    dst[D + 1] = l[rr];
                }
#pragma unroll
                for (int cc = 0; cc < S::VC; ++cc)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int j = 0; j < S::VW; j += 4) {
                            const int jj = cc * S::VW + j;
                            *reinterpret_cast<float4 *>(dst + cc * 8 * S::VW + S::VW * (2 * t4 + e) + j) =
                                make_float4(o[jj][2 * rr + e], o[jj + 1][2 * rr + e], o[jj + 2][2 * rr + e],
                                            o[jj + 3][2 * rr + e]);
                        }
            }
            if (tid < RT) again[tid] = 0;
            __syncthreads();
            const bool whole = b0 == 0 && b1 == it.nb;
            const int slot = pos == begin ? 0 : 1;
            if (!whole && b0 == 0 && tid == 0) {
                const long long last = ((item_at + it.nb) * nc + total - 1) / total - 1;  // the CTA with the item's end
                JoinRec r;
                r.parts = (int)(last - cta) + 1;
                r.s = s;
                r.tile = tile;
                r.h = h;
                r.slot = slot;
                r.pad[0] = r.pad[1] = r.pad[2] = 0;
                recs[cta] = r;
            }
            float *part = parts + (size_t)(2 * cta + slot) * RT * LD;
            constexpr int TPR = D / 4;  // threads a row, four dimensions each
            for (int i = tid; i < RT * TPR; i += kThr) {
                const int r = i / TPR, d0 = (i % TPR) * 4;
                if (r >= rows) break;
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) M = fmaxf(M, mg[w][r][D]);
                const float bs = M == -INFINITY ? 0.f : M;
                float L = 0.f;
                float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float f = ex2(mg[w][r][D] - bs);
                    const float4 v = *reinterpret_cast<const float4 *>(&mg[w][r][d0]);
                    L = fmaf(f, mg[w][r][D + 1], L);
                    O.x = fmaf(f, v.x, O.x);
                    O.y = fmaf(f, v.y, O.y);
                    O.z = fmaf(f, v.z, O.z);
                    O.w = fmaf(f, v.w, O.w);
                }
                if (whole) {
                    const float inv = L == 0.f ? 0.f : 1.f / L;
                    const int rr = r0 + r;
                    uint16_t *dst = p.out + (it.t0 + rr / p.G) * p.o_t + (long long)(h * p.G + rr % p.G) * p.o_h + d0;
                    *reinterpret_cast<uint2 *>(dst) =
                        make_uint2(cvt_bf2(O.x * inv, O.y * inv), cvt_bf2(O.z * inv, O.w * inv));
                    const float sum = fabsf(O.x) + fabsf(O.y) + fabsf(O.z) + fabsf(O.w) + L;
                    if (it.n > 1 && !(sum < INFINITY)) again[r] = 1;
                } else {
                    float *dst = part + r * LD;
                    if (d0 == 0) {
                        dst[D] = M;
                        dst[D + 1] = L;
                    }
                    *reinterpret_cast<float4 *>(dst + d0) = O;
                }
            }
            __syncthreads();  // the merge buffer is free again
            if (whole && it.n > 1)
                for (int r = warp; r < rows; r += kWarps)
                    if (again[r]) row_again<D, I8>(p, s, h, it.t0, it.n, it.len, r0 + r);
            pos = item_at + b1;
        }
    }
    // ---- rows that see nothing, and rows that break the rules
    for (int s = cta; s < c.n_seqs; s += gridDim.x) {
        bool bad = false;
        const Item it = item_of<UP>(p, s, &bad);
        if (bad && tid == 0) atomicOr(reinterpret_cast<uint32_t *>(c.state), kDevBounds);
        if (it.nb == 0)
            for (int i = tid; i < it.n * p.G * c.nkv * (D / 8); i += kThr) {
                const int r = i / (D / 8);
                *reinterpret_cast<uint4 *>(p.out + (it.t0 + r / (p.G * c.nkv)) * p.o_t +
                                           (long long)(r % (p.G * c.nkv)) * p.o_h + (i % (D / 8)) * 8) =
                    make_uint4(0u, 0u, 0u, 0u);
            }
    }
}

// Adds up the partial states of the item that CTA blockIdx.x began, for query
// row blockIdx.y of its tile: o = sum_i e^(m_i - M) o_i / sum_i e^(m_i - M) l_i.
// Four dimensions a thread; the states are dealt to the 512 / D groups of
// threads in turn, whose sums are then added in order.
template <int D, bool I8, int RT>
__global__ void __launch_bounds__(kThr) join_kernel(const __grid_constant__ AttnParams p) {
    using S = Shape<D, I8, RT>;
    constexpr int LD = S::LD, TPR = D / 4, GR = kThr / TPR;
    __shared__ float mx[kWarps];
    __shared__ __align__(16) float4 so[GR][TPR];
    __shared__ float sl[GR];
    __shared__ int bad_row;
    const int tid = threadIdx.x, cta = blockIdx.x, r = blockIdx.y;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const JoinRec rec = reinterpret_cast<const JoinRec *>(p.ws)[cta];
    if (rec.parts == 0) return;
    bool bad = false;
    const Item it = item_of<S::UP>(p, rec.s, &bad);
    const int row = rec.tile * RT + r;
    if (row >= it.n * p.G) return;
    const float *parts = p.ws + (size_t)p.ctas * (sizeof(JoinRec) / 4) + (size_t)r * LD;
    auto part = [&](int i) { return parts + (size_t)(2 * (cta + i) + (i == 0 ? rec.slot : 0)) * RT * LD; };
    float M = -INFINITY;
    for (int i = tid; i < rec.parts; i += kThr) M = fmaxf(M, __ldcg(part(i) + D));
    M = warp_max(M);
    if ((tid & 31) == 0) mx[tid >> 5] = M;
    if (tid == 0) bad_row = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, mx[w]);
    const float bs = M == -INFINITY ? 0.f : M;
    const int grp = tid / TPR, d0 = (tid % TPR) * 4;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
#pragma unroll 4
    for (int i = grp; i < rec.parts; i += GR) {
        const float *q = part(i);
        const float f = ex2(__ldcg(q + D) - bs);
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(q + d0));
        L = fmaf(f, __ldcg(q + D + 1), L);
        O.x = fmaf(f, v.x, O.x);
        O.y = fmaf(f, v.y, O.y);
        O.z = fmaf(f, v.z, O.z);
        O.w = fmaf(f, v.w, O.w);
    }
    so[grp][tid % TPR] = O;
    if (tid % TPR == 0) sl[grp] = L;
    __syncthreads();
    const int hq = rec.h * p.G + row % p.G, tok = it.t0 + row / p.G;
    if (grp == 0) {
        for (int k = 1; k < GR; ++k) {
            const float4 v = so[k][tid];
            O.x += v.x;
            O.y += v.y;
            O.z += v.z;
            O.w += v.w;
            L += sl[k];
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        *reinterpret_cast<uint2 *>(p.out + tok * p.o_t + hq * p.o_h + d0) =
            make_uint2(cvt_bf2(O.x * inv, O.y * inv), cvt_bf2(O.z * inv, O.w * inv));
        if (it.n > 1 && !(fabsf(O.x) + fabsf(O.y) + fabsf(O.z) + fabsf(O.w) + L < INFINITY)) bad_row = 1;
    }
    __syncthreads();
    if (bad_row && tid < 32) row_again<D, I8>(p, rec.s, rec.h, it.t0, it.n, it.len, row);
}

// ------------------------------------------------------------------ host side
size_t stream_ws_bytes(int sms, int d) {
    return (size_t)sms * kCtasPerSm * (sizeof(JoinRec) + (size_t)2 * 16 * (d + 4) * 4);
}

template <int D, bool I8, int RT>
static cudaError_t launch(const AttnParams &p, cudaStream_t st) {
    stream_kernel<D, I8, RT><<<p.ctas, kThr, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // the join's blocks may be set up while the last pieces are still at work
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)p.ctas, (unsigned)RT);
    cfg.blockDim = dim3(kThr);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel<D, I8, RT>, p);
}

cudaError_t stream_launch(const AttnParams &p0, int sms, cudaStream_t st) {
    AttnParams p = p0;
    p.ctas = sms * kCtasPerSm;
    const bool small = p.max_tokens * p.G <= 8;
    if (p.c.d == 64) {
        if (p.c.i8) return small ? launch<64, true, 8>(p, st) : launch<64, true, 16>(p, st);
        return small ? launch<64, false, 8>(p, st) : launch<64, false, 16>(p, st);
    }
    if (p.c.i8) return small ? launch<128, true, 8>(p, st) : launch<128, true, 16>(p, st);
    return small ? launch<128, false, 8>(p, st) : launch<128, false, 16>(p, st);
}

}  // namespace paged
}  // namespace tiles
