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
//
// INT8 cache: the codes are widened to FP16 (exactly: a byte permute and one
// subtraction a pair), so the MMAs take FP16. Queries are scaled by a power of two
// to below 2 (exact; what falls under 2^-24 of the largest is rounded). A weight
// times its value's scale enters as one FP16 number, 2^12 at most and relative to a
// power of two not below the largest scale so far: 2^-12 relative, 2^-37 of the
// largest absolute. Widening is what bounds this form, hence no remainder here.
//
// Measured on GB300: 64 rows of 32,768 (D 128, 32/8 heads) 1,316 us, 6.53 TB/s, 0.96 of
// the measured copy rate; 32 rows of 1-4,096 (16/8 heads) 54.7 us, 4.87 TB/s; one row of
// 1,024 (D 64) 10.2 us; INT8, 64 rows of up to 32,768 under a window of 4,096 (D 64)
// 76.6 us, 3.46 TB/s. (The join by the CTA that comes last, without a launch of its own:
// 1,358, 60 and 10.2 us, as its registers weigh on the loop.)
#include <cuda_runtime.h>

#include <algorithm>

#include "paged_device.cuh"

namespace tiles {
namespace paged {

constexpr int kWarps = 4;
constexpr int kThr = kWarps * 32;
// What 168 registers a thread allow. (An INT8 cache with 4 CTAs of 128 registers, which
// spill: 82 us in place of 77 for 64 rows of up to 32,768 under a window of 4,096.)
constexpr int kCtasPerSm = 3;
// The line counts an item as its units and kItemCost for its queries, its first loads and
// its merge (about 4 us, in which a CTA takes 8 units); a piece is at least kMinCost.
constexpr int kItemCost = 8, kMinCost = kWarps;

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
// INT8 codes as FP16 numbers, exactly: the byte c + 128 below 0x64 is 1024 + (c + 128),
// and 1152 less is c. half_codes: bytes 0 and 2 of the two halves already under 0x64.
__device__ __forceinline__ uint32_t half_codes(uint32_t biased) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(biased), "r"(0x64806480u));
    return r;
}
__device__ __forceinline__ uint32_t cvt_h2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// mma_rows8 and mma_m16n8k16 with FP16 operands
__device__ __forceinline__ void mma_rows8_h(float &c0, float &c1, uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1) {
    asm volatile("{\n\t.reg .f32 z2, z3;\n\t"
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, z2, z3}, {%2, %6, %3, %6}, {%4, %5},"
        " {%0, %1, %7, %7};\n\t}"
        : "+f"(c0), "+f"(c1)
        : "r"(a0), "r"(a2), "r"(b0), "r"(b1), "r"(0u), "f"(0.f));
}
__device__ __forceinline__ void mma_m16n8k16_h(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
        " {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One (row, KV head, query tile) item's geometry.
struct Item {
    int t0, n, len;       // first token, tokens, length
    int head, lo;         // positions seen by some token: [0, head) and [lo, len)
    int nhu, wu0, nb;     // units of the head part, first unit of the rest, units in all
    __device__ __forceinline__ int cost() const { return nb ? nb + kItemCost : 0; }
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
    static constexpr int NB = 128 / D;                 // 16-position blocks a unit
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
    after_previous();
    if (tid == 0) recs[cta].parts = 0;

    // ---- where this CTA's piece of the line begins
    auto tiles_of = [&](const Item &it) { return (it.n * p.G + RT - 1) / RT; };
    const int per = (c.n_seqs + kThr - 1) / kThr, sa = tid * per, sb = min(c.n_seqs, sa + per);
    long long mine = 0;
    for (int s = sa; s < sb; ++s) {
        bool bad = false;
        const Item it = item_of<UP>(p, s, &bad);
        mine += (long long)it.cost() * tiles_of(it) * c.nkv;
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
    // pieces: as many as there are CTAs, but not too small
    const long long nc = min((long long)p.ctas, max(1ll, total / kMinCost));
    const bool works = cta < nc && total > 0;
    const long long begin = works ? cta * total / nc : 0, end = works ? (cta + 1) * total / nc : 0;
    if (begin < end) {
        if (begin >= before && begin < before + mine) {  // one thread's rows hold the beginning
            long long at = before;
            int s = sa;
            for (; s < sb; ++s) {
                bool bad = false;
                const Item it = item_of<UP>(p, s, &bad);
                const long long u = (long long)it.cost() * tiles_of(it) * c.nkv;
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
        bool first = true;  // no item with units so far
        while (pos < end) {
            bool bad = false;
            const Item it = item_of<UP>(p, s, &bad);
            const int nt = tiles_of(it);
            const int cost = it.cost();
            const long long row_units = (long long)cost * nt * c.nkv;
            if (pos >= at + row_units) {
                at += row_units;
                ++s;
                continue;
            }
            const int idx = (int)((pos - at) / cost), h = idx / nt, tile = idx - h * nt;
            // of an item that begins at cost unit 0, cost unit kItemCost + b is unit b
            const long long item_at = at + (long long)idx * cost, upto = min(item_at + cost, end);
            const int b0 = max(0, (int)(pos - item_at) - kItemCost), b1 = (int)(upto - item_at) - kItemCost;
            if (b1 <= b0) {  // only the item's first cost units: the next CTA begins it
                pos = upto;
                continue;
            }
            const int r0 = tile * RT, rows = min(RT, it.n * p.G - r0);
            const int32_t *table = c.tables + (size_t)s * c.width;

            // ---- queries of rows g (and g + 8) in the MMA's k order
            uint32_t qf[RH][S::NS][2];
            int lim[RH];
            float qs[RH];  // INT8: the scores' factor besides the key's scale
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
                if constexpr (I8) {
                    float amax = 0.f;
#pragma unroll
                    for (int i = 0; i < S::NS; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            amax = fmaxf(amax, fmaxf(fabsf(bf_lo(qf[rr][i][e])), fabsf(bf_hi(qf[rr][i][e]))));
                    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
                    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
                    const uint32_t ex = min(max(__float_as_uint(amax) >> 23, 1u), 253u);
                    const float f = __uint_as_float((254u - ex) << 23);
                    qs[rr] = p.scale_log2 * __uint_as_float(ex << 23);
                    // codes 0 and 2 of a word are one register, 1 and 3 the other: so are the queries
#pragma unroll
                    for (int i = 0; i < S::NS; ++i) {
                        const float f0 = bf_lo(qf[rr][i][0]) * f, f1 = bf_hi(qf[rr][i][0]) * f, f2 = bf_lo(qf[rr][i][1]) * f,
                                    f3 = bf_hi(qf[rr][i][1]) * f;
                        qf[rr][i][0] = cvt_h2(f0, f2);
                        qf[rr][i][1] = cvt_h2(f1, f3);
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

            float vref = 0x1p-100f;  // INT8: what the weights' value scales are relative to, a power of two
            uint4 kr[NB][2][S::KC], vr[NB][4][S::VC];
            float2 ksc[I8 ? NB : 1][2], vsc[I8 ? NB : 1][2];
            auto unit_t0 = [&](int b) { return (b < it.nhu ? b : b - it.nhu + it.wu0) * UP; };
            // the pool's group of 16 rows with position tb (a multiple of 16); -1: nothing of it is seen, -2: no page
            auto pool_group = [&](int tb) {
                if (tb >= it.len || (tb + 16 <= it.lo && tb >= it.head)) return -1;
                const int page = __ldg(table + (tb >> c.psl));
                if (page < 0 || page >= c.n_pages) return -2;
                return ((page * c.nkv + h) << (c.psl - 4)) + ((tb & (c.ps - 1)) >> 4);
            };
            int krow[NB], nrow[NB];
            auto load_k = [&](const int (&row)[NB]) {
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
#pragma unroll
                        for (int cc = 0; cc < S::KC; ++cc) {
                            kr[i][a][cc] = make_uint4(0u, 0u, 0u, 0u);
                            if (row[i] >= 0)
                                kr[i][a][cc] =
                                    ld_stream16(c.k + (row[i] * 16ll + 8 * a + g) * (D * S::EB) + 64 * cc + 16 * t4);
                        }
                        if constexpr (I8) {
                            ksc[i][a] = make_float2(0.f, 0.f);
                            if (row[i] >= 0)
                                ksc[i][a] = __ldg(reinterpret_cast<const float2 *>(c.ks + row[i] * 16ll + 8 * a + 2 * t4));
                        }
                    }
            };
            auto load_v = [&](const int (&row)[NB]) {
#pragma unroll
                for (int i = 0; i < NB; ++i) {
#pragma unroll
                    for (int a = 0; a < 4; ++a)
#pragma unroll
                        for (int cc = 0; cc < S::VC; ++cc) {
                            vr[i][a][cc] = make_uint4(0u, 0u, 0u, 0u);
                            if (row[i] >= 0) {
                                const uint8_t *v = c.v + (row[i] * 16ll + 2 * t4 + (a & 1) + 8 * (a >> 1)) * (D * S::EB);
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
                                vsc[i][a] = __ldg(reinterpret_cast<const float2 *>(c.vs + row[i] * 16ll + 8 * a + 2 * t4));
                        }
                    }
                }
            };

            if (b0 + warp < b1) {
#pragma unroll
                for (int i = 0; i < NB; ++i) krow[i] = pool_group(unit_t0(b0 + warp) + 16 * i);
                load_k(krow);
            }
            for (int b = b0 + warp; b < b1; b += kWarps) {
                const int t0 = unit_t0(b);
                load_v(krow);
                const bool more = b + kWarps < b1;
                if (more) {
#pragma unroll
                    for (int i = 0; i < NB; ++i) nrow[i] = pool_group(unit_t0(b + kWarps) + 16 * i);
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
                                const int q = cc * (I8 ? 4 : 2) + st;
                                if constexpr (I8) {
                                    const uint32_t x = w[st] ^ 0x80808080u;
                                    const uint32_t k0 = half_codes(__byte_perm(x, 0x64646464u, 0x4240));
                                    const uint32_t k1 = half_codes(__byte_perm(x, 0x64646464u, 0x4341));
                                    if constexpr (RH == 1)
                                        mma_rows8_h(acc[0], acc[1], qf[0][q][0], qf[0][q][1], k0, k1);
                                    else
                                        mma_m16n8k16_h(acc, qf[0][q][0], qf[RH - 1][q][0], qf[0][q][1], qf[RH - 1][q][1], k0, k1);
                                } else if constexpr (RH == 1) {
                                    mma_rows8(acc[0], acc[1], qf[0][q][0], qf[0][q][1], w[2 * st], w[2 * st + 1]);
                                } else {
                                    mma_m16n8k16(acc, qf[0][q][0], qf[RH - 1][q][0], qf[0][q][1], qf[RH - 1][q][1], w[2 * st],
                                                 w[2 * st + 1]);
                                }
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 2 * RH; ++e) {
                            if constexpr (I8)
                                sc[i][a][e] = acc[e] * (qs[e / 2] * (e & 1 ? ksc[i][a].y : ksc[i][a].x));
                            else
                                sc[i][a][e] = acc[e] * p.scale_log2;
                        }
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
                float vscale = 1.f;
                if constexpr (I8) {
                    float vmax = 0.f;
#pragma unroll
                    for (int i = 0; i < NB; ++i)
#pragma unroll
                        for (int a = 0; a < 2; ++a) vmax = fmaxf(vmax, fmaxf(vsc[i][a].x, vsc[i][a].y));
                    vmax = fmaxf(vmax, __shfl_xor_sync(0xFFFFFFFFu, vmax, 1));
                    vmax = fmaxf(vmax, __shfl_xor_sync(0xFFFFFFFFu, vmax, 2));
                    if (vmax > vref) {  // the same in all lanes
                        const float nv = __uint_as_float(min((__float_as_uint(vmax) + 0x007FFFFFu) & 0x7F800000u, 0x7F000000u));
                        vscale = vref / nv;
                        vref = nv;
                        rise = true;
                    }
                }
                if (__any_sync(0xFFFFFFFFu, rise)) {
#pragma unroll
                    for (int rr = 0; rr < RH; ++rr) {
                        float corr = mn[rr] > m[rr] ? ex2(m[rr] - mn[rr]) : 1.f;
                        m[rr] = mn[rr];
                        l[rr] *= corr;
                        corr *= vscale;
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
                            const float w0 = ex2(sc[i][a][2 * rr] - base[rr]), w1 = ex2(sc[i][a][2 * rr + 1] - base[rr]);
                            l[rr] += w0 + w1;
                            if constexpr (I8) {
                                const float f = 4096.f / vref;
                                ph[rr][a] = cvt_h2(w0 * (vsc[i][a].x * f), w1 * (vsc[i][a].y * f));
                            } else {
                                const uint32_t hi = cvt_bf2(w0, w1);
                                ph[rr][a] = hi;
                                pl[rr][a] = cvt_bf2(w0 - bf_lo(hi), w1 - bf_hi(hi));
                            }
                        }
                    // ---- o += P V, one 8-column tile per dimension a lane holds
#pragma unroll
                    for (int cc = 0; cc < S::VC; ++cc) {
                        const uint32_t w[4][4] = {{vr[i][0][cc].x, vr[i][0][cc].y, vr[i][0][cc].z, vr[i][0][cc].w},
                                                  {vr[i][1][cc].x, vr[i][1][cc].y, vr[i][1][cc].z, vr[i][1][cc].w},
                                                  {vr[i][2][cc].x, vr[i][2][cc].y, vr[i][2][cc].z, vr[i][2][cc].w},
                                                  {vr[i][3][cc].x, vr[i][3][cc].y, vr[i][3][cc].z, vr[i][3][cc].w}};
                        if constexpr (I8) {
#pragma unroll
                            for (int q = 0; q < S::VW / 4; ++q) {
                                const uint32_t x0 = w[0][q] ^ 0x80808080u, x1 = w[1][q] ^ 0x80808080u;
                                const uint32_t x2 = w[2][q] ^ 0x80808080u, x3 = w[3][q] ^ 0x80808080u;
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    // the codes of two dimensions in rows (0, 1) and (2, 3)
                                    const uint32_t y0 = __byte_perm(x0, x1, h ? 0x7362 : 0x5140);
                                    const uint32_t y1 = __byte_perm(x2, x3, h ? 0x7362 : 0x5140);
#pragma unroll
                                    for (int e = 0; e < 2; ++e) {
                                        const uint32_t v0 = half_codes(__byte_perm(y0, 0x64646464u, e ? 0x4342 : 0x4140));
                                        const uint32_t v1 = half_codes(__byte_perm(y1, 0x64646464u, e ? 0x4342 : 0x4140));
                                        float(&oj)[2 * RH] = o[cc * S::VW + 4 * q + 2 * h + e];
                                        if constexpr (RH == 1)
                                            mma_rows8_h(oj[0], oj[1], ph[0][0], ph[0][1], v0, v1);
                                        else
                                            mma_m16n8k16_h(oj, ph[0][0], ph[1][0], ph[0][1], ph[1][1], v0, v1);
                                    }
                                }
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < S::VW; ++j) {
                                const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
                                const uint32_t v0 = __byte_perm(w[0][j / 2], w[1][j / 2], sel);
                                const uint32_t v1 = __byte_perm(w[2][j / 2], w[3][j / 2], sel);
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
                }
                if (more) {
#pragma unroll
                    for (int i = 0; i < NB; ++i) krow[i] = nrow[i];
                }
            }

            // ---- merge the warps' states
            if constexpr (I8) {
                const float f = vref / 4096.f;
#pragma unroll
                for (int j = 0; j < S::VC * S::VW; ++j)
#pragma unroll
                    for (int e = 0; e < 2 * RH; ++e) o[j][e] *= f;
            }
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
            const int slot = first ? 0 : 1;
            first = false;
            if (!whole && b0 == 0 && tid == 0) {
                const long long last = ((item_at + cost) * nc + total - 1) / total - 1;  // the CTA with the item's end
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
            pos = upto;
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
    __shared__ __align__(16) float4 so[GR][TPR];
    __shared__ float2 sl[GR];
    __shared__ int bad_row;
    const int tid = threadIdx.x, cta = blockIdx.x, r = blockIdx.y;
    after_previous();
    const JoinRec rec = reinterpret_cast<const JoinRec *>(p.ws)[cta];
    if (rec.parts == 0) return;
    bool bad = false;
    const Item it = item_of<S::UP>(p, rec.s, &bad);
    const int row = rec.tile * RT + r;
    if (row >= it.n * p.G) return;
    const float *parts = p.ws + (size_t)p.ctas * (sizeof(JoinRec) / 4) + (size_t)r * LD;
    auto part = [&](int i) { return parts + (size_t)(2 * (cta + i) + (i == 0 ? rec.slot : 0)) * RT * LD; };
    // a group's own running maximum, so that states and maxima are read at once
    const int grp = tid / TPR, d0 = (tid % TPR) * 4;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f, M = -INFINITY;
    for (int i0 = grp; i0 < rec.parts; i0 += 4 * GR) {
        float4 v[4];
        float2 ml[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + k * GR;
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            ml[k] = make_float2(-INFINITY, 0.f);
            if (i < rec.parts) {
                ml[k] = __ldcg(reinterpret_cast<const float2 *>(part(i) + D));
                v[k] = __ldcg(reinterpret_cast<const float4 *>(part(i) + d0));
            }
        }
        const float nm = fmaxf(M, fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)));
        const float bs = nm == -INFINITY ? 0.f : nm, f0 = ex2(M - bs);
        M = nm;
        L *= f0;
        O.x *= f0;
        O.y *= f0;
        O.z *= f0;
        O.w *= f0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float f = ex2(ml[k].x - bs);
            L = fmaf(f, ml[k].y, L);
            O.x = fmaf(f, v[k].x, O.x);
            O.y = fmaf(f, v[k].y, O.y);
            O.z = fmaf(f, v[k].z, O.z);
            O.w = fmaf(f, v[k].w, O.w);
        }
    }
    so[grp][tid % TPR] = O;
    if (tid % TPR == 0) sl[grp] = make_float2(M, L);
    if (tid == 0) bad_row = 0;
    __syncthreads();
    const int hq = rec.h * p.G + row % p.G, tok = it.t0 + row / p.G;
    if (grp == 0) {
        float top = -INFINITY;
#pragma unroll
        for (int k = 0; k < GR; ++k) top = fmaxf(top, sl[k].x);
        const float bs = top == -INFINITY ? 0.f : top;
        O = make_float4(0.f, 0.f, 0.f, 0.f);
        L = 0.f;
#pragma unroll
        for (int k = 0; k < GR; ++k) {
            const float f = ex2(sl[k].x - bs);
            const float4 v = so[k][tid];
            L = fmaf(f, sl[k].y, L);
            O.x = fmaf(f, v.x, O.x);
            O.y = fmaf(f, v.y, O.y);
            O.z = fmaf(f, v.z, O.z);
            O.w = fmaf(f, v.w, O.w);
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
    const cudaError_t e = launch_next(stream_kernel<D, I8, RT>, dim3((unsigned)p.ctas), dim3(kThr), 0, st, p);
    if (e != cudaSuccess) return e;
    return launch_next(join_kernel<D, I8, RT>, dim3((unsigned)p.ctas, (unsigned)RT), dim3(kThr), 0, st, p);
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
