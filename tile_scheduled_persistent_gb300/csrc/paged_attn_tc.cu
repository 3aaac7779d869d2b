// Attention of many query rows per (sequence, KV head) over a paged KV cache:
// prompts, pieces of prompts, draft tokens, on the fifth-generation tensor
// cores.
//
//   out_r = sum_t softmax_t(scale q_r . K_t) V_t   over the positions t row r sees
//
// The query heads of a KV head and the tokens of a sequence are rows of one
// matrix (row = token * group + head of the group), so a KV head's keys and
// values are read once for all of them. A CTA works on two tiles of 128 rows
// (a "pair") and walks the positions in blocks of 128:
//   - the loader (one warp): each page of a block as boxes of page_size x 64
//     dimensions into a ring of shared-memory blocks (K, V, K, V ...), 128-byte
//     swizzle. The values that no row may see (behind the end, missing pages) are
//     set to zero in shared memory, as 0 * NaN would not vanish. With an INT8
//     cache the loader is four warps that read the codes, widen them to BF16
//     (exactly) and store them in the same layout; the scales go beside them.
//   - the MMA issuer (one warp): S_i = Q_i K^T (128 x 128 in tensor memory), and,
//     when the softmax has turned S_i into weights, O_i += P_i V with P_i read from
//     tensor memory. While one tile's rows are in the softmax the tensor cores work
//     on the other tile. At D 64 the weights have columns of their own, and the
//     next scores are computed as soon as the last are read.
//   - the softmax of a row by one thread (D 64, INT8) or two (D 128, half a row each,
//     as there the chain from scores to weights is what the tensor cores wait for):
//     reference and sum in FP32. The reference is a maximum seen some blocks ago, so
//     that no thread waits for another's; a weight may then be above 1, which costs
//     no accuracy in floating point. O_i is rescaled when the reference rises, by 8
//     powers of two at least. What a late reference cannot hold, a weight or sum
//     beyond 2^127, comes out infinite or NaN, and the row is computed again position
//     by position, as it is where 0 * inf met a value that other rows see.
//   - the planner (one warp): what each role has to know of the next pairs.
// Weights enter P V as BF16 (2^-8 relative at most, either way): a second product for
// the remainder would cost half as much again where the tensor cores are the bound,
// and the output is BF16 itself.
// The work is cut as in the streaming kernel: the blocks of all pairs form one
// line, each CTA (one per SM) takes an equal piece, pairs that several CTAs share
// are joined afterwards. Every wait is bounded; past the limit the CTA records a
// timeout, lets its copies and MMAs finish (bounded too), frees its tensor memory
// and returns.
//
// Measured on GB300: a prompt of 4,096 (D 128, 32/8 heads, pages of 64) 128 us with the
// join, 1,075 TFLOP/s, 0.56 of the measured dense BF16 rate; 256 tokens at 32,768 (D 64)
// 84 us, 0.43; INT8 pages 262 and 154 us. A block of both tiles takes 3,000 cycles at
// D 128, of which the tensor cores need 2,048; at D 64 2,800 of 1,024, there the softmax
// is the longer part.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "paged_device.cuh"

namespace tiles {
namespace paged {

constexpr int kBlock = 128;      // positions a block
constexpr int kTile = 128;       // query rows a tile
constexpr int kPair = 2 * kTile; // query rows a CTA works on at a time
constexpr int kMaxRing = 8;
constexpr int kMaskRing = 16;
constexpr unsigned long long kTimeoutNs = 2000000000ull;
// The line in which the work is cut counts a pair as its blocks and kPairCost
// blocks' time for its queries, its output and the change from one to the next.
constexpr int kPairCost = 4;
constexpr float kRise = 8.0f;    // powers of two a row's scores may pass its reference by before it is set anew

template <int D, bool I8>
struct TcShape {
    static constexpr int HALF = kBlock * 128;           // bytes: 128 rows of 64 BF16
    static constexpr int BLOCK = HALF * (D / 64);       // one block of K or V, or a query tile
    static constexpr int RING = D == 128 ? 4 : 8;
    // threads a query row's softmax is shared by
    static constexpr int HALVES = D == 64 || I8 ? 1 : 2;
    // warpgroups: HALVES of softmax for each tile; one of the MMA issuer, the loader and the
    // planner; with an INT8 cache one of loaders, as widening takes four warps
    static constexpr int SOFTMAX = 8 * HALVES, THREADS = (SOFTMAX + 4 + (I8 ? 4 : 0)) * 32, LOADERS = I8 ? 128 : 32;
    static constexpr int LOADER = SOFTMAX + (I8 ? 4 : 1);  // its first warp
    // registers a thread after the split; the sums are the launch's: 2 x 208 + 88 = 3 x 168 of
    // 384 threads, 4 x 104 + 64 = 5 x 96 of 640, 2 x 184 + 56 + 88 = 4 x 128 of 512
    static constexpr int REG_SOFTMAX = I8 ? 184 : HALVES == 1 ? 208 : 104, REG_ISSUE = I8 ? 56 : HALVES == 1 ? 88 : 64,
                         REG_LOAD = 88;
    // tensor memory, 512 columns: scores of the two tiles (128 each), O (D each) and, at D 64,
    // room for the weights of their own; at D 128 they take the place of the scores
    static constexpr bool SPLIT = D == 64;
    static constexpr int O_COL = 256, P_COL = SPLIT ? 384 : 0, P_TILE = SPLIT ? 64 : 128,
                         P_HALF = SPLIT || HALVES == 1 ? 32 : 64;
    static_assert(O_COL + 2 * D <= (SPLIT ? P_COL : 512) && P_COL + P_TILE + P_HALF + 32 <= 512, "512 columns");
    static constexpr int PART = kPair * (D + 2);        // floats of a partial state: o [D / 4][row][4], m [row], l [row]
    // bytes: row maxima of the last four blocks and the sums at a pair's end, of a tile's halves;
    // a kilobyte a softmax warp for the output on its way
    static constexpr int TOPS = HALVES == 2 ? 5 * 2 * 2 * kTile * 4 : 0, STAGE = SOFTMAX * 1024;
    static constexpr int SCALES = I8 ? 2 * 16 * kBlock * 4 : 0;  // bytes: a block's K and V scales, by block number
};

// What the roles need to know of a piece of work: a pair's blocks [b0, b1). b1 == 0: no more.
struct Seg {
    int s, h, m, t0, n, len;         // row, KV head, pair; the row's first token, tokens, length
    int rows, b0, b1, nb;            // query rows of the pair; blocks, and how many the pair has
    int hi, lo, head, nhb, wb0;      // positions [0, head) and [lo, hi) are seen; see PairSpan
    int all_hi[2], all_lo[2];        // positions that every row of a tile sees
    int slot;                        // of a partial state
    uint32_t q_at[kPair], o_at[kPair];  // where the query rows lie in q and out, in 16-byte units
};
constexpr int kSegRing = 3;

struct Ctl {
    uint64_t full[kMaxRing], empty[kMaxRing], fix, drain, q_ready[2], s_full[2], s_free[2], p_full[2], o_done[2], x_ready[2][4];
    uint64_t seg_full[kSegRing], seg_empty[kSegRing];
    uint32_t tmem, abort, again;     // again: some row of the output came out infinite or NaN
    uint32_t mask[kMaskRing];    // pages of a key block that are there, by block number
    int seg_s, seg_h, seg_m;
    long long seg_at, scan[20];
    Seg seg[kSegRing];
};

struct SegRec {
    int parts, s, h, m, slot, pad[3];
};

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) {  // K-major, 128-byte swizzle, 8-row groups 1024 bytes apart
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
           ((uint64_t)2 << 61);
}
// MN-major, 128-byte swizzle: 64 consecutive elements of N a row of 128 bytes,
// the next 64 a half block further (leading offset), groups of 8 k-rows 1024
// bytes apart (stride offset)
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t lead) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ uint32_t idesc(int n, bool b_mn) {  // M 128, BF16 x BF16 -> FP32
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}
// Four MMAs over 64 of the k index, executed by a whole converged warp; one lane,
// the same one every time, issues. (Issued from a branch that a single lane takes,
// an MMA cost 190-240 cycles whatever its size, as its descriptors then live in
// ordinary registers; this way the tensor core's own rate, 64 cycles at M 128,
// N 128, K 16.) SS: K-major A and B in shared memory, 32 bytes a step. TS: A in
// tensor memory, 8 columns a step, MN-major B, 16 rows of 128 bytes a step.
__device__ __forceinline__ void mma4_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, t, e;\n\t.reg .b64 a, b;\n\t"
        "elect.sync _|e, 0xFFFFFFFF;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, t, e;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\t"
        "elect.sync _|e, 0xFFFFFFFF;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "add.s32 a, %1, 8;\n\tadd.s64 b, %2, 128;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
        "add.s32 a, %1, 16;\n\tadd.s64 b, %2, 256;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
        "add.s32 a, %1, 24;\n\tadd.s64 b, %2, 384;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void commit(uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xFFFFFFFF;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

#define R8(a, o) "=r"(a[o]), "=r"(a[o + 1]), "=r"(a[o + 2]), "=r"(a[o + 3]), "=r"(a[o + 4]), "=r"(a[o + 5]), "=r"(a[o + 6]), "=r"(a[o + 7])
#define V8(a, o) "r"(a[o]), "r"(a[o + 1]), "r"(a[o + 2]), "r"(a[o + 3]), "r"(a[o + 4]), "r"(a[o + 5]), "r"(a[o + 6]), "r"(a[o + 7])
// 64, or 16, consecutive columns of this thread's tensor-memory lane, complete on return
__device__ __forceinline__ void tld64(uint32_t t, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, "
        "%38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, "
        "%60, %61, %62, %63}, [%64];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : R8(r, 0), R8(r, 8), R8(r, 16), R8(r, 24), R8(r, 32), R8(r, 40), R8(r, 48), R8(r, 56)
        : "r"(t)
        : "memory");
}
// two times 64, with one wait
__device__ __forceinline__ void tld128(uint32_t t, uint32_t (&r)[128]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%128];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, %80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95, %96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, %112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%129];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : R8(r, 0), R8(r, 8), R8(r, 16), R8(r, 24), R8(r, 32), R8(r, 40), R8(r, 48), R8(r, 56), R8(r, 64), R8(r, 72),
          R8(r, 80), R8(r, 88), R8(r, 96), R8(r, 104), R8(r, 112), R8(r, 120)
        : "r"(t), "r"(t + 64)
        : "memory");
}
__device__ __forceinline__ void tld16(uint32_t t, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : R8(r, 0), R8(r, 8)
        : "r"(t)
        : "memory");
}
__device__ __forceinline__ void tst16(uint32_t t, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(t),
        V8(r, 0), V8(r, 8)
        : "memory");
}
__device__ __forceinline__ void tst_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// two FP32 operations in one instruction
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// the lowest n bits
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }

// ------------------------------------------------------------------ the line of blocks
// Pair m of (row, head): query rows 256 m .. of n G, the positions that some
// row of it sees, as blocks: nhb of [0, head), the rest from block wb0 on.
struct PairSpan {
    int rows, p_first, p_last, head, lo, hi, nhb, wb0, nb;
    __device__ __forceinline__ int cost() const { return nb ? nb + kPairCost : 0; }
};
__device__ __forceinline__ PairSpan pair_span(const AttnParams &p, const RowSpan &r, int m) {
    PairSpan a;
    const int r0 = m * kPair;
    a.rows = min(kPair, r.n * p.G - r0);
    const int base = r.len - r.n;
    a.p_first = base + group_div(p, r0);
    a.p_last = base + group_div(p, max(0, r0 + a.rows - 1));
    a.hi = max(0, a.p_last + 1);
    visible_span(p, a.hi, a.p_first, &a.head, &a.lo);
    a.nhb = (a.head + kBlock - 1) / kBlock;
    a.wb0 = a.lo / kBlock;
    if (a.nhb > a.wb0) a.nhb = a.wb0;
    a.nb = a.rows > 0 ? a.nhb + (a.hi + kBlock - 1) / kBlock - a.wb0 : 0;
    return a;
}
__device__ __forceinline__ int pairs_of(const AttnParams &p, const RowSpan &r) { return (r.n * p.G + kPair - 1) / kPair; }

// Cost of one head of each of 32 rows (one a lane): rows of several pairs are
// added up by the whole warp.
__device__ __forceinline__ long long row_cost(const AttnParams &p, const RowSpan &r, int lane) {
    const int np = pairs_of(p, r);
    long long nb = np == 1 ? pair_span(p, r, 0).cost() : 0;
    uint32_t many = __ballot_sync(0xFFFFFFFFu, np > 1);
    while (many) {
        const int src = __ffs(many) - 1;
        many &= many - 1;
        RowSpan q;
        q.t0 = 0;
        q.n = __shfl_sync(0xFFFFFFFFu, r.n, src);
        q.len = __shfl_sync(0xFFFFFFFFu, r.len, src);
        const int k = pairs_of(p, q);
        long long sum = 0;
        for (int m = lane; m < k; m += 32) sum += pair_span(p, q, m).cost();
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (lane == src) nb = sum;
    }
    return nb;
}

// A walk over the pairs from (s, h, m) on; every role of the CTA walks alike.
struct Walk {
    int s, h, m;
    RowSpan r;
    PairSpan a;
    __device__ __forceinline__ void load(const AttnParams &p) {
        bool bad = false;
        r = row_span(p, s, &bad);
        a = pair_span(p, r, m);
    }
    // the next pair with blocks; only called where more blocks follow
    __device__ __forceinline__ void next(const AttnParams &p) {
        do {
            if (++m >= pairs_of(p, r)) {
                m = 0;
                if (++h >= p.c.nkv || r.n == 0) {
                    h = 0;
                    if (++s >= p.c.n_seqs) {
                        s = p.c.n_seqs - 1;
                        a.nb = 0;
                        return;
                    }
                    bool bad = false;
                    r = row_span(p, s, &bad);
                }
            }
            a = pair_span(p, r, m);
        } while (a.nb == 0);
    }
};

// False past the deadline, or once another role of the CTA has given up.
__device__ __forceinline__ bool bounded_wait(uint64_t *bar, uint32_t parity, unsigned long long deadline,
                                             volatile uint32_t *abort) {
    for (uint32_t spin = 0;; ++spin) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((spin & 63u) == 63u && (*abort || global_timer() > deadline)) {
            *abort = 1;
            return false;
        }
    }
}

// Rows that came out infinite or NaN, of the pairs that this CTA has computed whole:
// its line from cost unit `at` of pair (s, h, m) on. Warp `warp` of `warps`.
template <int D, bool I8>
__device__ __noinline__ void rows_again(const AttnParams &p, int s, int h, int m, int at, long long left, int warp, int warps) {
    const int lane = threadIdx.x & 31;
    Walk w;
    w.s = s;
    w.h = h;
    w.m = m;
    w.load(p);
    while (left > 0) {
        const int used = (int)min((long long)(w.a.cost() - at), left);
        if (at <= kPairCost && at + used == w.a.cost())
            for (int x = warp; x < w.a.rows; x += warps) {
                const int r = w.m * kPair + x, tok = group_div(p, r), hq = w.h * p.G + r - tok * p.G;
                const uint16_t *o = p.out + (w.r.t0 + tok) * p.o_t + hq * p.o_h;
                bool finite = true;
#pragma unroll
                for (int d = 0; d < D; d += 32) finite &= (o[d + lane] & 0x7F80u) != 0x7F80u;
                if (!__all_sync(0xFFFFFFFFu, finite)) row_again<D, I8>(p, w.s, w.h, w.r.t0, w.r.n, w.r.len, r);
            }
        left -= used;
        at = 0;
        if (left > 0) w.next(p);
    }
}

// ------------------------------------------------------------------ the kernel
template <int D, bool I8>
__global__ void __launch_bounds__(TcShape<D, I8>::THREADS, 1)
    tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ TensorMap mk, const __grid_constant__ TensorMap mv) {
    using S = TcShape<D, I8>;
    constexpr int RING = S::RING, NW = S::THREADS / 32;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint8_t *sq = sm;                     // two query tiles
    uint8_t *ring = sm + 2 * S::BLOCK;    // RING blocks
    float(*tops)[2][2][kTile] = reinterpret_cast<float(*)[2][2][kTile]>(ring + RING * S::BLOCK + S::SCALES);
    uint8_t *stages = ring + RING * S::BLOCK + S::SCALES + S::TOPS;
    Ctl *ctl = reinterpret_cast<Ctl *>(stages + S::STAGE);
    float(*scale)[kMaskRing][kBlock] = reinterpret_cast<float(*)[kMaskRing][kBlock]>(ring + RING * S::BLOCK);  // INT8
    const View &c = p.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
    SegRec *recs = reinterpret_cast<SegRec *>(p.ws);
    float *parts = p.ws + (size_t)p.ctas * (sizeof(SegRec) / 4);
    after_previous();
    if (smem_u32(sm) & 1023u) {  // the swizzle counts on it
        if (tid == 0) {
            recs[cta].parts = 0;
            atomicOr(reinterpret_cast<uint32_t *>(c.state), kDevBounds);
        }
        return;
    }
    if (tid == 0) {
        recs[cta].parts = 0;
        for (int i = 0; i < RING; ++i) {
            mbar_init(&ctl->full[i], I8 ? S::LOADERS : 1);
            mbar_init(&ctl->empty[i], 1);
        }
        mbar_init(&ctl->fix, 1);
        mbar_init(&ctl->drain, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->q_ready[i], 128 * S::HALVES);
            mbar_init(&ctl->s_full[i], 1);
            mbar_init(&ctl->p_full[i], 128 * S::HALVES);
            for (int k = 0; k < 4; ++k) mbar_init(&ctl->x_ready[i][k], 64);
            mbar_init(&ctl->s_free[i], 128 * S::HALVES);
            mbar_init(&ctl->o_done[i], 1);
        }
        for (int i = 0; i < kSegRing; ++i) {
            mbar_init(&ctl->seg_full[i], 1);
            mbar_init(&ctl->seg_empty[i], S::SOFTMAX + 1 + S::LOADERS / 32);
        }
        ctl->abort = ctl->again = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // ---- this CTA's piece of the line: warp w sums rows [w per, (w + 1) per)
    const int per = (c.n_seqs + NW - 1) / NW, sa = warp * per, sb = min(c.n_seqs, sa + per);
    long long mine = 0;
    for (int s0 = sa; s0 < sb; s0 += 32) {
        RowSpan r = {0, 0, 0};
        bool bad = false;
        if (s0 + lane < sb) r = row_span(p, s0 + lane, &bad);
        mine += row_cost(p, r, lane);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, o);
    mine *= c.nkv;
    if (lane == 0) ctl->scan[warp] = mine;
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < NW; ++w) {
        if (w < warp) before += ctl->scan[w];
        total += ctl->scan[w];
    }
    // pieces of at least one block and its pair's cost
    const long long nc = min((long long)p.ctas, max(1ll, total / (kPairCost + 1)));
    const long long begin = cta < nc ? cta * total / nc : 0, end = cta < nc ? (cta + 1) * total / nc : 0;
    if (begin < end && begin >= before && begin < before + mine) {
        // the row, then the head, then the pair that holds block `begin`
        long long at = before;
        bool hit = false;
        for (int s0 = sa; s0 < sb && !hit; s0 += 32) {
            RowSpan r = {0, 0, 0};
            bool bad = false;
            if (s0 + lane < sb) r = row_span(p, s0 + lane, &bad);
            const long long nb = row_cost(p, r, lane);
            long long x = nb * c.nkv;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
                if (lane >= o) x += y;
            }
            const uint32_t in = __ballot_sync(0xFFFFFFFFu, begin < at + x);
            if (in) {
                const int src = __ffs(in) - 1;
                const long long row_nb = __shfl_sync(0xFFFFFFFFu, nb, src);
                const long long row_at = at + __shfl_sync(0xFFFFFFFFu, x, src) - row_nb * c.nkv;
                RowSpan q;
                q.t0 = 0;
                q.n = __shfl_sync(0xFFFFFFFFu, r.n, src);
                q.len = __shfl_sync(0xFFFFFFFFu, r.len, src);
                const int h = (int)((begin - row_at) / row_nb);
                long long pos = row_at + h * row_nb;
                const int np = pairs_of(p, q);
                for (int m0 = 0; m0 < np; m0 += 32) {
                    int k = m0 + lane < np ? pair_span(p, q, m0 + lane).cost() : 0, y = k;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int z = __shfl_up_sync(0xFFFFFFFFu, y, o);
                        if (lane >= o) y += z;
                    }
                    const uint32_t got = __ballot_sync(0xFFFFFFFFu, begin < pos + y);
                    if (got) {
                        if (lane == __ffs(got) - 1) {
                            ctl->seg_s = s0 + src;
                            ctl->seg_h = h;
                            ctl->seg_m = m0 + lane;
                            ctl->seg_at = pos + y - k;
                        }
                        break;
                    }
                    pos += __shfl_sync(0xFFFFFFFFu, y, 31);
                }
                hit = true;
            }
            at += __shfl_sync(0xFFFFFFFFu, x, 31);
        }
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl->tmem)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = ctl->tmem;
    volatile uint32_t *abort = &ctl->abort;
    // set anew for each piece of work, so that it bounds a wait and not the kernel
    unsigned long long deadline = global_timer() + kTimeoutNs;
    bool ok = true;
    // MMAs and copies this thread has issued, for the way out
    int issued = 0;

    if (begin < end) {
        auto warp_wait = [&](uint64_t *bar, uint32_t parity) {
            ok = __all_sync(0xFFFFFFFFu, bounded_wait(bar, parity & 1u, deadline, abort));
            return ok;
        };
        // the k-th piece of work; false at the end (or after a timeout)
        auto seg_begin = [&](uint32_t k) {
            deadline = global_timer() + kTimeoutNs;
            return warp_wait(&ctl->seg_full[k % kSegRing], k / kSegRing) && ctl->seg[k % kSegRing].b1 > 0;
        };
        auto seg_peek = [&](uint32_t k) { return warp_wait(&ctl->seg_full[k % kSegRing], k / kSegRing); };
        auto seg_end = [&](uint32_t k) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->seg_empty[k % kSegRing]);
        };
        // ================================================ planner: the CTA's pieces, a few ahead of their use
        auto planner = [&]() {
            Walk w;
            w.s = ctl->seg_s;
            w.h = ctl->seg_h;
            w.m = ctl->seg_m;
            w.load(p);
            uint32_t k = 0;
            auto slot_free = [&]() {
                deadline = global_timer() + kTimeoutNs;
                return k < kSegRing || warp_wait(&ctl->seg_empty[k % kSegRing], k / kSegRing - 1u);
            };
            // in cost units: where the work begins in its first pair, how much there is. Of a pair
            // that begins at unit 0, units kPairCost + b are block b.
            int at = (int)(begin - ctl->seg_at);
            long long left = end - begin;
            bool first = true;
            while (left > 0) {
                const int used = (int)min((long long)(w.a.cost() - at), left), b0 = max(0, at - kPairCost), b1 = max(0, at + used - kPairCost);
                if (b0 < b1) {
                    if (!slot_free()) break;
                    Seg &g = ctl->seg[k % kSegRing];
                    for (int x = lane; x < w.a.rows; x += 32) {
                        const int r = w.m * kPair + x, tok = group_div(p, r), hq = w.h * p.G + r - tok * p.G;
                        const long long q_at = (w.r.t0 + tok) * p.q_t + hq * p.q_h;
                        g.q_at[x] = (uint32_t)(q_at >> 3);
                        g.o_at[x] = (uint32_t)(((w.r.t0 + tok) * p.o_t + hq * p.o_h) >> 3);
                        prefetch_l2(p.q + q_at);  // its queries on their way to L2
                        if (D == 128) prefetch_l2(p.q + q_at + 64);
                    }
                    __syncwarp();
                    if (lane == 0) {
                        g.s = w.s;
                        g.h = w.h;
                        g.m = w.m;
                        g.t0 = w.r.t0;
                        g.n = w.r.n;
                        g.len = w.r.len;
                        g.rows = w.a.rows;
                        g.b0 = b0;
                        g.b1 = b1;
                        g.nb = w.a.nb;
                        g.hi = w.a.hi;
                        g.lo = w.a.lo;
                        g.head = w.a.head;
                        g.nhb = w.a.nhb;
                        g.wb0 = w.a.wb0;
                        for (int i = 0; i < 2; ++i) {
                            const int ra = w.m * kPair + i * kTile, rz = min(ra + kTile, w.m * kPair + w.a.rows) - 1;
                            g.all_hi[i] = w.r.len - w.r.n + group_div(p, ra);
                            g.all_lo[i] = p.window > 0 ? w.r.len - w.r.n + group_div(p, max(ra, rz)) - p.window + 1 : 0;
                        }
                        g.slot = first ? 0 : 1;
                        if (b0 == 0 && b1 < w.a.nb) {  // others finish this pair
                            SegRec rec;
                            const long long pair_end = end - left - at + w.a.cost();
                            rec.parts = (int)((pair_end * nc + total - 1) / total - 1 - cta) + 1;
                            rec.s = w.s;
                            rec.h = w.h;
                            rec.m = w.m;
                            rec.slot = g.slot;
                            rec.pad[0] = rec.pad[1] = rec.pad[2] = 0;
                            recs[cta] = rec;
                        }
                        mbar_arrive(&ctl->seg_full[k % kSegRing]);
                    }
                    ++k;
                    first = false;
                }
                left -= used;
                at = 0;
                if (left > 0) w.next(p);
            }
            if (ok && slot_free() && lane == 0) {
                ctl->seg[k % kSegRing].b1 = 0;
                mbar_arrive(&ctl->seg_full[k % kSegRing]);
            }
            __syncwarp();
        };
        // ================================================ loader
        auto loader = [&]() {
            const int lt = tid - S::LOADER * 32;  // thread of the loader
            int n = 0;                     // blocks of K and V so far
            uint32_t kb = 0, fixes = 0;    // key blocks, repaired blocks so far
            for (uint32_t sk = 0; seg_begin(sk); ++sk) {
                const Seg &g = ctl->seg[sk % kSegRing];
                const int b1 = g.b1, hi = g.hi, lo = g.lo, head = g.head, nhb = g.nhb, wb0 = g.wb0, hh = g.h;
                const int32_t *table = c.tables + (size_t)g.s * c.width;
                for (int b = g.b0; b < b1 && ok; ++b) {
                    const int t0 = (b < nhb ? b : b - nhb + wb0) * kBlock, npg = kBlock >> c.psl;
                    // lane i: page i of the block, -1 where nothing of it is seen, or it is missing
                    int page = -1;
                    if (lane < npg) {
                        const int pa = t0 + (lane << c.psl), pe = pa + c.ps;
                        if (pa < hi && (pe > lo || pa < head)) {
                            page = __ldg(table + (pa >> c.psl));
                            if (page < 0 || page >= c.n_pages) {
                                page = -1;
                                atomicOr(reinterpret_cast<uint32_t *>(c.state), kDevBounds);
                            }
                        }
                    }
                    const uint32_t have = __ballot_sync(0xFFFFFFFFu, page >= 0);
                    // bits of 16 positions, for the softmax
                    uint32_t mask16 = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) mask16 |= ((have >> ((16 * i) >> c.psl)) & 1u) << i;
                    for (int kv = 0; kv < 2 && ok; ++kv, ++n) {
                        const int st = n % RING, round = n / RING;
                        if (round > 0 && !warp_wait(&ctl->empty[st], (uint32_t)(round - 1))) break;
                        uint8_t *dst = ring + st * S::BLOCK;
                        if (kv == 0 && lt == 0) ctl->mask[kb % kMaskRing] = mask16;
                        if constexpr (!I8) {
                            // rows of V that nothing may read: zero them once the copies are in
                            const bool repair = kv == 1 && (have != (1u << npg) - 1u || t0 + kBlock > hi);
                            uint64_t *bar = repair ? &ctl->fix : &ctl->full[st];
                            if (lane == 0) mbar_expect_tx(bar, (uint32_t)(__popc(have) * c.ps * D * 2));
                            __syncwarp();
                            if (page >= 0) {
                                const int z = page * c.nkv + hh;
#pragma unroll
                                for (int hf = 0; hf < D / 64; ++hf)
                                    tensor_g2s_3d(dst + hf * S::HALF + lane * c.ps * 128, kv ? &mv : &mk, 64 * hf, 0, z, bar);
                            }
                            if (repair) {
                                if (!warp_wait(&ctl->fix, fixes)) break;
                                ++fixes;
                                for (int i = lane; i < kBlock * (D / 8); i += 32) {
                                    const int row = i / (D / 8), u = i % (D / 8);
                                    if (!((mask16 >> (row / 16)) & 1u) || t0 + row >= hi)
                                        *reinterpret_cast<uint4 *>(dst + (u / 8) * S::HALF + row * 128 + (((u % 8) ^ (row & 7)) << 4)) =
                                            make_uint4(0u, 0u, 0u, 0u);
                                }
                                fence_proxy_async_smem();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(&ctl->full[st]);
                            }
                        } else {
                            // 16 codes a step: a row is D / 16 steps
                            const uint8_t *pool = kv ? c.v : c.k;
                            const float *scales = kv ? c.vs : c.ks;
                            constexpr int UPR = D / 16, STEPS = kBlock * UPR / S::LOADERS, AT_ONCE = 4;
                            static_assert(STEPS % AT_ONCE == 0, "whole groups of loads");
#pragma unroll
                            for (int r = lt; r < kBlock; r += S::LOADERS) {
                                const int pg = __shfl_sync(0xFFFFFFFFu, page, r >> c.psl);
                                float f = 0.f;
                                if (pg >= 0 && t0 + r < hi)
                                    f = __ldg(scales + ((size_t)pg * c.nkv + hh) * c.ps + (r & (c.ps - 1)));
                                scale[kv][kb % kMaskRing][r] = f;
                            }
#pragma unroll 1
                            for (int k0 = 0; k0 < STEPS; k0 += AT_ONCE) {
                                uint4 w4[AT_ONCE];
#pragma unroll
                                for (int k = 0; k < AT_ONCE; ++k) {
                                    const int i = lt + S::LOADERS * (k0 + k), row = i / UPR, u = i % UPR;
                                    const int pg = __shfl_sync(0xFFFFFFFFu, page, row >> c.psl);
                                    w4[k] = make_uint4(0u, 0u, 0u, 0u);
                                    if (pg >= 0 && (kv == 0 || t0 + row < hi))
                                        w4[k] = __ldg(reinterpret_cast<const uint4 *>(
                                            pool + (((size_t)pg * c.nkv + hh) * c.ps + (row & (c.ps - 1))) * D + 16 * u));
                                }
#pragma unroll
                                for (int k = 0; k < AT_ONCE; ++k) {
                                    const int i = lt + S::LOADERS * (k0 + k), row = i / UPR, u = i % UPR;
                                    const uint32_t x[4] = {w4[k].x, w4[k].y, w4[k].z, w4[k].w};
                                    uint32_t y[8];
#pragma unroll
                                    for (int j = 0; j < 4; ++j) codes_bf16x2(x[j], y[2 * j], y[2 * j + 1]);
#pragma unroll
                                    for (int j = 0; j < 2; ++j) {
                                        const int uu = 2 * u + j;
                                        *reinterpret_cast<uint4 *>(dst + (uu / 8) * S::HALF + row * 128 + (((uu % 8) ^ (row & 7)) << 4)) =
                                            make_uint4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
                                    }
                                }
                            }
                            fence_proxy_async_smem();
                            mbar_arrive(&ctl->full[st]);
                        }
                    }
                    ++kb;
                }
                seg_end(sk);
            }
            issued = n;
        };
        // ================================================ MMA issuer
        auto issuer = [&]() {
            const uint32_t id_s = idesc(kBlock, false), id_o = idesc(D, true);
            int n = 0;  // ring blocks of the segments before
            uint32_t seg[2] = {0, 0}, freed[2] = {0, 0}, given[2] = {0, 0};  // tile's segments, scores read, weights given
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                warp_wait(bar, parity);
                fence_after();
                return ok;
            };
            auto copied = [&](int x) { return warp_wait(&ctl->full[x % RING], (uint32_t)(x / RING)); };
            auto s_mma = [&](int i, int x) {
                const uint64_t a = desc_k(smem_u32(sq + i * S::BLOCK)), b = desc_k(smem_u32(ring + x % RING * S::BLOCK));
#pragma unroll
                for (int h = 0; h < D / 64; ++h) mma4_ss(tmem + 128 * i, a + h * (S::HALF >> 4), b + h * (S::HALF >> 4), id_s, h);
                commit(&ctl->s_full[i]);
            };
            auto pv_mma = [&](int i, int x, uint32_t acc) {
                const uint64_t bv = desc_mn(smem_u32(ring + x % RING * S::BLOCK), S::HALF);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    mma4_ts(tmem + S::O_COL + D * i, tmem + S::P_COL + S::P_TILE * i + S::P_HALF * h, bv + (uint64_t)(h * 512), id_o,
                            h > 0 ? 1u : acc);
                commit(&ctl->o_done[i]);
            };
            for (uint32_t sg = 0; seg_begin(sg); ++sg) {
                const int last_tile = ctl->seg[sg % kSegRing].rows > kTile ? 1 : 0;
                const int nb = ctl->seg[sg % kSegRing].b1 - ctl->seg[sg % kSegRing].b0;
                // ring block of the segment's j-th keys: n + 2 j, of its values: n + 2 j + 1
                if (!copied(n)) break;
                for (int i = 0; i <= last_tile; ++i) {
                    if (!warp_wait(&ctl->q_ready[i], seg[i])) break;
                    ++seg[i];
                    issued = 1;
                    s_mma(i, n);
                }
                if (!ok) break;
                commit(&ctl->empty[n % RING]);
                auto give = [&](int i, int j) {  // tile i's weights of block j times the values
                    if (!wait(&ctl->p_full[i], given[i])) return false;
                    ++given[i];
                    pv_mma(i, n + 2 * j + 1, j > 0);
                    if (i == last_tile) commit(&ctl->empty[(n + 2 * j + 1) % RING]);
                    return true;
                };
                for (int j = 0; j < nb; ++j) {
                    // what the tensor cores need besides the weights is there long before them
                    if (!copied(n + 2 * j + 1) || (j + 1 < nb && !copied(n + 2 * j + 2))) break;
                    if constexpr (S::SPLIT) {
                        // the next scores as soon as these have been read; the second tile half a step behind
                        for (int i = 0; i <= last_tile; ++i) {
                            if (j + 1 < nb) {
                                if (!wait(&ctl->s_free[i], freed[i])) break;
                                s_mma(i, n + 2 * j + 2);
                                if (i == last_tile) commit(&ctl->empty[(n + 2 * j + 2) % RING]);
                            } else if (!wait(&ctl->s_free[i], freed[i])) {
                                break;
                            }
                            ++freed[i];
                            if (last_tile == 0) {
                                if (!give(0, j)) break;
                            } else if (i == 0) {
                                if (j > 0 && !give(1, j - 1)) break;
                            } else if (!give(0, j)) {
                                break;
                            }
                        }
                        if (ok && last_tile && j + 1 == nb) give(1, j);
                    } else {
                        // the weights lie in the scores' place: the product first
                        for (int i = 0; i <= last_tile; ++i) {
                            if (!give(i, j)) break;
                            if (j + 1 < nb) {
                                s_mma(i, n + 2 * j + 2);
                                if (i == last_tile) commit(&ctl->empty[(n + 2 * j + 2) % RING]);
                            }
                        }
                    }
                    if (!ok) break;
                }
                if (!ok) break;
                n += 2 * nb;
                seg_end(sg);
            }
        };
        // ================================================ softmax, a query row (or half of one) a thread
        if (I8 && warp >= S::LOADER) {
            regs_down<S::REG_LOAD>();
            loader();
        } else if (warp >= S::SOFTMAX) {
            regs_down<S::REG_ISSUE>();
            if (warp == S::SOFTMAX)
                issuer();
            else if (warp == S::SOFTMAX + 3)
                planner();
            else if (!I8 && warp == S::LOADER)
                loader();
        } else {
            regs_up<S::REG_SOFTMAX>();
            // a thread's positions of a block, its dimensions of O, 16-byte units of those
            constexpr int HV = S::HALVES, CW = kBlock / HV, DW = D / HV, U = DW / 8;
            const int i = warp / (4 * HV), half = HV == 1 ? 0 : (warp >> 2) & 1, row = tid & 127;
            const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
            // this thread's scores; its weights (where they take the scores' place, then its own: the
            // other half's thread may still be reading); its part of O
            const uint32_t s_tm = tmem + 128 * i + CW * half + lanes;
            const uint32_t p_tm = tmem + S::P_COL + S::P_TILE * i + S::P_HALF * half + lanes;
            const uint32_t o_tm = tmem + S::O_COL + D * i + DW * half + lanes;
            uint64_t *x_ready = &ctl->x_ready[i][warp & 3];
            auto top_of = [&](uint32_t slot, int h) -> volatile float & { return tops[slot][i][h][row]; };
            uint32_t xs = 0;  // exchanges with the other half so far
            auto exchange = [&](uint32_t slot, float v, float alone) {  // the other half's value
                if (HV == 1) return alone;
                top_of(slot, half) = v;
                mbar_arrive(x_ready);
                warp_wait(x_ready, xs);
                ++xs;
                return top_of(slot, half ^ 1);
            };
            // unit u of this half of query row r of the tile in shared memory
            auto staged = [&](int r, int u) {
                const int x = half * U + u;
                return reinterpret_cast<uint4 *>(sq + i * S::BLOCK + (x / 8) * S::HALF + r * 128 + (((x % 8) ^ (r & 7)) << 4));
            };
            uint32_t step = 0, kb = 0, n = 0;  // n: ring blocks before the current key block
            uint4 qx[U];
            bool held = false;  // the next segment's queries are in shared memory already
            auto load_q = [&](uint32_t k) {
                const Seg &g = ctl->seg[k % kSegRing];
#pragma unroll
                for (int v = 0; v < U; ++v) {
                    const int r = 32 * (warp & 3) + v * (32 / U) + lane / U;
                    qx[v] = make_uint4(0u, 0u, 0u, 0u);
                    if (i * kTile + r < g.rows)
                        qx[v] = __ldg(reinterpret_cast<const uint4 *>(p.q) + g.q_at[i * kTile + r] + (half * U + lane % U));
                }
            };
            auto give_q = [&]() {
#pragma unroll
                for (int v = 0; v < U; ++v) *staged(32 * (warp & 3) + v * (32 / U) + lane / U, lane % U) = qx[v];
                fence_proxy_async_smem();
                mbar_arrive(&ctl->q_ready[i]);
            };
            uint8_t *stage = stages + warp * 1024;
            for (uint32_t sg = 0; seg_begin(sg); ++sg) {
                const Seg &g = ctl->seg[sg % kSegRing];
                const int r0 = g.m * kPair + i * kTile;  // the tile's first query row
                const int rows = min(kTile, g.rows - i * kTile);
                const int b0 = g.b0, b1 = g.b1;
                if (rows <= 0) {
                    kb += (uint32_t)(b1 - b0);
                    n += 2u * (uint32_t)(b1 - b0);
                    seg_end(sg);
                    continue;
                }
                // queries: U lanes a row, so that a warp reads whole 64- or 128-byte runs
                if (!held) {
                    load_q(sg);
                    give_q();
                }
                held = false;
                const int lim = row < rows ? g.len - g.n + group_div(p, r0 + row) : -1;
                const int all_hi = g.all_hi[i], all_lo = g.all_lo[i];
                // rows that see nothing need no maximum
                float mx = lim < 0 ? 0.f : -INFINITY, l = 0.f, top1 = -INFINITY, top2 = -INFINITY;
                for (int b = b0; b < b1; ++b, ++kb, n += 2) {
                    if (!warp_wait(&ctl->s_full[i], step)) break;
                    ++step;
                    fence_after();
                    // written before the other half's weights of the last block, so visible now
                    const float other2 = HV == 2 && b - b0 >= 2 ? top_of((kb + 2) & 3, half ^ 1) : -INFINITY;
                    const int t0 = (b < g.nhb ? b : b - g.nhb + g.wb0) * kBlock + CW * half;  // of this thread's positions
                    const uint32_t mask = ctl->mask[kb % kMaskRing] >> (CW / 16 * half);
                    uint32_t x[CW];
                    if constexpr (CW == 128)
                        tld128(s_tm, x);
                    else
                        tld64(s_tm, x);
                    if constexpr (S::SPLIT) {
                        fence_before();
                        mbar_arrive(&ctl->s_free[i]);
                    }
                    if constexpr (I8) {
                        const float4 *ks = reinterpret_cast<const float4 *>(scale[0][kb % kMaskRing] + CW * half);
#pragma unroll
                        for (int j = 0; j < CW / 4; ++j) {
                            const float4 f = ks[j];
                            x[4 * j] = __float_as_uint(__uint_as_float(x[4 * j]) * f.x);
                            x[4 * j + 1] = __float_as_uint(__uint_as_float(x[4 * j + 1]) * f.y);
                            x[4 * j + 2] = __float_as_uint(__uint_as_float(x[4 * j + 2]) * f.z);
                            x[4 * j + 3] = __float_as_uint(__uint_as_float(x[4 * j + 3]) * f.w);
                        }
                    }
                    if ((mask & low_bits(CW / 16)) != low_bits(CW / 16) || t0 + CW - 1 > all_hi || t0 < all_lo) {
                        // a bit per position (what is seen is a range of the row and the sinks)
#pragma unroll
                        for (int k = 0; k < CW / 32; ++k) {
                            const int tb = t0 + 32 * k;
                            uint32_t see = low_bits(lim + 1 - tb);
                            if (p.window > 0) see &= ~low_bits(lim - p.window + 1 - tb) | low_bits(p.sinks - tb);
                            see &= ((mask >> (2 * k)) & 1u ? 0xFFFFu : 0u) | ((mask >> (2 * k + 1)) & 1u ? 0xFFFF0000u : 0u);
                            // most 32s of positions are seen by all of a warp's rows
                            if (__any_sync(0xFFFFFFFFu, see != 0xFFFFFFFFu)) {
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    if (!((see >> j) & 1u)) x[32 * k + j] = 0xFF800000u;
                            }
                        }
                    }
                    auto block_top = [&]() {
                        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int j = 0; j < CW; j += 8)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                m4[k] = max3(m4[k], __uint_as_float(x[j + k]), __uint_as_float(x[j + 4 + k]));
                        return max3(fmaxf(m4[0], m4[1]), m4[2], m4[3]) * p.scale_log2;
                    };
                    // the row's reference: what both halves had seen two blocks ago
                    const float seen = HV == 1 ? top1 : fmaxf(top2, other2);
                    if (__any_sync(0xFFFFFFFFu, mx == -INFINITY || seen > mx + kRise)) {
                        float nm = seen > mx + kRise ? seen : mx;
                        if (__any_sync(0xFFFFFFFFu, mx == -INFINITY)) {  // rows that have seen nothing yet
                            const float t = block_top(), u = fmaxf(t, exchange(kb & 3, t, t));
                            if (!ok) break;
                            if (mx == -INFINITY) nm = u;
                        }
                        // in two factors: what O and l hold may be as far above 1 as the reference rises
                        const float corr = nm > mx ? ex2(0.5f * (mx - nm)) : 1.f;
                        mx = nm;
                        l = l * corr * corr;
                        if (b > b0) {
                            // the last P V must be complete (without SPLIT it was issued before this block's S)
                            if (S::SPLIT && !warp_wait(&ctl->o_done[i], step - 2u)) break;
                            fence_after();
#pragma unroll 1
                            for (int d = 0; d < DW; d += 16) {
                                uint32_t o[16];
                                tld16(o_tm + d, o);
#pragma unroll
                                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * corr * corr);
                                tst16(o_tm + d, o);
                            }
                        }
                    }
                    // (a reference may lag far behind: a weight overflows only beyond 2^127 of it, which
                    // the output's check for infinities sees; so every fourth block will do)
                    auto take_top = [&]() {
                        top2 = top1;
                        top1 = b - b0 < 2 || (b & 3) == 3 ? block_top() : -INFINITY;
                    };
                    // with 104 registers the scores had better not be needed after their weights (prompt of
                    // 4,096 129.1 -> 127.1 us); with 208 it comes after them (256 tokens at 32,768 86.0, before: 86.8)
                    if (HV == 2) take_top();
                    const float base = mx == -INFINITY ? 0.f : mx;
                    const uint64_t sc2 = pack2(p.scale_log2, p.scale_log2), nb2 = pack2(-base, -base);
                    uint64_t ls[2] = {0ull, 0ull};  // sums of even and odd positions, two chains
                    const float *vs = nullptr;
                    if constexpr (I8) {
                        // the value block's scales: its copy is in once the block after the keys is full
                        if (!warp_wait(&ctl->full[(n + 1) % RING], (n + 1) / RING)) break;
                        vs = scale[1][kb % kMaskRing] + CW * half;
                    }
                    // the last weights have been used
                    if (S::SPLIT && b > b0 && !warp_wait(&ctl->o_done[i], step - 2u)) break;
                    if (S::SPLIT) fence_after();
#pragma unroll
                    for (int q = 0; q < CW / 32; ++q) {
                        uint32_t pk[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const int k = q * 32 + 2 * j;
                            float e0, e1;
                            unpack2(fma2(pack2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), sc2, nb2), e0, e1);
                            e0 = ex2(e0);
                            e1 = ex2(e1);
                            const uint64_t both = pack2(e0, e1);
                            if constexpr (I8) {
                                const float2 f = *reinterpret_cast<const float2 *>(vs + k);
                                e0 *= f.x;
                                e1 *= f.y;
                            }
                            pk[j] = cvt_bf2(e0, e1);
                            ls[j & 1] = add2(ls[j & 1], both);
                        }
                        tst16(p_tm + 16 * q, pk);
                    }
                    tst_wait();
                    fence_before();
                    mbar_arrive(&ctl->p_full[i]);
                    // off the path to the next product
                    float l0, l1;
                    unpack2(add2(ls[0], ls[1]), l0, l1);
                    l += l0 + l1;
                    if (HV == 1) take_top();
                    if (HV == 2) top_of(kb & 3, half) = top1;
                }
                // ---- the pair's output, or this piece's state
                if (!ok) break;
                if (!seg_peek(sg + 1)) break;
                held = i * kTile < ctl->seg[(sg + 1) % kSegRing].rows && ctl->seg[(sg + 1) % kSegRing].b1 > 0;
                if (held) load_q(sg + 1);
                if (!warp_wait(&ctl->o_done[i], step - 1u)) break;
                fence_after();
                // the next pair's queries first: its scores are computed while this output is written
                if (held) give_q();
                l += exchange(4, l, 0.f);
                if (!ok) break;
                if (b0 == 0 && b1 == g.nb) {
                    const float inv = l == 0.f ? 0.f : l < INFINITY ? 1.f / l : l - l;  // (a sum beyond FP32: NaN)
                    float sum = 0.f;
#pragma unroll 1
                    for (int d = 0; d < DW; d += 16) {
                        uint32_t o[16];
                        tld16(o_tm + d, o);
                        float v[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            v[k] = __uint_as_float(o[k]) * inv;
                            sum += fabsf(v[k]);
                        }
                        // through shared memory, so that whole sectors are written
                        const int flip = (lane >> 2) & 1;
                        *reinterpret_cast<uint4 *>(stage + lane * 32 + (flip << 4)) =
                            make_uint4(cvt_bf2(v[0], v[1]), cvt_bf2(v[2], v[3]), cvt_bf2(v[4], v[5]), cvt_bf2(v[6], v[7]));
                        *reinterpret_cast<uint4 *>(stage + lane * 32 + ((flip ^ 1) << 4)) =
                            make_uint4(cvt_bf2(v[8], v[9]), cvt_bf2(v[10], v[11]), cvt_bf2(v[12], v[13]), cvt_bf2(v[14], v[15]));
                        __syncwarp();
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int x = 16 * h + (lane >> 1), u = lane & 1, r = 32 * (warp & 3) + x;
                            if (r < rows)
                                reinterpret_cast<uint4 *>(p.out)[g.o_at[i * kTile + r] + ((DW * half + d) / 8 + u)] =
                                    *reinterpret_cast<const uint4 *>(stage + x * 32 + ((u ^ ((x >> 2) & 1)) << 4));
                        }
                        __syncwarp();
                    }
                    fence_before();
                    if (row < rows && !(sum < INFINITY)) ctl->again = 1;
                } else {
                    // with the sum's powers of two in the reference, so that the join's factors are those of
                    // the weights themselves, however far the reference has lagged
                    float *dst = parts + (size_t)(2 * cta + g.slot) * S::PART;
                    const int pr = i * kTile + row, up = l >= 1.f && l < INFINITY ? min(ilogbf(l), 126) : 0;
                    const float down = __uint_as_float((uint32_t)(127 - up) << 23);  // 2^-up
#pragma unroll 1
                    for (int d = 0; d < DW; d += 16) {
                        uint32_t o[16];
                        tld16(o_tm + d, o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * down);
#pragma unroll
                        for (int k = 0; k < 16; k += 4)
                            *reinterpret_cast<uint4 *>(dst + (size_t)((DW * half + d + k) / 4 * kPair + pr) * 4) =
                                make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                    }
                    fence_before();
                    if (half == 0) {
                        dst[D * kPair + pr] = mx + (float)up;
                        dst[(D + 1) * kPair + pr] = l * down;
                    }
                }
                seg_end(sg);
            }
        }
    }
    // ---- pairs that see nothing, rows that break the rules
    for (int s = cta; s < c.n_seqs; s += gridDim.x) {
        bool bad = false;
        const RowSpan r = row_span(p, s, &bad);
        if (bad && tid == 0) atomicOr(reinterpret_cast<uint32_t *>(c.state), kDevBounds);
        for (int m = 0; m < pairs_of(p, r); ++m) {
            const PairSpan a = pair_span(p, r, m);
            if (a.nb) break;  // later tokens see more
            for (int i = tid; i < a.rows * c.nkv * (D / 8); i += S::THREADS) {
                const int u = i % (D / 8), x = i / (D / 8), h = x % c.nkv, q = m * kPair + x / c.nkv;
                *reinterpret_cast<uint4 *>(p.out + (r.t0 + q / p.G) * p.o_t + (long long)(h * p.G + q % p.G) * p.o_h + 8 * u) =
                    make_uint4(0u, 0u, 0u, 0u);
            }
        }
    }
    // ---- the way out: after a timeout, what is in flight ends first
    if (!ok) {
        if (lane == 0) atomicOr(reinterpret_cast<uint32_t *>(c.state), kDevTimeout);
        uint32_t never = 0;
        deadline = global_timer() + kTimeoutNs;
        if (warp == S::SOFTMAX && issued) {
            commit(&ctl->drain);
            bounded_wait(&ctl->drain, 0u, deadline, &never);
        }
        if (!I8 && warp == S::LOADER && lane == 0)
            for (int k = max(0, issued - RING); k < issued; ++k)
                bounded_wait(&ctl->full[k % RING], (uint32_t)(k / RING) & 1u, deadline, &never);
    }
    fence_before();
    __syncthreads();
    if (warp == 0) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
    // ---- rows that came out infinite or NaN, now that no role waits for another
    if (begin < end && ctl->again && !ctl->abort && warp < S::SOFTMAX)
        rows_again<D, I8>(p, ctl->seg_s, ctl->seg_h, ctl->seg_m, (int)(begin - ctl->seg_at), end - begin, warp, S::SOFTMAX);
}

// Adds up the states of the pair that CTA blockIdx.x began, 32 of its query rows a
// block: a row a lane and 4 dimensions a warp and step, as the states are laid out;
// the output goes through shared memory, so that rows are written in whole lines.
template <int D, bool I8>
__global__ void __launch_bounds__(256) tc_join_kernel(const __grid_constant__ AttnParams p) {
    using S = TcShape<D, I8>;
    constexpr int E = D / 32;
    __shared__ __align__(16) uint16_t so[32][D + 8];
    __shared__ int again[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cta = blockIdx.x, q0 = blockIdx.y * 32;
    after_previous();
    const SegRec rec = reinterpret_cast<const SegRec *>(p.ws)[cta];
    if (rec.parts == 0) return;
    bool bad = false;
    const RowSpan r = row_span(p, rec.s, &bad);
    const int rows = min(32, r.n * p.G - rec.m * kPair - q0);  // of this block
    if (rows <= 0) return;
    if (warp == 0) again[lane] = 0;
    __syncthreads();
    const float *parts = p.ws + (size_t)p.ctas * (sizeof(SegRec) / 4);
    auto part = [&](int i) { return parts + (size_t)(2 * (cta + i) + (i == 0 ? rec.slot : 0)) * S::PART; };
    const int q = q0 + lane;
    if (lane < rows) {
        float M = -INFINITY;
#pragma unroll 4
        for (int i = 0; i < rec.parts; ++i) M = fmaxf(M, __ldcg(part(i) + D * kPair + q));
        const float base = M == -INFINITY ? 0.f : M;
        float4 o[E];
        float l = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
        for (int i = 0; i < rec.parts; ++i) {
            const float *a = part(i);
            const float f = ex2(__ldcg(a + D * kPair + q) - base);
            l = fmaf(f, __ldcg(a + (D + 1) * kPair + q), l);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float4 v = __ldcg(reinterpret_cast<const float4 *>(a) + (size_t)(warp + 8 * e) * kPair + q);
                o[e].x = fmaf(f, v.x, o[e].x);
                o[e].y = fmaf(f, v.y, o[e].y);
                o[e].z = fmaf(f, v.z, o[e].z);
                o[e].w = fmaf(f, v.w, o[e].w);
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        float sum = l;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            sum += fabsf(o[e].x) + fabsf(o[e].y) + fabsf(o[e].z) + fabsf(o[e].w);
            *reinterpret_cast<uint2 *>(&so[lane][4 * (warp + 8 * e)]) =
                make_uint2(cvt_bf2(o[e].x * inv, o[e].y * inv), cvt_bf2(o[e].z * inv, o[e].w * inv));
        }
        if (!(sum < INFINITY)) again[lane] = 1;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * (D / 8); i += 256) {
        const int row = i / (D / 8), u = i % (D / 8), x = rec.m * kPair + q0 + row, tok = group_div(p, x);
        *reinterpret_cast<uint4 *>(p.out + (r.t0 + tok) * p.o_t + (long long)(rec.h * p.G + x - tok * p.G) * p.o_h + 8 * u) =
            *reinterpret_cast<const uint4 *>(&so[row][8 * u]);
    }
    __syncthreads();
    for (int row = warp; row < rows; row += 8)
        if (again[row]) row_again<D, I8>(p, rec.s, rec.h, r.t0, r.n, r.len, rec.m * kPair + q0 + row);
}

// ------------------------------------------------------------------ host side
size_t tc_ws_bytes(int sms, int d) { return (size_t)sms * (sizeof(SegRec) + (size_t)2 * kPair * (d + 2) * 4); }

template <int D, bool I8>
static cudaError_t launch(const AttnParams &p, cudaStream_t st) {
    using S = TcShape<D, I8>;
    constexpr int smem = (2 + S::RING) * S::BLOCK + S::SCALES + S::TOPS + S::STAGE + (int)sizeof(Ctl);
    static_assert(smem > 116 * 1024 && smem <= kSmemLimit, "one CTA per SM, so that none waits for tensor memory");
    TensorMap mk, mv;
    if constexpr (I8) {
        std::memset(&mk, 0, sizeof mk);
        mv = mk;
    } else {
        const uint64_t blocks = (uint64_t)p.c.n_pages * p.c.nkv;
        if (!encode_bf16_3d(&mk, p.c.k, D, (uint64_t)p.c.ps, blocks, (uint32_t)p.c.ps) ||
            !encode_bf16_3d(&mv, p.c.v, D, (uint64_t)p.c.ps, blocks, (uint32_t)p.c.ps))
            return cudaErrorInvalidValue;
    }
    cudaError_t e = cudaFuncSetAttribute(tc_kernel<D, I8>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if ((e = launch_next(tc_kernel<D, I8>, dim3((unsigned)p.ctas), dim3(S::THREADS), smem, st, p, mk, mv)) != cudaSuccess) return e;
    return launch_next(tc_join_kernel<D, I8>, dim3((unsigned)p.ctas, kPair / 32), dim3(256), 0, st, p);
}

cudaError_t tc_launch(const AttnParams &p0, int sms, cudaStream_t st) {
    AttnParams p = p0;
    p.ctas = sms;
    if (p.c.d == 64) return p.c.i8 ? launch<64, true>(p, st) : launch<64, false>(p, st);
    return p.c.i8 ? launch<128, true>(p, st) : launch<128, false>(p, st);
}

}  // namespace paged
}  // namespace tiles
