// The paged KV cache: its layout and checks, the pages' life (resize with
// copy-on-write, fork, trim, compact), and appending rows (the pages' own cache
// is dense and of one sequence; a pool of shared pages has no counterpart
// there).
//
// The page tables, lengths and reference counts stay on the device, so that no
// call waits for the host and all can be captured. Deciding which page goes
// where is a small amount of work in a strict order (rows in order, lowest free
// page first), so one CTA does it, with block-wide counts in place of a loop
// over rows; moving the pages' bytes is a second kernel over the whole GPU that
// reads the list the first one left.
#include <cuda_runtime.h>

#include <algorithm>

#include "megakernel.cuh"
#include "paged_internal.h"

namespace tiles {
namespace paged {

constexpr int kBookThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kRowsShared = 2048;  // rows whose first slot and length resize keeps in shared memory

// Words that other threads of the kernel change: read at L2.
__device__ __forceinline__ int ldw(const int32_t *p) { return __ldcg(p); }

struct Book {
    int32_t *status, *copies, *refs, *writers, *lowest, *src, *dst, *freelist, *first, *kinds;
};
__host__ __device__ __forceinline__ Book book_of(int32_t *state, int P, int n_seqs) {
    Book b;
    b.status = state + kStateStatus;
    b.copies = state + kStateCopies;
    b.refs = state + kStateRefs;
    b.writers = b.refs + P;
    b.lowest = b.refs + 2 * (size_t)P;
    b.src = b.refs + 3 * (size_t)P;
    b.dst = b.refs + 4 * (size_t)P;
    b.freelist = b.refs + 5 * (size_t)P;
    b.first = b.refs + kStateArrays * (size_t)P;
    b.kinds = b.first + n_seqs;
    return b;
}

// Exclusive sum over the block's threads, in thread order; *total the sum.
__device__ __forceinline__ int block_excl(int v, int *warps, int *total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // the last call's values have been read
    if (lane == 31) warps[w] = x;
    __syncthreads();
    if (w == 0) {
        int t = lane < (int)(blockDim.x >> 5) ? warps[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, t, o);
            if (lane >= o) t += y;
        }
        warps[lane] = t;
    }
    __syncthreads();
    *total = warps[(blockDim.x >> 5) - 1];
    return x - v + (w ? warps[w - 1] : 0);
}

// ------------------------------------------------------------------ resize
// One CTA, in steps with a barrier between them:
//   1. rows that shrink drop their pages, a warp a row (reference counts go down);
//   2. the pages that growing rows will write ("slots": row s, table entry j) are
//      numbered in order; from here on a thread takes a slot;
//   3. slots whose page is shared: count the page's writers and find the lowest
//      row among them, which keeps the page if every holder writes;
//   4. the slots that need a page, numbered in order;
//   5. the lowest free pages, as many as needed;
//   6. they are handed out in order, and the pages whose contents move are listed.
// What bounds it is the chain of dependent L2 accesses (a step reads what the one
// before it wrote, so counts and table words go through L2), hence a slot a thread
// with its page, count and decision in registers. More than kBookThreads slots
// take further rounds, whose decisions wait in memory (kinds). 72 rows that all grow
// by one: 9 us with the launch (a warp a row, reading everything anew in each step: 18).
__global__ void __launch_bounds__(kBookThreads) resize_kernel(View c, const int32_t *__restrict__ new_lens) {
    __shared__ int warps[32], first_s[kRowsShared], len_s[kRowsShared], new_s[kRowsShared];
    __shared__ int n_copies;
    const Book b = book_of(c.state, c.n_pages, c.n_seqs);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool shared = c.n_seqs <= kRowsShared;
    after_previous();
    const int P = c.n_pages, W = c.width, ps = c.ps;
    uint32_t flags = 0;
    if (tid == 0) n_copies = 0;

    // row s: old and new length; a row that is left alone has new == old
    auto row = [&](int s, int *len, int *nl) {
        *len = ldw(c.lens + s);
        int n = __ldg(new_lens + s);
        if (*len < 0 || (long long)*len > (long long)W * ps || (long long)n > (long long)W * ps) {
            flags |= kDevBounds;
            n = *len;
        }
        *nl = n < 0 ? *len : n;
    };

    // 1, 2: a thread a row, then a warp each row that shrinks
    long long slots = 0;
    for (int s0 = 0; s0 < c.n_seqs; s0 += kBookThreads) {
        const int s = s0 + tid;
        int len = 0, nl = 0;
        if (s < c.n_seqs) row(s, &len, &nl);
        const int mine = nl > len ? ((nl + ps - 1) >> c.psl) - (len >> c.psl) : 0;
        int sum;
        const int before = block_excl(mine, warps, &sum);
        if (s < c.n_seqs && shared) {
            first_s[s] = (int)slots + before;
            len_s[s] = len;
            new_s[s] = nl;
        } else if (s < c.n_seqs) {
            b.first[s] = (int)slots + before;
        }
        slots += sum;
    }
    __syncthreads();
    for (int s = warp; s < c.n_seqs; s += kBookThreads / 32) {
        int len, nl;
        if (shared) {
            len = len_s[s];
            nl = new_s[s];
        } else {
            row(s, &len, &nl);
        }
        if (nl >= len) continue;
        int32_t *t = c.tables + (size_t)s * W;
        for (int j = ((nl + ps - 1) >> c.psl) + lane; j < W; j += 32) {
            const int page = t[j];
            if (page == -1) continue;
            if (page >= 0 && page < P)
                atomicSub(b.refs + page, 1);
            else
                flags |= kDevBounds;
            t[j] = -1;
        }
        __syncwarp();
        if (lane == 0) c.lens[s] = nl;
    }
    __syncthreads();
    const int C = (int)slots;  // at most n_seqs * W
    // slot k's row: the last with first[s] <= k (rows without slots share the next row's first)
    auto first_of = [&](int s) { return shared ? first_s[s] : ldw(b.first + s); };
    auto row_of = [&](int k) {
        int lo = 0, n = c.n_seqs;
        while (n > 1) {
            const int h = n / 2;
            if (first_of(lo + h) <= k) {
                lo += h;
                n -= h;
            } else {
                n = h;
            }
        }
        return lo;
    };
    int my_s = 0, my_j = 0, my_len = 0, my_page = -1, my_ref = 0, my_kind = 0;  // of the first round's slot
    auto slot = [&](int k, int *s, int *j, int *len, int *page, int *ref) {
        *s = row_of(k);
        *len = shared ? len_s[*s] : ldw(c.lens + *s);
        *j = (*len >> c.psl) + k - first_of(*s);
        *page = ldw(c.tables + (size_t)*s * W + *j);
        *ref = *page >= 0 && *page < P ? ldw(b.refs + *page) : 0;
    };
    // 3
    for (int k = tid; k < C; k += kBookThreads) {
        int s, j, len, page, ref;
        slot(k, &s, &j, &len, &page, &ref);
        if (ref > 1) {
            b.writers[page] = 0;  // the same words from every writer
            b.lowest[page] = 0x7FFFFFFF;
        }
        if (k == tid) {
            my_s = s;
            my_j = j;
            my_len = len;
            my_page = page;
            my_ref = ref;
        }
    }
    __syncthreads();
    for (int k = tid; k < C; k += kBookThreads) {
        int s = my_s, j = my_j, len = my_len, page = my_page, ref = my_ref;
        if (k != tid) slot(k, &s, &j, &len, &page, &ref);
        if (ref > 1) {
            atomicAdd(b.writers + page, 1);
            atomicMin(b.lowest + page, s);
        }
    }
    __syncthreads();
    // 4. kinds: 0 has its own page, 1 needs one, 2 needs one in place of a shared one
    int need = 0, my_rank = 0;
    for (int k0 = 0; k0 < C; k0 += kBookThreads) {
        const int k = k0 + tid;
        int kind = 0;
        if (k < C) {
            int s = my_s, j = my_j, len = my_len, page = my_page, ref = my_ref;
            if (k0) slot(k, &s, &j, &len, &page, &ref);
            if (page < 0 || page >= P)
                kind = 1;
            else if (ref > 1)
                kind = ldw(b.writers + page) == ref && ldw(b.lowest + page) == s ? 0 : 2;
            if (k0)
                b.kinds[k] = kind;
            else
                my_kind = kind;
        }
        int sum;
        const int before = block_excl(kind != 0, warps, &sum);
        if (k0 == 0) my_rank = before;
        need += sum;
    }
    // 5
    int found = 0;
    for (int p0 = 0; p0 < P && found < need; p0 += 4 * kBookThreads) {
        const int p = p0 + 4 * tid;
        bool fr[4];
        int n = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            fr[i] = p + i < P && ldw(b.refs + p + i) <= 0;
            n += fr[i];
        }
        int sum, at;
        at = found + block_excl(n, warps, &sum);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (fr[i]) b.freelist[at++] = p + i;
        found += sum;
    }
    __syncthreads();
    // 6
    if (found < need) {
        flags |= kDevNoPages;
    } else {
        int given = 0;
        for (int k0 = 0; k0 < C; k0 += kBookThreads) {
            const int k = k0 + tid;
            int s = my_s, j = my_j, len = my_len, page = my_page, ref, kind = my_kind, rank = my_rank;
            if (k0) {
                kind = 0;
                if (k < C) {
                    slot(k, &s, &j, &len, &page, &ref);
                    kind = ldw(b.kinds + k);
                }
                int sum;
                rank = given + block_excl(kind != 0, warps, &sum);
                given += sum;
            } else if (C > kBookThreads) {
                block_excl(kind != 0, warps, &given);
            }
            if (k >= C || kind == 0) continue;
            if (kind == 1 && page != -1) flags |= kDevBounds;
            const int fresh = ldw(b.freelist + rank);
            c.tables[(size_t)s * W + j] = fresh;
            b.refs[fresh] = 1;
            if (kind == 2) {
                atomicSub(b.refs + page, 1);
                if ((long long)j * ps < len) {
                    const int i = atomicAdd(&n_copies, 1);
                    b.src[i] = page;
                    b.dst[i] = fresh;
                }
            }
        }
        __syncthreads();  // the lengths have been read
        for (int s = tid; s < c.n_seqs; s += kBookThreads) {
            int len = 0, nl = 0;
            if (shared) {
                len = len_s[s];
                nl = new_s[s];
            } else {
                row(s, &len, &nl);
            }
            if (nl > len) c.lens[s] = nl;
        }
    }
    if (flags) atomicOr(reinterpret_cast<uint32_t *>(b.status), flags);
    __syncthreads();
    if (tid == 0) *b.copies = n_copies;
}

// ------------------------------------------------------------------ moving pages
// Copies page src[i] to dst[i] in every layer of both pools, i < the count the
// kernel before left. A page of one layer is contiguous in its pool. Sources
// and targets are different pages, so the order does not matter. Bound by the
// memory: each 16-byte word is read once and written once, four in flight per
// thread (540 MB moved in 160 us, 6.8 TB/s, the measured copy rate). With remap, also
// rewrites the page tables (compact).
__device__ __forceinline__ void move_bytes(const uint8_t *src, uint8_t *dst, long long n16, long long i, long long step) {
    const uint4 *a = reinterpret_cast<const uint4 *>(src);
    uint4 *d = reinterpret_cast<uint4 *>(dst);
    for (; i + 3 * step < n16; i += 4 * step) {
        const uint4 x0 = __ldcs(a + i), x1 = __ldcs(a + i + step), x2 = __ldcs(a + i + 2 * step),
                    x3 = __ldcs(a + i + 3 * step);
        __stcs(d + i, x0);
        __stcs(d + i + step, x1);
        __stcs(d + i + 2 * step, x2);
        __stcs(d + i + 3 * step, x3);
    }
    for (; i < n16; i += step) __stcs(d + i, __ldcs(a + i));
}

__global__ void __launch_bounds__(kMoveThreads) move_kernel(View c, int remap) {
    const Book b = book_of(c.state, c.n_pages, c.n_seqs);
    after_previous();
    const int n = *b.copies;
    const long long block = (long long)c.nkv * c.ps * c.d * (c.i8 ? 1 : 2), scales = (long long)c.nkv * c.ps * 4;
    // one work item: a page of one layer of K or of V
    const long long items = (long long)n * c.n_layers * 2;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int kv = (int)(it & 1);
        const long long r = it >> 1;
        const int i = (int)(r % n);
        const long long layer = r / n;
        const long long from = layer * c.n_pages + b.src[i], to = layer * c.n_pages + b.dst[i];
        uint8_t *pool = kv ? c.v : c.k;
        move_bytes(pool + from * block, pool + to * block, block / 16, threadIdx.x, kMoveThreads);
        if (c.i8) {
            uint8_t *sc = reinterpret_cast<uint8_t *>(kv ? c.vs : c.ks);
            move_bytes(sc + from * scales, sc + to * scales, scales / 16, threadIdx.x, kMoveThreads);
        }
    }
    if (remap) {
        const long long total = (long long)c.n_seqs * c.width;
        for (long long i = (long long)blockIdx.x * kMoveThreads + threadIdx.x; i < total;
             i += (long long)gridDim.x * kMoveThreads) {
            const int page = c.tables[i];
            if (page >= 0 && page < c.n_pages) {
                const int to = b.writers[page];
                if (to != page) c.tables[i] = to;
            } else if (page != -1) {
                atomicOr(reinterpret_cast<uint32_t *>(b.status), kDevBounds);
            }
        }
    }
}

// ------------------------------------------------------------------ fork
// One warp per row.
__global__ void __launch_bounds__(32) fork_kernel(View c, const int32_t *__restrict__ src_rows) {
    const Book b = book_of(c.state, c.n_pages, c.n_seqs);
    const int s = blockIdx.x, lane = threadIdx.x, W = c.width;
    after_previous();
    const int from = src_rows[s];
    if (from < 0) return;
    bool ok = from < c.n_seqs && from != s && src_rows[from] < 0 && c.lens[s] == 0;
    int32_t *t = c.tables + (size_t)s * W;
    if (ok) {
        bool empty = true;
        for (int j = lane; j < W; j += 32) empty &= t[j] == -1;
        ok = __all_sync(0xFFFFFFFFu, empty);
    }
    int len = 0;
    if (ok) {
        len = c.lens[from];
        ok = len >= 0 && (long long)len <= (long long)W * c.ps;
    }
    if (!ok) {
        if (lane == 0) atomicOr(reinterpret_cast<uint32_t *>(b.status), kDevBounds);
        return;
    }
    const int32_t *f = c.tables + (size_t)from * W;
    for (int j = lane; j < (len + c.ps - 1) / c.ps; j += 32) {
        const int page = f[j];
        if (page >= 0 && page < c.n_pages) {
            atomicAdd(b.refs + page, 1);
            t[j] = page;
        } else if (page != -1) {
            atomicOr(reinterpret_cast<uint32_t *>(b.status), kDevBounds);
        }
    }
    if (lane == 0) c.lens[s] = len;
}

// ------------------------------------------------------------------ trim
// One warp per row: pages that begin at or behind `sinks` and end at or before
// position len - window.
__global__ void __launch_bounds__(32) trim_kernel(View c, int window, int sinks) {
    const Book b = book_of(c.state, c.n_pages, c.n_seqs);
    const int s = blockIdx.x, lane = threadIdx.x, ps = c.ps;
    after_previous();
    int len = c.lens[s];
    if (len > c.width * ps) len = c.width * ps;
    const int last = len - window;  // positions <= last are seen by no later token
    int32_t *t = c.tables + (size_t)s * c.width;
    const int j0 = (int)(((long long)sinks + ps - 1) / ps);
    for (long long j = j0 + lane; j < c.width && (j + 1) * ps - 1 <= last; j += 32) {
        const int page = t[j];
        if (page == -1) continue;
        if (page >= 0 && page < c.n_pages)
            atomicSub(b.refs + page, 1);
        else
            atomicOr(reinterpret_cast<uint32_t *>(b.status), kDevBounds);
        t[j] = -1;
    }
}

// ------------------------------------------------------------------ compact
// One CTA: the pages' new places (writers[page]) and the list of moves; the
// tables follow in move_kernel.
__global__ void __launch_bounds__(kBookThreads) compact_kernel(View c) {
    __shared__ int warps[32];
    const Book b = book_of(c.state, c.n_pages, c.n_seqs);
    const int tid = threadIdx.x, P = c.n_pages;
    after_previous();
    int live = 0, sum;
    for (int p = tid; p < P; p += kBookThreads) live += b.refs[p] > 0;
    block_excl(live, warps, &sum);
    const int n_live = sum;
    int holes = 0, movers = 0;
    for (int p0 = 0; p0 < P; p0 += kBookThreads) {
        const int p = p0 + tid;
        const bool lv = p < P && b.refs[p] > 0;
        const bool hole = p < P && !lv && p < n_live, mover = lv && p >= n_live;
        if (p < P) b.writers[p] = p;
        const int ah = holes + block_excl(hole, warps, &sum);
        holes += sum;
        const int am = movers + block_excl(mover, warps, &sum);
        movers += sum;
        if (hole) b.dst[ah] = p;
        if (mover) b.src[am] = p;
    }
    __syncthreads();
    for (int i = tid; i < movers; i += kBookThreads) {  // as many holes as movers
        const int from = b.src[i], to = b.dst[i];
        b.writers[from] = to;
        b.refs[to] = b.refs[from];
        b.refs[from] = 0;
    }
    if (tid == 0) *b.copies = movers;
}

// ------------------------------------------------------------------ append
// One warp per token and group of its rows; lanes take 8 elements each, so a row
// is D / 8 lanes and a warp holds 256 / D rows (K and V rows of the token's heads) a
// step. Bound by the chain from a token's number to its row's place (offsets, length,
// page), so the rows are read before it, four steps at once. INT8 rows are quantized
// by the lanes that hold them (s = max |x| / 127 over the row, a butterfly over D / 8
// lanes). 64 tokens of 8 heads at D 128 4.1 us with the launch; 10,570 tokens at D 64
// (43 MB) 8.2 us, 5.3 TB/s.
constexpr int kAppendWarps = 8, kAppendSteps = 4;

// The row of token t: the last s with cu[s] <= t, or -1 for padding.
__device__ __forceinline__ int row_of_token(const int32_t *__restrict__ cu, int n_seqs, int t, int lane) {
    int lo = 0, n = n_seqs + 1;  // the answer + 1 = number of cu entries <= t, searched in [lo, lo + n)
    while (n > 32) {
        const int step = (n + 31) / 32, i = lo + lane * step;
        const bool le = i < lo + n && __ldg(cu + i) <= t;
        const int k = __popc(__ballot_sync(0xFFFFFFFFu, le));
        if (k == 0) return -1;
        const int at = lo + (k - 1) * step;
        n = min(step, lo + n - at);
        lo = at;
    }
    const bool le = lane < n && __ldg(cu + lo + lane) <= t;
    const int k = lo + __popc(__ballot_sync(0xFFFFFFFFu, le)) - 1;
    return k >= n_seqs ? -1 : k;
}

template <int D, bool I8>
__global__ void __launch_bounds__(kAppendWarps * 32)
    append_kernel(View c, const uint16_t *__restrict__ k, long long k_t, long long k_h, const uint16_t *__restrict__ v,
                  long long v_t, long long v_h, const int32_t *__restrict__ cu, int n_tokens) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;  // lanes a row, rows a warp and step
    const int lane = threadIdx.x & 31, sub = lane / LPR, e = (lane % LPR) * 8;
    const int t = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    after_previous();
    if (t >= n_tokens) return;
    const int rows = 2 * c.nkv;  // (K or V, head)
    const int r_first = blockIdx.y * kAppendSteps * RPW, r_step = gridDim.y * kAppendSteps * RPW;
    uint4 xs[kAppendSteps];
    auto load = [&](int r0) {
#pragma unroll
        for (int i = 0; i < kAppendSteps; ++i) {
            const int r = r0 + i * RPW + sub;
            const bool isv = r >= c.nkv;
            const int h = isv ? r - c.nkv : r;
            xs[i] = make_uint4(0u, 0u, 0u, 0u);
            if (r < rows)
                xs[i] = __ldg(reinterpret_cast<const uint4 *>(isv ? v + t * v_t + h * v_h + e : k + t * k_t + h * k_h + e));
        }
    };
    load(r_first);
    int s, pos;
    if (cu) {
        s = row_of_token(cu, c.n_seqs, t, lane);
        if (s < 0) return;
        pos = __ldg(c.lens + s) - __ldg(cu + s + 1) + t;
    } else {
        s = t;
        pos = __ldg(c.lens + s) - 1;
    }
    if (pos < 0) return;
    int page = -1;
    if (pos < c.width * c.ps) page = __ldg(c.tables + (size_t)s * c.width + (pos >> c.psl));
    if (page < 0 || page >= c.n_pages) {
        if (lane == 0) atomicOr(reinterpret_cast<uint32_t *>(c.state), kDevBounds);
        return;
    }
    for (int r0 = r_first; r0 < rows; r0 += r_step) {
        if (r0 != r_first) load(r0);
#pragma unroll
        for (int i0 = 0; i0 < kAppendSteps; ++i0) {
            const int r = r0 + i0 * RPW + sub;
            const bool in = r < rows, isv = r >= c.nkv;
            const int h = isv ? r - c.nkv : r;
            const uint4 x = xs[i0];
            const size_t at = ((size_t)page * c.nkv + h) * c.ps + (pos & (c.ps - 1));  // row of the layer's pool
            if constexpr (!I8) {
                if (in) *reinterpret_cast<uint4 *>((isv ? c.v : c.k) + (at * D + e) * 2) = x;
            } else {
                float f[8], amax = 0.f;
                unpack8(x, f);
                if (in && !isv && c.k_shift) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = __fsub_rn(f[i], __ldg(c.k_shift + h * D + e + i));
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
                const float sc = __fdiv_rn(amax, 127.0f);
                uint32_t w[2] = {0u, 0u};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float qf = sc > 0.f ? rintf(__fdiv_rn(f[i], sc)) : 0.f;
                    const int q = (int)fminf(fmaxf(qf, -127.f), 127.f);
                    w[i / 4] |= ((uint32_t)q & 0xFFu) << (8 * (i % 4));
                }
                if (in) {
                    *reinterpret_cast<uint2 *>((isv ? c.v : c.k) + at * D + e) = make_uint2(w[0], w[1]);
                    if (e == 0) (isv ? c.vs : c.ks)[at] = sc;
                }
            }
        }
    }
}

// One warp per token.
__global__ void __launch_bounds__(32) positions_kernel(const int32_t *__restrict__ lens, int n_seqs,
                                                       const int32_t *__restrict__ cu, int max_pos, int32_t *pos,
                                                       uint32_t *status) {
    const int t = blockIdx.x, lane = threadIdx.x;
    after_previous();
    int p = -1;
    if (cu) {
        const int s = row_of_token(cu, n_seqs, t, lane);
        if (s >= 0) p = __ldg(lens + s) - __ldg(cu + s + 1) + t;
    } else {
        p = __ldg(lens + t) - 1;
    }
    if (lane) return;
    if (p >= max_pos) {
        atomicOr(status, kDevBounds);
        p = -1;
    }
    pos[t] = p < 0 ? -1 : p;
}

cudaError_t positions_launch(const tiles_paged_cache &cache, const int32_t *cu, int n_tokens, int max_pos, int32_t *pos,
                             uint32_t *status, cudaStream_t st) {
    return launch_next(positions_kernel, dim3((unsigned)n_tokens), dim3(32), 0, st, cache.lens, cache.desc.n_seqs, cu, max_pos, pos,
                       status);
}

}  // namespace paged
}  // namespace tiles

using namespace tiles;
using namespace tiles::paged;

namespace {

bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool al4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

tiles_status_t check_desc(const tiles_paged_desc &d) {
    if (d.n_layers < 1 || d.n_kv_heads < 1 || d.head_dim < 1 || d.page_size < 1 || d.n_pages < 1 || d.n_seqs < 1 ||
        d.table_width < 1 || (d.kv_format != TILES_KV_BF16 && d.kv_format != TILES_KV_INT8))
        return TILES_ERR_INVALID_ARG;
    if (d.head_dim != 64 && d.head_dim != 128) return TILES_ERR_UNSUPPORTED;
    if (d.page_size != 16 && d.page_size != 32 && d.page_size != 64 && d.page_size != 128) return TILES_ERR_UNSUPPORTED;
    const long long lim = 0x7FFFFFFFll;
    if ((long long)d.n_pages * d.n_kv_heads > lim / d.n_layers ||
        (long long)d.n_pages * d.n_kv_heads > lim / (d.page_size / 16) ||
        (long long)d.table_width * d.page_size > lim / 4 ||
        (long long)d.n_seqs * d.n_kv_heads > lim / 16 || (long long)d.n_seqs * d.table_width > lim)
        return TILES_ERR_UNSUPPORTED;
    return TILES_OK;
}

void layout_of(const tiles_paged_desc &d, tiles_paged_layout *o) {
    const int64_t rows = (int64_t)d.n_layers * d.n_pages * d.n_kv_heads * d.page_size;
    if (d.kv_format == TILES_KV_INT8) {
        o->k_scale_off = o->v_scale_off = (rows * d.head_dim + 255) / 256 * 256;
        o->k_bytes = o->v_bytes = o->k_scale_off + rows * 4;
    } else {
        o->k_scale_off = o->v_scale_off = 0;
        o->k_bytes = o->v_bytes = rows * d.head_dim * 2;
    }
    o->state_bytes = 4 * ((int64_t)kStateRefs + (int64_t)kStateArrays * d.n_pages + d.n_seqs + (int64_t)d.n_seqs * d.table_width);
}

tiles_status_t check_cache(const tiles_paged_cache *c) {
    if (!c) return TILES_ERR_INVALID_ARG;
    const tiles_status_t st = check_desc(c->desc);
    if (st != TILES_OK) return st;
    if (!c->k || !c->v || !c->tables || !c->lens || !c->state || !al16(c->k) || !al16(c->v) || !al4(c->tables) ||
        !al4(c->lens) || !al16(c->state) || !al4(c->k_shift) || (c->k_shift && c->desc.kv_format != TILES_KV_INT8))
        return TILES_ERR_INVALID_ARG;
    return TILES_OK;
}

}  // namespace

tiles_status_t tiles::paged::cache_check(const tiles_paged_cache *cache) { return check_cache(cache); }

namespace {

// The pools from `layer` on.
View view_of(const tiles_paged_cache &c, int layer) {
    const tiles_paged_desc &d = c.desc;
    tiles_paged_layout lay;
    layout_of(d, &lay);
    const size_t rows = (size_t)layer * d.n_pages * d.n_kv_heads * d.page_size;
    const bool i8 = d.kv_format == TILES_KV_INT8;
    View v;
    v.k = static_cast<uint8_t *>(c.k) + rows * d.head_dim * (i8 ? 1 : 2);
    v.v = static_cast<uint8_t *>(c.v) + rows * d.head_dim * (i8 ? 1 : 2);
    v.ks = i8 ? reinterpret_cast<float *>(static_cast<uint8_t *>(c.k) + lay.k_scale_off) + rows : nullptr;
    v.vs = i8 ? reinterpret_cast<float *>(static_cast<uint8_t *>(c.v) + lay.v_scale_off) + rows : nullptr;
    v.tables = c.tables;
    v.lens = c.lens;
    v.state = c.state;
    v.k_shift = c.k_shift ? c.k_shift + (size_t)layer * d.n_kv_heads * d.head_dim : nullptr;
    v.n_layers = d.n_layers;
    v.nkv = d.n_kv_heads;
    v.d = d.head_dim;
    v.ps = d.page_size;
    v.psl = d.page_size == 16 ? 4 : d.page_size == 32 ? 5 : d.page_size == 64 ? 6 : 7;
    v.n_pages = d.n_pages;
    v.n_seqs = d.n_seqs;
    v.width = d.table_width;
    v.i8 = i8;
    return v;
}

tiles_status_t sm_count(int *sms) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return TILES_ERR_CUDA;
    return TILES_OK;
}

// Up to 16 query rows a (sequence, KV head) fit one MMA tile of the streaming
// kernel, which is bound by the cache's bytes; more go to the tensor cores, as each
// further tile reads the pages again. (17 tokens of one sequence, group 2, 1,023
// positions, D 64: 21.5 us there, 30.7 us streaming.)
bool streams(int G, int max_tokens) { return (long long)G * max_tokens <= 16; }

int64_t attn_ws_bytes(const tiles_paged_desc &d, int n_q_heads, int max_tokens, int sms) {
    return (int64_t)(streams(n_q_heads / d.n_kv_heads, max_tokens) ? stream_ws_bytes(sms, d.head_dim)
                                                                  : tc_ws_bytes(sms, d.head_dim));
}

tiles_status_t launched(cudaError_t e) { return e == cudaSuccess ? TILES_OK : TILES_ERR_CUDA; }

}  // namespace

extern "C" {

tiles_status_t tiles_paged_get_layout(const tiles_paged_desc *desc, tiles_paged_layout *out) {
    if (!desc || !out) return TILES_ERR_INVALID_ARG;
    const tiles_status_t st = check_desc(*desc);
    if (st == TILES_OK) layout_of(*desc, out);
    return st;
}

tiles_status_t tiles_paged_reset(const tiles_paged_cache *cache, void *stream) {
    const tiles_status_t st = check_cache(cache);
    if (st != TILES_OK) return st;
    const tiles_paged_desc &d = cache->desc;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    tiles_paged_layout lay;
    layout_of(d, &lay);
    if (cudaMemsetAsync(cache->tables, 0xFF, (size_t)d.n_seqs * d.table_width * 4, cs) != cudaSuccess ||
        cudaMemsetAsync(cache->lens, 0, (size_t)d.n_seqs * 4, cs) != cudaSuccess ||
        cudaMemsetAsync(cache->state, 0, (size_t)lay.state_bytes, cs) != cudaSuccess)
        return TILES_ERR_CUDA;
    return TILES_OK;
}

tiles_status_t tiles_paged_resize(const tiles_paged_cache *cache, const int32_t *new_lens, void *stream) {
    tiles_status_t st = check_cache(cache);
    if (st != TILES_OK) return st;
    int sms = 0;
    if (!new_lens || !al4(new_lens)) return TILES_ERR_INVALID_ARG;
    if ((st = sm_count(&sms)) != TILES_OK) return st;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const View v = view_of(*cache, 0);
    if ((st = launched(launch_next(resize_kernel, dim3(1), dim3(kBookThreads), 0, cs, v, new_lens))) != TILES_OK) return st;
    return launched(launch_next(move_kernel, dim3((unsigned)(sms * 8)), dim3(kMoveThreads), 0, cs, v, 0));
}

tiles_status_t tiles_paged_fork(const tiles_paged_cache *cache, const int32_t *src_rows, void *stream) {
    const tiles_status_t st = check_cache(cache);
    if (st != TILES_OK) return st;
    if (!src_rows || !al4(src_rows)) return TILES_ERR_INVALID_ARG;
    return launched(launch_next(fork_kernel, dim3((unsigned)cache->desc.n_seqs), dim3(32), 0,
                                reinterpret_cast<cudaStream_t>(stream), view_of(*cache, 0), src_rows));
}

tiles_status_t tiles_paged_trim(const tiles_paged_cache *cache, int32_t window, int32_t sinks, void *stream) {
    const tiles_status_t st = check_cache(cache);
    if (st != TILES_OK) return st;
    if (window < 1 || sinks < 0) return TILES_ERR_INVALID_ARG;
    return launched(launch_next(trim_kernel, dim3((unsigned)cache->desc.n_seqs), dim3(32), 0,
                                reinterpret_cast<cudaStream_t>(stream), view_of(*cache, 0), window, sinks));
}

tiles_status_t tiles_paged_compact(const tiles_paged_cache *cache, void *stream) {
    tiles_status_t st = check_cache(cache);
    if (st != TILES_OK) return st;
    int sms = 0;
    if ((st = sm_count(&sms)) != TILES_OK) return st;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const View v = view_of(*cache, 0);
    if ((st = launched(launch_next(compact_kernel, dim3(1), dim3(kBookThreads), 0, cs, v))) != TILES_OK) return st;
    return launched(launch_next(move_kernel, dim3((unsigned)(sms * 8)), dim3(kMoveThreads), 0, cs, v, 1));
}

tiles_status_t tiles_paged_append(const tiles_paged_cache *cache, int32_t layer, const void *k, int64_t k_stride_token,
                                  int64_t k_stride_head, const void *v, int64_t v_stride_token,
                                  int64_t v_stride_head, const int32_t *cu_tokens, int32_t n_tokens, void *stream) {
    const tiles_status_t st = check_cache(cache);
    if (st != TILES_OK) return st;
    const tiles_paged_desc &d = cache->desc;
    if (layer < 0 || layer >= d.n_layers || n_tokens < 0 || (!cu_tokens && n_tokens != d.n_seqs) || !al4(cu_tokens))
        return TILES_ERR_INVALID_ARG;
    if (n_tokens == 0) return TILES_OK;
    if (!k || !v || !al16(k) || !al16(v) || k_stride_token % 8 || k_stride_head % 8 || v_stride_token % 8 ||
        v_stride_head % 8)
        return TILES_ERR_INVALID_ARG;
    const View c = view_of(*cache, layer);
    const uint16_t *kp = static_cast<const uint16_t *>(k), *vp = static_cast<const uint16_t *>(v);
    // a warp's steps a token: all at once, so that a token's rows go to as few warps as that takes
    const int steps = (2 * d.n_kv_heads * d.head_dim / 8 + 31) / 32;
    const int gy = std::min((steps + kAppendSteps - 1) / kAppendSteps, 65535);
    const dim3 grid((unsigned)((n_tokens + kAppendWarps - 1) / kAppendWarps), (unsigned)gy);
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    auto go = [&](auto kernel) {
        return launched(launch_next(kernel, grid, dim3(kAppendWarps * 32), 0, cs, c, kp, (long long)k_stride_token,
                                    (long long)k_stride_head, vp, (long long)v_stride_token, (long long)v_stride_head, cu_tokens,
                                    n_tokens));
    };
    if (d.head_dim == 64) return c.i8 ? go(append_kernel<64, true>) : go(append_kernel<64, false>);
    return c.i8 ? go(append_kernel<128, true>) : go(append_kernel<128, false>);
}

tiles_status_t tiles_paged_workspace_bytes(const tiles_paged_desc *desc, int32_t n_q_heads, int32_t max_tokens,
                                           int64_t *bytes) {
    if (!desc || !bytes || max_tokens < 1) return TILES_ERR_INVALID_ARG;
    tiles_status_t st = check_desc(*desc);
    if (st != TILES_OK) return st;
    if (n_q_heads < 1 || n_q_heads % desc->n_kv_heads) return TILES_ERR_INVALID_ARG;
    if (n_q_heads / desc->n_kv_heads > 16) return TILES_ERR_UNSUPPORTED;
    int sms = 0;
    if ((st = sm_count(&sms)) != TILES_OK) return st;
    *bytes = attn_ws_bytes(*desc, n_q_heads, max_tokens, sms);
    return TILES_OK;
}

tiles_status_t tiles_paged_attention(const tiles_paged_cache *cache, int32_t layer, int32_t n_q_heads, const void *q,
                                     int64_t q_stride_token, int64_t q_stride_head, void *out,
                                     int64_t out_stride_token, int64_t out_stride_head, const int32_t *cu_tokens,
                                     int32_t n_tokens, int32_t max_tokens, float scale, int32_t window,
                                     int32_t sinks, void *workspace, int64_t workspace_bytes, void *stream) {
    tiles_status_t st = check_cache(cache);
    if (st != TILES_OK) return st;
    const tiles_paged_desc &d = cache->desc;
    if (layer < 0 || layer >= d.n_layers || n_q_heads < 1 || n_q_heads % d.n_kv_heads || n_tokens < 0 ||
        max_tokens < 1 || window < 0 || sinks < 0 || !(scale > 0.f) || scale > 1e30f || !al4(cu_tokens) ||
        (!cu_tokens && n_tokens != d.n_seqs))
        return TILES_ERR_INVALID_ARG;
    if (n_q_heads / d.n_kv_heads > 16 || (long long)n_tokens * (n_q_heads / d.n_kv_heads) >= (1ll << 28))
        return TILES_ERR_UNSUPPORTED;
    if (n_tokens == 0) return TILES_OK;
    if (!q || !out || !al16(q) || !al16(out) || q_stride_token % 8 || q_stride_head % 8 || out_stride_token % 8 ||
        out_stride_head % 8 || q_stride_token < 0 || q_stride_head < 0 || out_stride_token < 0 || out_stride_head < 0 ||
        (out_stride_token < d.head_dim && n_tokens > 1) || (out_stride_head < d.head_dim && n_q_heads > 1) ||
        !workspace || !al16(workspace))
        return TILES_ERR_INVALID_ARG;
    // the kernels address q and out in 16-byte units of 32 bits
    for (const int64_t *st : {&q_stride_token, &out_stride_token})
        if ((double)n_tokens * (double)*st + (double)n_q_heads * (double)(st == &q_stride_token ? q_stride_head : out_stride_head) >=
            8.0 * 4294967296.0)
            return TILES_ERR_UNSUPPORTED;
    if (max_tokens > n_tokens) max_tokens = n_tokens;
    int sms = 0;
    if ((st = sm_count(&sms)) != TILES_OK) return st;
    if (workspace_bytes < attn_ws_bytes(d, n_q_heads, max_tokens, sms)) return TILES_ERR_CAPACITY;
    AttnParams p;
    p.c = view_of(*cache, layer);
    p.q = static_cast<const uint16_t *>(q);
    p.out = static_cast<uint16_t *>(out);
    p.q_t = q_stride_token;
    p.q_h = q_stride_head;
    p.o_t = out_stride_token;
    p.o_h = out_stride_head;
    p.cu = cu_tokens;
    p.n_tokens = n_tokens;
    p.max_tokens = max_tokens;
    p.G = n_q_heads / d.n_kv_heads;
    p.g_mul = (unsigned)(((1ull << 32) + (unsigned)p.G - 1) / (unsigned)p.G);
    p.scale_log2 = (float)((double)scale * 1.4426950408889634);
    // a window as long as the longest row hides nothing
    const int cap = d.table_width * d.page_size;
    p.window = window >= cap ? 0 : window;
    p.sinks = p.window > 0 ? std::min(sinks, cap) : 0;
    p.ws = static_cast<float *>(workspace);
    p.ctas = 0;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = streams(p.G, max_tokens) ? stream_launch(p, sms, cs) : tc_launch(p, sms, cs);
    return e == cudaSuccess ? TILES_OK : TILES_ERR_CUDA;
}

tiles_status_t tiles_paged_status(const tiles_paged_cache *cache, void *stream) {
    const tiles_status_t st = check_cache(cache);
    if (st != TILES_OK) return st;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    uint32_t word = 0;
    if (cudaMemcpyAsync(&word, cache->state, 4, cudaMemcpyDeviceToHost, cs) != cudaSuccess ||
        cudaStreamSynchronize(cs) != cudaSuccess)
        return TILES_ERR_CUDA;
    if (word && (cudaMemsetAsync(cache->state, 0, 4, cs) != cudaSuccess || cudaStreamSynchronize(cs) != cudaSuccess))
        return TILES_ERR_CUDA;
    if (word & kDevBounds) return TILES_ERR_DEVICE_BOUNDS;
    if (word & kDevNoPages) return TILES_ERR_CAPACITY;
    if (word & kDevTimeout) return TILES_ERR_TIMEOUT;
    return TILES_OK;
}

}  // extern "C"
