// The paged KV cache's internals shared by its page management (paged_cache.cu)
// and its attention (paged_attn.cu, paged_attn_tc.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "tiles_internal.h"

namespace tiles {
// A 3-D BF16 tensor map (runtime.cu): `blocks` dense blocks of `rows` rows of d
// elements, boxes of box_rows rows x 64 elements, 128-byte swizzle. False if
// the driver refuses it.
bool encode_bf16_3d(TensorMap *out, const void *base, uint64_t d, uint64_t rows, uint64_t blocks, uint32_t box_rows);

namespace paged {

// int32 words of the state buffer: the status word, then (at kStateRefs) the
// reference counts and working memory of n_pages words each (writers, lowest,
// copy sources, copy targets, free list), then n_seqs words (each row's first slot)
// and n_seqs table_width words (what slots need)
constexpr int kStateStatus = 0, kStateCopies = 1, kStateRefs = 16;
constexpr int kStateArrays = 6;

// device status bits beyond kDevTimeout and kDevBounds
constexpr uint32_t kDevNoPages = 4u;

// Launches a kernel that may be set up while the one before it on the stream still
// runs; each begins with after_previous(), so it reads nothing of that kernel's early.
// About a microsecond less between two kernels of a decoding step.
template <typename... P, typename... A>
cudaError_t launch_next(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A cache as the kernels see it (one layer's pools for append and attention).
struct View {
    uint8_t *k, *v;      // pools of layer 0, or of the call's layer
    float *ks, *vs;      // INT8: scales, likewise
    int32_t *tables, *lens, *state;
    const float *k_shift;  // of the call's layer, or null
    int n_layers, nkv, d, ps, psl, n_pages, n_seqs, width, i8;  // psl: log2 of the page size ps
};

struct AttnParams {
    View c;
    const uint16_t *q;
    uint16_t *out;
    long long q_t, q_h, o_t, o_h;  // strides in elements
    const int32_t *cu;             // null: one token a row
    int n_tokens, max_tokens, G;
    unsigned g_mul;                // ceil(2^32 / G): see group_div
    float scale_log2;              // scale * log2(e): the softmax runs on powers of two
    int window, sinks;
    float *ws;
    int ctas;                      // CTAs that share the work
};

// x / G for 0 <= x < 2^28: g_mul = (2^32 + e) / G with 0 <= e < G <= 16, so the
// product's error x e / 2^32 stays below 1 / G.
__device__ __forceinline__ int group_div(const AttnParams &p, int x) {
    return p.G == 1 ? x : (int)__umulhi((unsigned)x, p.g_mul);
}

// Row s's tokens in the call (first token, count) and its length; a row that
// breaks the rules (token offsets out of order or range, more than max_tokens)
// has no tokens, and a length beyond the table is cut to it: *bad says so.
struct RowSpan {
    int t0, n, len;
};
__device__ __forceinline__ RowSpan row_span(const AttnParams &p, int s, bool *bad) {
    RowSpan r;
    int len = __ldg(p.c.lens + s);
    if (p.cu) {
        const int a = __ldg(p.cu + s), b = __ldg(p.cu + s + 1);
        r.t0 = a;
        r.n = b - a;
        if (a < 0 || b < a || b > p.n_tokens || r.n > p.max_tokens) {
            *bad = true;
            r.t0 = r.n = 0;
        }
    } else {
        r.t0 = s;
        r.n = 1;
    }
    const int cap = p.c.width * p.c.ps;
    if (len < 0 || len > cap) {
        *bad = true;
        len = len < 0 ? 0 : cap;
    }
    r.len = len;
    return r;
}

// Positions some token of row (len, n) sees: [0, head) and [lo, len), head <= lo.
__device__ __forceinline__ void visible_span(const AttnParams &p, int len, int first_pos, int *head, int *lo) {
    *lo = 0;
    *head = 0;
    if (p.window > 0) {
        const int l = first_pos - p.window + 1;
        if (l > 0) {
            *lo = l < len ? l : len;
            *head = p.sinks < *lo ? p.sinks : *lo;
        }
    }
}

// The host-side checks of a cache (paged_cache.cu).
tiles_status_t cache_check(const tiles_paged_cache *cache);
// pos[t] = the position of token t (offsets as for tiles_paged_append), -1 for
// padding; a position at or beyond max_pos counts as none and is recorded in
// *status (a plan's word) as kDevBounds.
cudaError_t positions_launch(const tiles_paged_cache &cache, const int32_t *cu, int n_tokens, int max_pos, int32_t *pos,
                             uint32_t *status, cudaStream_t st);

// Streaming attention (paged_attn.cu): up to 16 query rows a (row, KV head).
size_t stream_ws_bytes(int sms, int d);
cudaError_t stream_launch(const AttnParams &p, int sms, cudaStream_t st);

// Attention on the tensor cores (paged_attn_tc.cu): any number of query rows.
size_t tc_ws_bytes(int sms, int d);
cudaError_t tc_launch(const AttnParams &p, int sms, cudaStream_t st);

}  // namespace paged
}  // namespace tiles
