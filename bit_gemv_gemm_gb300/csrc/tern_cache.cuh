// tern_cache.cuh -- the paged key/value cache as the kernels see it: argument
// checks shared by the entry points, and the per-sequence view with its
// device-side bounds checks.  Internal.
//
// The cache is pages of page_size slots, one token a slot, kv_heads heads of
// head_dim bf16 values.  Key j of sequence b sits in slot j % page_size of page
// table[b][j / page_size].  The strides of the layout are free (multiples of 8
// elements), so both [page][head][slot][d] and [page][slot][head][d] work.
#pragma once

#include "tern_common.cuh"

namespace tern {

struct CacheView {
    int pages, page_size, kv_heads, head_dim;
    long long page_stride, head_stride, slot_stride;   // elements
};

// Sequences of new tokens over cached keys.
struct SeqView {
    const int* table;     // [B][width] page ids
    const int* lens;      // [B] cached keys, the new tokens' included
    const int* q_start;   // [B + 1] first new token of each sequence; null: T / B each
    int width, B, T, max_new;
};

// One sequence: its new tokens q0 .. q0 + n - 1, its keys 0 .. len - 1.  Values
// that do not fit the call's arrays are cut to what does and reported.
struct Seq {
    int q0, n, len;
};
__device__ __forceinline__ Seq load_seq(const SeqView& s, int page_size, int b, int* err) {
    Seq r;
    bool bad = false;
    if (s.q_start) {
        const int a = s.q_start[b], e = s.q_start[b + 1];
        r.q0 = min(max(a, 0), s.T);
        r.n = min(max(e, r.q0), s.T) - r.q0;
        bad = a != r.q0 || e != r.q0 + r.n || r.n > s.max_new;
        r.n = min(r.n, s.max_new);
    } else {
        r.n = s.T / s.B;
        r.q0 = b * r.n;
    }
    const int len = s.lens[b];
    const long long room = (long long)s.width * page_size;
    r.len = (int)min((long long)max(len, 0), room);
    if (bad || len != r.len) report_device_error(err, TERN_DEVERR_CACHE_SEQUENCE);
    return r;
}
// A page id from the table, checked against the pool.  A bad one is reported and
// read as page 0 (the call's output is then undefined)...
__device__ __forceinline__ int checked_page(int id, int pages, int* err) {
    if ((unsigned)id < (unsigned)pages) return id;
    report_device_error(err, TERN_DEVERR_CACHE_PAGE);
    return 0;
}
// ... but never written: page 0 is another sequence's.  -1 where the id is bad.
__device__ __forceinline__ int checked_page_to_write(int id, int pages, int* err) {
    if ((unsigned)id < (unsigned)pages) return id;
    report_device_error(err, TERN_DEVERR_CACHE_PAGE);
    return -1;
}

// launch_pdl with clusters of `cluster` CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_clusters(void (*kernel)(KArgs...), unsigned cluster, dim3 grid, dim3 block, size_t smem,
                                cudaStream_t stream, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

inline bool aligned_to(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline tern_status make_cache_view(const tern_cache_layout* l, CacheView* v) {
    if (!l) return TERN_ERR_NULL;
    if (l->pages < 1 || l->page_size < 16 || l->page_size % 16 != 0 || l->page_size > 65536 || l->kv_heads < 1 ||
        l->kv_heads > 65535 || l->head_dim < 8 || l->head_dim % 8 != 0 || l->head_dim > 1024)
        return TERN_ERR_SHAPE;
    const long long d = l->head_dim;
    // distinct (page, head, slot) must not overlap: each stride covers a head's values
    if (l->slot_stride < d || l->head_stride < d || l->page_stride < d || l->slot_stride % 8 || l->head_stride % 8 ||
        l->page_stride % 8 || l->slot_stride >= (1LL << 37) || l->head_stride >= (1LL << 37) ||
        l->page_stride >= (1LL << 37))
        return TERN_ERR_SHAPE;
    *v = CacheView{l->pages, l->page_size, l->kv_heads, l->head_dim, l->page_stride, l->head_stride, l->slot_stride};
    return TERN_OK;
}
// The most keys a table row may name: indices stay well inside 32 bits.
constexpr long long kMaxKeys = 1LL << 30;

inline tern_status make_seq_view(const int* table, int width, int page_size, const int* lens, const int* q_start, int B,
                                 int T, int max_new, SeqView* s) {
    if (B < 1 || B > 65535 || width < 1 || T < 0 || max_new < 0 || (long long)width * page_size > kMaxKeys)
        return TERN_ERR_SHAPE;
    if (!q_start && T % B != 0) return TERN_ERR_SHAPE;
    if (!table || !lens) return TERN_ERR_NULL;
    if (!aligned_to(table, 4) || !aligned_to(lens, 4) || !aligned_to(q_start, 4)) return TERN_ERR_ALIGN;
    // (no sequence brings more than all T: a max_new that allows more chooses no other kernel)
    *s = SeqView{table, lens, q_start, width, B, T, q_start ? (max_new < T ? max_new : T) : T / B};
    return TERN_OK;
}

}  // namespace tern
