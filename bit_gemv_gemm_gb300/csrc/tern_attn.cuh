// tern_attn.cuh -- what the attention kernels share: their arguments, the
// split of the keys over CTAs, the tensor maps of the cache.  Internal.
#pragma once

#include <math.h>

#include "tern_cache.cuh"
#include "tern_mma.cuh"
#include "tern_sm100.cuh"

namespace tern {

constexpr int kMaxSms = 160;                      // the workspace is sized for this many
constexpr size_t kAttnCounterBytes = 4096;
constexpr uint64_t kAttnWaitNs = 1000000000ull;   // 1 s: far beyond any real wait

struct AttnArgs {
    const __nv_bfloat16* q;
    long long q_stride;
    CacheView c;
    SeqView s;
    int q_heads, group;
    float scale_log2;        // scale * log2(e): scores are kept in powers of two
    int window;
    __nv_bfloat16* out;
    float* lse;
    unsigned* counters;      // one per CTA, 0 between calls
    float* partial;          // two slots per CTA
};

// The keys [j0, j1) that the query rows [r0, r1) of a sequence see together;
// row r is (token r / group, head r % group).
__device__ __forceinline__ void keys_of_rows(const Seq& q, int group, int window, int r0, int r1, int& j0, int& j1) {
    const int first = q.len - q.n + r0 / group, last = q.len - q.n + (r1 - 1) / group;
    j1 = max(last + 1, 0);
    j0 = window > 0 ? max(first - window + 1, 0) : 0;
}

// Keys are handed out in units of kUnit, row tile by row tile: the units of
// all (sequence, key head, row tile) items, in that order, are cut into one
// equal contiguous share per CTA, whatever the sequences' lengths.  An item
// that no key reaches counts one unit (its rows are written as zeros).
template <int UNIT>
__device__ __forceinline__ int item_units(const Seq& q, int group, int window, int r0, int r1) {
    int j0, j1;
    keys_of_rows(q, group, window, r0, r1, j0, j1);
    return j1 > j0 ? (j1 - 1) / UNIT - j0 / UNIT + 1 : 1;
}
template <int UNIT>
__device__ __forceinline__ long long head_units(const Seq& q, int group, int window, int rows) {
    const int all = q.n * group;
    long long sum = 0;
    for (int r = 0; r < all; r += rows) sum += item_units<UNIT>(q, group, window, r, min(r + rows, all));
    return sum;
}
__host__ __device__ inline long long unit_begin(long long total, int P, int c) { return total * c / P; }
__device__ inline int unit_owner(long long total, int P, long long u) {
    int c = (int)((u * P) / total);
    while (c + 1 < P && unit_begin(total, P, c + 1) <= u) ++c;
    while (c > 0 && unit_begin(total, P, c) > u) --c;
    return c;
}

// A cache array as the TMA sees it: [page][head][d / 64][slot][64 values], a
// box of `rows` slots of one head, each 64 values a 128-byte swizzled row.
inline bool make_cache_map(CUtensorMap* m, const void* base, const CacheView& c, int box_rows, int box_chunks) {
    auto enc = get_encode();
    if (!enc) return false;
    const cuuint64_t dim[5] = {64, (cuuint64_t)c.page_size, (cuuint64_t)(c.head_dim / 64), (cuuint64_t)c.kv_heads,
                               (cuuint64_t)c.pages};
    const cuuint64_t stride[4] = {(cuuint64_t)c.slot_stride * 2, 128, (cuuint64_t)c.head_stride * 2,
                                  (cuuint64_t)c.page_stride * 2};
    const cuuint32_t box[5] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_chunks, 1, 1};
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dim, stride, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
__device__ __forceinline__ void tma_load_cache(uint32_t dst, const CUtensorMap* m, int slot, int chunk, int head,
                                               int page, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], "
        "[%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(0), "r"(slot), "r"(chunk), "r"(head), "r"(page), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void fence_proxy_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Launchers of the kernels (each checks nothing: the entry point has).
cudaError_t launch_attn_rows(const AttnArgs& a, const void* k, const void* v, int max_rows, int sms, cudaStream_t stream);
size_t attn_rows_workspace();

}  // namespace tern
