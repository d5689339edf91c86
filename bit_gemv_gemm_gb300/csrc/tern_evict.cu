// tern_evict.cu -- eviction from the paged cache by accumulated attention
// weight.  Of each sequence and key head it keeps the `recent` last keys and,
// of those before them, the ones with the largest mass, `budget` in all; the
// kept keys move, in order, to pages of their own.
//
// Selection (one CTA a sequence and head) finds the smallest kept mass by
// radix selection over the masses as ordered 32-bit integers, a byte a pass
// from the highest, and then writes the kept indices with a running count, so
// equal masses go to the lowest index.  The move is a copy, 16 bytes a thread.
#include "tern_cache.cuh"

namespace tern {
namespace {

__device__ int g_evict_error;

constexpr int kSelThreads = 1024;

struct EvictArgs {
    const __nv_bfloat16 *k, *v;
    CacheView c;
    const float* mass;
    const int *table, *lens;
    int width, B, budget, recent;
    __nv_bfloat16 *dk, *dv;
    CacheView dc;
    float* dmass;
    const int* dtable;
    int dwidth;
    int* keep;
    int* dlens;
};

// Floats as integers of the same order; -0 counts as 0 and NaN as the lowest.
__device__ __forceinline__ uint32_t order_of(float m) {
    if (m != m) return 0u;
    const uint32_t u = __float_as_uint(m + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int evict_len(const EvictArgs& a, int b) {
    const int len = a.lens[b];
    const long long room = (long long)a.width * a.c.page_size;
    const int cut = (int)min((long long)max(len, 0), room);
    if (cut != len) report_device_error(&g_evict_error, TERN_DEVERR_CACHE_SEQUENCE);
    return cut;
}
__device__ __forceinline__ float mass_at(const EvictArgs& a, int b, int hk, int j) {
    const int page = checked_page(a.table[(long long)b * a.width + j / a.c.page_size], a.c.pages, &g_evict_error);
    return a.mass[((long long)page * a.c.kv_heads + hk) * a.c.page_size + j % a.c.page_size];
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const EvictArgs a) {
    __shared__ int hist[256];
    __shared__ int pick[2];
    __shared__ int warp_gt[32], warp_eq[32];
    pdl_launch_dependents();
    pdl_wait();
    const int b = blockIdx.y, hk = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int len = evict_len(a, b), kept = min(len, a.budget), recent = min(a.recent, kept);
    const int cand = len - recent, want = kept - recent;   // the first `cand` keys give `want`
    int* keep = a.keep + ((long long)b * a.c.kv_heads + hk) * a.budget;
    if (hk == 0 && tid == 0) a.dlens[b] = kept;
    for (int i = want + tid; i < a.budget; i += kSelThreads) keep[i] = i < kept ? cand + i - want : -1;
    uint32_t prefix = 0;
    int left = want;   // to be taken among the keys that share the prefix
    if (want > 0 && want < cand) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
            __syncthreads();
            for (int j = tid; j < cand; j += kSelThreads) {
                const uint32_t u = order_of(mass_at(a, b, hk, j));
                if (shift == 24 || (u >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(u >> shift) & 255], 1);
            }
            __syncthreads();
            if (tid == 0) {
                int above = 0, d = 255;
                while (d > 0 && above + hist[d] < left) above += hist[d--];
                pick[0] = d;
                pick[1] = above;
            }
            __syncthreads();
            prefix |= (uint32_t)pick[0] << shift;
            left -= pick[1];
            __syncthreads();
        }
    } else {
        left = cand;   // all of them, or none
    }
    if (want == 0) return;
    const bool all = want >= cand;
    int gt0 = 0, eq0 = 0;
    for (int base = 0; base < cand; base += kSelThreads) {
        const int j = base + tid;
        bool gt = false, eq = false;
        if (j < cand) {
            const uint32_t u = all ? 0u : order_of(mass_at(a, b, hk, j));
            gt = !all && u > prefix;
            eq = all || u == prefix;
        }
        const unsigned mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) {
            warp_gt[warp] = __popc(mg);
            warp_eq[warp] = __popc(me);
        }
        __syncthreads();
        int g = gt0, e = eq0;
        for (int w = 0; w < 32; ++w) {
            if (w < warp) {
                g += warp_gt[w];
                e += warp_eq[w];
            }
            gt0 += warp_gt[w];
            eq0 += warp_eq[w];
        }
        g += __popc(mg & ((1u << lane) - 1u));
        e += __popc(me & ((1u << lane) - 1u));
        if (gt || (eq && e < left)) keep[g + min(e, left)] = j;
        __syncthreads();
    }
}

// One warp a kept key of one head.
__global__ void __launch_bounds__(256) move_kernel(const EvictArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int b = blockIdx.z, hk = blockIdx.y, lane = threadIdx.x & 31, D = a.c.head_dim;
    for (int i = blockIdx.x * 8 + (threadIdx.x >> 5); i < a.budget; i += gridDim.x * 8) {
        const int j = a.keep[((long long)b * a.c.kv_heads + hk) * a.budget + i];
        if (j < 0) return;
        const int page = checked_page(a.table[(long long)b * a.width + j / a.c.page_size], a.c.pages, &g_evict_error);
        const int dpage = checked_page(a.dtable[(long long)b * a.dwidth + i / a.dc.page_size], a.dc.pages, &g_evict_error);
        const int slot = j % a.c.page_size, dslot = i % a.dc.page_size;
        const long long from = page * a.c.page_stride + hk * a.c.head_stride + slot * a.c.slot_stride;
        const long long to = dpage * a.dc.page_stride + hk * a.dc.head_stride + dslot * a.dc.slot_stride;
        for (int d = lane * 8; d < D; d += 256) {
            *reinterpret_cast<uint4*>(a.dk + to + d) = *reinterpret_cast<const uint4*>(a.k + from + d);
            *reinterpret_cast<uint4*>(a.dv + to + d) = *reinterpret_cast<const uint4*>(a.v + from + d);
        }
        if (lane == 0)
            a.dmass[((long long)dpage * a.dc.kv_heads + hk) * a.dc.page_size + dslot] =
                a.mass[((long long)page * a.c.kv_heads + hk) * a.c.page_size + slot];
    }
}

}  // namespace

cudaError_t read_evict_device_error(int* code) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_evict_error, sizeof(int));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_evict_error, &zero, sizeof(int));
}

}  // namespace tern

using namespace tern;

extern "C" size_t tern_cache_evict_workspace_bytes(int B, int kv_heads, int max_keys) {
    if (B < 1 || kv_heads < 1 || max_keys < 0) return 0;
    return 256;
}

extern "C" tern_status tern_cache_evict(const void* k_cache, const void* v_cache, const tern_cache_layout* layout,
                                        const float* mass, const int* table, int table_width, const int* lens, int B,
                                        int budget, int recent, void* dst_k, void* dst_v,
                                        const tern_cache_layout* dst_layout, float* dst_mass, const int* dst_table,
                                        int dst_table_width, int* keep, int* dst_lens, void* workspace,
                                        size_t workspace_bytes, tern_stream_t stream) {
    set_launch_count(0);
    EvictArgs a;
    tern_status st = make_cache_view(layout, &a.c);
    if (st == TERN_OK) st = make_cache_view(dst_layout, &a.dc);
    if (st != TERN_OK) return st;
    if (a.c.kv_heads != a.dc.kv_heads || a.c.head_dim != a.dc.head_dim || B < 1 || B > 65535 || table_width < 1 ||
        dst_table_width < 1 || budget < 1 || recent < 0 || recent > budget ||
        (long long)dst_table_width * a.dc.page_size < budget || (long long)table_width * a.c.page_size > 0x7fffffffLL)
        return TERN_ERR_SHAPE;
    if (!k_cache || !v_cache || !mass || !table || !lens || !dst_k || !dst_v || !dst_mass || !dst_table || !keep ||
        !dst_lens)
        return TERN_ERR_NULL;
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(dst_k) || !aligned16(dst_v) || !aligned_to(mass, 4) ||
        !aligned_to(table, 4) || !aligned_to(lens, 4) || !aligned_to(dst_mass, 4) || !aligned_to(dst_table, 4) ||
        !aligned_to(keep, 4) || !aligned_to(dst_lens, 4))
        return TERN_ERR_ALIGN;
    if (!workspace ||
        workspace_bytes < tern_cache_evict_workspace_bytes(B, a.c.kv_heads, table_width * a.c.page_size))
        return TERN_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return TERN_ERR_ALIGN;
    st = check_device(nullptr);
    if (st != TERN_OK) return st;
    a.k = static_cast<const __nv_bfloat16*>(k_cache);
    a.v = static_cast<const __nv_bfloat16*>(v_cache);
    a.mass = mass;
    a.table = table;
    a.lens = lens;
    a.width = table_width;
    a.B = B;
    a.budget = budget;
    a.recent = recent;
    a.dk = static_cast<__nv_bfloat16*>(dst_k);
    a.dv = static_cast<__nv_bfloat16*>(dst_v);
    a.dmass = dst_mass;
    a.dtable = dst_table;
    a.dwidth = dst_table_width;
    a.keep = keep;
    a.dlens = dst_lens;
    if (launch_pdl(select_kernel, dim3(a.c.kv_heads, B), dim3(kSelThreads), 0, (cudaStream_t)stream, true, a) !=
        cudaSuccess)
        return TERN_ERR_CUDA;
    const int grid = (budget + 31) / 32 < 1024 ? (budget + 31) / 32 : 1024;
    if (launch_pdl(move_kernel, dim3(grid, a.c.kv_heads, B), dim3(256), 0, (cudaStream_t)stream, true, a) !=
        cudaSuccess)
        return TERN_ERR_CUDA;
    set_launch_count(2);
    return TERN_OK;
}
