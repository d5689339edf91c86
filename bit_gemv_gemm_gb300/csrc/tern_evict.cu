// tern_evict.cu -- eviction from the paged cache by accumulated attention
// weight.  Of each sequence and key head it keeps the `recent` last keys and,
// of those before them, the ones with the largest mass, `budget` in all; the
// kept keys move, in order, to pages of their own.
//
// One cluster of up to eight CTAs a sequence and head; a CTA takes an equal
// part of the keys and keeps their masses in shared memory, as integers of the
// same order, so the cache's masses are read once.
//   * The smallest kept mass is found by radix selection from the top, a byte a
//     pass: each CTA counts its keys by digit, every CTA adds the cluster's histograms
//     through distributed shared memory, a thread a digit, and finds the one that
//     the selection ends in.  (11 bits a pass, three passes, moved eight times
//     the words between the SMs, at 10 us a pass.)
//   * From the CTAs' and warps' counts every warp knows where its kept keys begin
//     in the result (equal masses go to the lowest index) and lists them there.
//   * The list is then copied, each CTA an equal part of it: K, V and mass, 16
//     bytes a thread, the rows of two keys in flight a thread and the places of
//     the next two looked up meanwhile.
// Bound by the copy: each kept key's rows are read and written once.  A CTA is a
// chain of waits (lengths, masses, selection, table, rows), so four
// share an SM, and the clusters are as large as lets all CTAs run at once:
// sixteen sequences of 20000 keys cut to 4096, eight heads, take 365 us with one
// CTA an SM, 142 with four in clusters of four (512 CTAs, one wave; 3.9 TB/s of the rows).
#include <cooperative_groups.h>

#include "tern_cache.cuh"

namespace tern {
namespace {

namespace cg = cooperative_groups;

__device__ int g_evict_error;

constexpr int kMaxCluster = 8, kThreads = 256, kWarps = kThreads / 32, kCtas = 4;   // an SM
constexpr int kBits = 8, kBins = 1 << kBits;
constexpr int kMaxHeld = 40 * 1024;          // masses a CTA holds; longer shares are read again each pass
constexpr int kSmallHeld = 10 * 1024;        // so many leave room for kCtas CTAs

struct EvictArgs {
    const __nv_bfloat16 *k, *v;
    CacheView c;
    const float* mass;
    const int *table, *lens;
    int width, B, budget, recent, held;      // held: masses that shared memory has room for
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

struct Way {   // where a key's rows and mass lie, and where they go (to < 0: nowhere, a bad page id)
    long long from, to, mass, dmass;
};

struct Shared {
    int hist[2][kBins];          // by pass parity: a CTA may be counting while another still reads
    int counts[2];               // of this CTA's keys: above the smallest kept mass, equal to it
    int warp_a[kWarps], warp_b[kWarps];   // the same by warp
    int digit, above;
};

__global__ void __launch_bounds__(kThreads, kCtas)
evict_kernel(const EvictArgs a) {
    extern __shared__ uint32_t held[];       // ordered masses of this CTA's keys
    __shared__ Shared sm;
    cg::cluster_group cluster = cg::this_cluster();
    pdl_launch_dependents();
    pdl_wait();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int item = blockIdx.x / ctas, b = item / a.c.kv_heads, hk = item % a.c.kv_heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int len = a.lens[b];
    {
        const long long room = (long long)a.width * a.c.page_size;
        const int cut = (int)min((long long)max(len, 0), room);
        if (cut != len && tid == 0) report_device_error(&g_evict_error, TERN_DEVERR_CACHE_SEQUENCE);
        len = cut;
    }
    const int kept = min(len, a.budget), recent = min(a.recent, kept);
    const int cand = len - recent, want = kept - recent;   // the first `cand` keys give `want`
    const int per = (len + ctas - 1) / ctas;
    const int j_lo = min(rank * per, len), j_hi = min(j_lo + per, len), n = max(min(j_hi, cand) - j_lo, 0);
    const int* trow = a.table + (long long)b * a.width;
    auto page_of = [&](int j) {
        return checked_page(trow[(unsigned)j / (unsigned)a.c.page_size], a.c.pages, &g_evict_error);
    };
    auto mass_index = [&](int page, int j) {
        return ((long long)page * a.c.kv_heads + hk) * a.c.page_size + (unsigned)j % (unsigned)a.c.page_size;
    };
    auto ordered = [&](int x) {   // candidate x of this CTA
        return x < a.held ? held[x] : order_of(a.mass[mass_index(page_of(j_lo + x), j_lo + x)]);
    };
    int* keep = a.keep + ((long long)b * a.c.kv_heads + hk) * a.budget;
    if (rank == 0) {
        if (hk == 0 && tid == 0) a.dlens[b] = kept;
        for (int i = kept + tid; i < a.budget; i += kThreads) keep[i] = -1;
    }

    uint32_t prefix = 0;
    int left = want;   // to be taken among the keys that share the prefix
    const bool choose = want > 0 && want < cand;
    if (choose) {
#pragma unroll 4
        for (int x = tid; x < min(n, a.held); x += kThreads)
            held[x] = order_of(a.mass[mass_index(page_of(j_lo + x), j_lo + x)]);
#pragma unroll 1
        for (int shift = 32 - kBits, pass = 0; shift >= 0; shift -= kBits, ++pass) {
            const uint32_t known = pass == 0 ? 0u : 0xffffffffu << (shift + kBits);
            int* hist = sm.hist[pass & 1];
            for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
            __syncthreads();
#pragma unroll 4
            for (int x = tid; x < n; x += kThreads) {
                const uint32_t u = ordered(x);
                if ((u & known) == (prefix & known)) atomicAdd(&hist[(u >> shift) & (uint32_t)(kBins - 1)], 1);
            }
            cluster.sync();
            // digits from the top, one a thread; the running sum says which of them the selection ends in
            int own = 0;
            if (tid < kBins)
#pragma unroll kMaxCluster
                for (int r = 0; r < ctas; ++r) own += cluster.map_shared_rank(hist, r)[kBins - 1 - tid];
            int x = own;
#pragma unroll
            for (int k = 1; k < 32; k <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, k);
                if (lane >= k) x += y;
            }
            if (lane == 31) sm.warp_a[warp] = x;
            __syncthreads();
            int before = x - own;
            for (int w = 0; w < warp; ++w) before += sm.warp_a[w];
            if (tid < kBins && before < left && before + own >= left) {
                sm.digit = kBins - 1 - tid;
                sm.above = before;
            }
            __syncthreads();
            prefix |= (uint32_t)sm.digit << shift;
            left -= sm.above;
        }
    } else {
        left = want > 0 ? cand : 0;   // all of them, or none
    }

    // how many of this warp's candidates (a run of its own) are above the smallest kept mass, and equal to it
    const int run = ((n + kWarps - 1) / kWarps + 31) / 32 * 32, x_lo = min(warp * run, n), x_hi = min(x_lo + run, n);
    int gt = 0, eq = 0;
    if (choose) {
#pragma unroll 4
        for (int x = x_lo + lane; x < x_hi; x += 32) {
            const uint32_t u = ordered(x);
            gt += u > prefix;
            eq += u == prefix;
        }
#pragma unroll
        for (int k = 16; k; k >>= 1) {
            gt += __shfl_xor_sync(0xffffffffu, gt, k);
            eq += __shfl_xor_sync(0xffffffffu, eq, k);
        }
    } else {
        eq = x_hi - x_lo;
    }
    __syncthreads();   // warp_a has been read
    if (lane == 0) {
        sm.warp_a[warp] = gt;
        sm.warp_b[warp] = eq;
    }
    __syncthreads();
    int gt_before = 0, eq_before = 0;
    {
        int g = 0, e = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) {
                gt_before = g;
                eq_before = e;
            }
            g += sm.warp_a[w];
            e += sm.warp_b[w];
        }
        if (tid == 0) {
            sm.counts[0] = g;
            sm.counts[1] = e;
        }
    }
    cluster.sync();
    for (int r = 0; r < rank; ++r) {
        const int* c = cluster.map_shared_rank(sm.counts, r);
        gt_before += c[0];
        eq_before += c[1];
    }
    // the list: this warp's kept candidates, then the recent keys of this CTA's part
    if (want > 0)
        for (int x0 = x_lo; x0 < x_hi; x0 += 32) {
            const int x = x0 + lane;
            const uint32_t u = choose && x < x_hi ? ordered(x) : 0u;
            const bool is_gt = choose && x < x_hi && u > prefix, is_eq = x < x_hi && (!choose || u == prefix);
            const unsigned mg = __ballot_sync(0xffffffffu, is_gt), me = __ballot_sync(0xffffffffu, is_eq);
            const unsigned under = (1u << lane) - 1u;
            const int g = gt_before + __popc(mg & under), e = eq_before + __popc(me & under);
            if (is_gt || (is_eq && e < left)) keep[g + min(e, left)] = j_lo + x;
            gt_before += __popc(mg);
            eq_before += __popc(me);
        }
    for (int j = max(j_lo, cand) + tid; j < j_hi; j += kThreads) keep[want + j - cand] = j;
    __threadfence();
    cluster.sync();   // the whole list is written (and this CTA's counts have been read)

    auto way = [&](int j, int i) {
        const int page = page_of(j), dpage = checked_page_to_write(a.dtable[(long long)b * a.dwidth + (unsigned)i / (unsigned)a.dc.page_size],
                                                           a.dc.pages, &g_evict_error);
        const int slot = (unsigned)j % (unsigned)a.c.page_size, dslot = (unsigned)i % (unsigned)a.dc.page_size;
        const long long from = page * a.c.page_stride + hk * a.c.head_stride + slot * a.c.slot_stride;
        const long long to = dpage < 0 ? -1 : dpage * a.dc.page_stride + hk * a.dc.head_stride + dslot * a.dc.slot_stride;
        return Way{from, to, mass_index(page, j), ((long long)dpage * a.dc.kv_heads + hk) * a.dc.page_size + dslot};
    };
    // keys i_lo .. i_hi - 1 of the list; threads in groups of `lanes` (D / 8, at most 32) a row
    const int part = (kept + ctas - 1) / ctas, i_lo = min(rank * part, kept), i_hi = min(i_lo + part, kept);
    const int D = a.c.head_dim, lanes = D >= 256 ? 32 : D > 64 ? 16 : 8, groups = kThreads / lanes;
    const int l0 = tid % lanes * 8;
    int i = i_lo + tid / lanes;
    if (i >= i_hi) return;
    auto place = [&](int x) { return way(__ldcg(keep + min(x, i_hi - 1)), min(x, i_hi - 1)); };
    Way p = place(i), q = place(i + groups);
    for (; i < i_hi; i += 2 * groups) {
        const Way p0 = p, q0 = q;
        const bool one = p0.to >= 0, two = q0.to >= 0 && i + groups < i_hi, more = i + 2 * groups < i_hi;
        for (int d = l0; d < D; d += lanes * 8) {
            const uint4 k0 = __ldcs(reinterpret_cast<const uint4*>(a.k + p0.from + d));
            const uint4 v0 = __ldcs(reinterpret_cast<const uint4*>(a.v + p0.from + d));
            const uint4 k1 = __ldcs(reinterpret_cast<const uint4*>(a.k + q0.from + d));
            const uint4 v1 = __ldcs(reinterpret_cast<const uint4*>(a.v + q0.from + d));
            if (d == l0 && more) {
                p = place(i + 2 * groups);
                q = place(i + 3 * groups);
            }
            if (one) {
                *reinterpret_cast<uint4*>(a.dk + p0.to + d) = k0;
                *reinterpret_cast<uint4*>(a.dv + p0.to + d) = v0;
            }
            if (two) {
                *reinterpret_cast<uint4*>(a.dk + q0.to + d) = k1;
                *reinterpret_cast<uint4*>(a.dv + q0.to + d) = v1;
            }
        }
        if (l0 >= D && more) {   // a lane past the row's end
            p = place(i + 2 * groups);
            q = place(i + 3 * groups);
        }
        if (l0 == 0) {
            if (one) a.dmass[p0.dmass] = a.mass[p0.mass];
            if (two) a.dmass[q0.dmass] = a.mass[q0.mass];
        }
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

extern "C" tern_status tern_cache_evict(const void* k_cache, const void* v_cache, const tern_cache_layout* layout,
                                        const float* mass, const int* table, int table_width, const int* lens, int B,
                                        int budget, int recent, void* dst_k, void* dst_v,
                                        const tern_cache_layout* dst_layout, float* dst_mass, const int* dst_table,
                                        int dst_table_width, int* keep, int* dst_lens, tern_stream_t stream) {
    set_launch_count(0);
    EvictArgs a;
    tern_status st = make_cache_view(layout, &a.c);
    if (st == TERN_OK) st = make_cache_view(dst_layout, &a.dc);
    if (st != TERN_OK) return st;
    if (a.c.kv_heads != a.dc.kv_heads || a.c.head_dim != a.dc.head_dim || B < 1 || B > 65535 || table_width < 1 ||
        dst_table_width < 1 || budget < 1 || recent < 0 || recent > budget ||
        (long long)dst_table_width * a.dc.page_size < budget || (long long)table_width * a.c.page_size > kMaxKeys ||
        (long long)B * a.c.kv_heads > 0x7fffffffLL / kMaxCluster)
        return TERN_ERR_SHAPE;
    if (!k_cache || !v_cache || !mass || !table || !lens || !dst_k || !dst_v || !dst_mass || !dst_table || !keep ||
        !dst_lens)
        return TERN_ERR_NULL;
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(dst_k) || !aligned16(dst_v) || !aligned_to(mass, 4) ||
        !aligned_to(table, 4) || !aligned_to(lens, 4) || !aligned_to(dst_mass, 4) || !aligned_to(dst_table, 4) ||
        !aligned_to(keep, 4) || !aligned_to(dst_lens, 4))
        return TERN_ERR_ALIGN;
    // one head's cluster writes a sequence's new length while another's may still read the old
    const uintptr_t old_at = reinterpret_cast<uintptr_t>(lens), new_at = reinterpret_cast<uintptr_t>(dst_lens);
    if (old_at < new_at + 4 * (uintptr_t)B && new_at < old_at + 4 * (uintptr_t)B) return TERN_ERR_SHAPE;
    int sms = 0;
    st = check_device(&sms);
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
    const long long room = (long long)table_width * a.c.page_size, items = (long long)B * a.c.kv_heads;
    int ctas = kMaxCluster;
    while (ctas > 1 && items * ctas > (long long)kCtas * sms && room / (ctas / 2) <= kSmallHeld) ctas /= 2;
    const long long share = (room + ctas - 1) / ctas;
    a.held = (int)(share < kMaxHeld ? share : kMaxHeld);
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return TERN_ERR_CUDA;
    if (!attr_set[dev]) {
        if (cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxHeld * 4) != cudaSuccess)
            return TERN_ERR_CUDA;
        attr_set[dev] = true;
    }
    if (launch_pdl_clusters(evict_kernel, (unsigned)ctas, dim3((unsigned)(items * ctas)), dim3(kThreads),
                            (size_t)a.held * 4, (cudaStream_t)stream, a) != cudaSuccess)
        return TERN_ERR_CUDA;
    set_launch_count(1);
    return TERN_OK;
}
