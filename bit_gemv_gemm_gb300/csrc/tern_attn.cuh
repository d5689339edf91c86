// tern_attn.cuh -- what the attention kernels share: their arguments, the
// split of the keys over CTAs, the tensor maps of the cache.  Internal.
#pragma once

#include <math.h>

#include <algorithm>
#include <cmath>

#include "tern_cache.cuh"
#include "tern_mma.cuh"
#include "tern_sm100.cuh"

namespace tern {

constexpr int kMaxSms = 160;                      // the workspace is sized for this many
constexpr size_t kAttnCounterBytes = TERN_ATTENTION_COUNTER_BYTES;   // 8 counters a CTA
static_assert(kAttnCounterBytes >= 8 * kMaxSms * sizeof(unsigned), "counters");
constexpr uint64_t kAttnWaitNs = 1000000000ull;   // 1 s: far beyond any real wait

struct AttnArgs {
    const __nv_bfloat16* q;
    long long q_stride;
    CacheView c;
    SeqView s;
    int q_heads, group;
    int tiles;               // row tiles of the longest sequence
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

// Keys are handed out in units of UNIT: the units of all items, in the order
// (sequence, row tile, key head), are cut into one equal contiguous share per
// CTA, whatever the sequences' lengths.  An item counts `cost` units more than
// its keys have, for what it costs to begin and end one.
struct Item {
    int b, rt, hk;
    Seq q;
    int rows, j0, j1, units;   // its rows, the keys they see together, and its units
    long long at;              // its first unit
};
// The extent of an item by its (b, rt, q): a row tile of R rows over the keys
// it sees.  units = 0: the sequence has no such item.
template <int UNIT, int COST>
struct RowTileExtent {
    static constexpr int kUnit = UNIT, kCost = COST;
    int R, group, window;
    __device__ __forceinline__ void operator()(Item& t) const {
        const int r0 = t.rt * R, all = t.q.n * group;
        t.rows = min(R, all - r0);
        if (t.rows <= 0) {
            t.rows = t.units = 0;
            return;
        }
        keys_of_rows(t.q, group, window, r0, r0 + t.rows, t.j0, t.j1);
        t.units = COST + (t.j1 > t.j0 ? (t.j1 - 1) / UNIT - t.j0 / UNIT + 1 : 0);
    }
};
__host__ __device__ inline long long unit_begin(long long total, int P, int c) {
    const long long x = total * c;
    return x <= 0x7fffffff ? (long long)((unsigned)x / (unsigned)P) : x / P;
}
__device__ inline int unit_owner(long long total, int P, long long u) {
    const long long x = u * P;
    int c = x <= 0x7fffffff ? (int)((unsigned)x / (unsigned)total) : (int)(x / total);
    while (c + 1 < P && unit_begin(total, P, c + 1) <= u) ++c;
    while (c > 0 && unit_begin(total, P, c) > u) --c;
    return c;
}

// What units [w, we) of an item are in key units: `n` from `first` on.  A
// segment of an item that has keys, but none of them, is `skip`ped; an item
// without keys (zeros are written) goes to the share that holds its first unit.
struct Segment {
    long long we;
    int first, n;
    bool whole, skip;
};
template <typename Extent>
__device__ __forceinline__ Segment segment_of(const Extent&, const Item& t, long long w, long long w1) {
    Segment s;
    s.we = min(w1, t.at + t.units);
    const int lo = max((int)(w - t.at) - Extent::kCost, 0), hi = max((int)(s.we - t.at) - Extent::kCost, 0);
    const int all = t.units - Extent::kCost;
    s.n = hi - lo;
    s.first = (t.j1 > t.j0 ? t.j0 / Extent::kUnit : 0) + lo;
    s.whole = s.n == all;
    s.skip = all > 0 ? s.n == 0 : w != t.at;
    return s;
}

// The next item, past row tiles that a sequence does not have; `tiles` row
// tiles are counted for every sequence.
template <typename Extent>
__device__ __forceinline__ void next_item(const SeqView& sv, const CacheView& cv, const Extent& extent, int tiles,
                                          Item& t, int* err) {
    t.at += t.units;
    if (++t.hk < cv.kv_heads) return;
    t.hk = 0;
    do {
        if (++t.rt >= tiles) {
            t.rt = 0;
            if (++t.b >= sv.B) return;
            t.q = load_seq(sv, cv.page_size, t.b, err);
        }
        extent(t);
    } while (t.units == 0);
}

// Share `share` of at most `shares`, [w0, w1) of all units, and the item that
// holds w0; P shares of at least min_units each.  Called by all THREADS threads
// of a CTA; false: no share.
// `sm`: 8 + THREADS / 32 words of shared memory.
//
// A call begins with this, so its latency counts (one token over 500 keys: a
// third of the kernel): the thread that finds the item hands it on through
// shared memory instead of every thread reading the lengths again, and the
// divisions are 32-bit ones where the numbers allow (a 64-bit one is a loop).
template <int THREADS, typename Extent>
__device__ bool find_share(const SeqView& sv, const CacheView& cv, const Extent& extent, int tiles, int min_units,
                           int share, int shares, long long* sm, int* err, long long& total, int& P, long long& w0, long long& w1, Item& t) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, Hk = cv.kv_heads;
    const long long all = (long long)sv.B * tiles;
    const long long per = all <= THREADS ? 1 : (all + THREADS - 1) / THREADS;
    const long long f0 = min((long long)threadIdx.x * per, all), f1 = min(f0 + per, all);
    auto units_of = [&](long long f) {
        t.b = f <= 0x7fffffff ? (int)((unsigned)f / (unsigned)tiles) : (int)(f / tiles);
        t.rt = (int)(f - (long long)t.b * tiles);
        t.q = load_seq(sv, cv.page_size, t.b, err);
        extent(t);
        return (long long)t.units * Hk;
    };
    long long mine = 0;
    for (long long f = f0; f < f1; ++f) mine += units_of(f);
    long long x = mine;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, k);
        if (lane >= k) x += y;
    }
    if (lane == 31) sm[8 + warp] = x;
    __syncthreads();
    long long before = x - mine;
    total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        const long long v = sm[8 + w];
        if (w < warp) before += v;
        total += v;
    }
    const long long most = total <= 0x7fffffff ? ((unsigned)total + min_units - 1) / (unsigned)min_units
                                               : (total + min_units - 1) / min_units;
    P = (int)min((long long)shares, most);
    if (share >= P) return false;
    w0 = unit_begin(total, P, share);
    w1 = unit_begin(total, P, share + 1);
    if (w0 >= before && w0 < before + mine) {
        long long at = before;
        for (long long f = f0; f < f1; ++f) {
            const long long u = per == 1 ? mine : units_of(f);
            if (w0 < at + u) break;
            at += u;
        }
        const long long in = w0 - at;   // below kv_heads * units, which may pass 32 bits
        t.hk = in <= 0xffffffffLL ? (int)((unsigned)in / (unsigned)t.units) : (int)(in / t.units);
        t.at = at + (long long)t.hk * t.units;
        int* o = reinterpret_cast<int*>(sm);
        o[0] = t.b;
        o[1] = t.rt;
        o[2] = t.hk;
        o[3] = t.q.q0;
        o[4] = t.q.n;
        o[5] = t.q.len;
        sm[3] = t.at;
    }
    __syncthreads();
    const int* o = reinterpret_cast<const int*>(sm);
    t.b = o[0];
    t.rt = o[1];
    t.hk = o[2];
    t.q = Seq{o[3], o[4], o[5]};
    t.at = sm[3];
    extent(t);
    return true;
}

// The most shares that a call's work fills (host: the lengths are on the device;
// no item has more units than this).  Where there are few items, each is cut into
// at most sqrt(units) parts: a part costs the join about what a unit costs, so
// units / parts + parts is least there (16 rows over one key head of 32k keys, 1000
// strips: 16, 32, 48, 304 parts 35, 28, 29, 73 us; of 130k keys 103, 62, 51 us).
inline long long most_shares(const AttnArgs& a, int unit, int cost, int min_units, long long shares) {
    const long long room = (long long)a.s.width * a.c.page_size;
    const long long keys = a.window > 0 && a.window + (long long)a.s.max_new < room ? a.window + (long long)a.s.max_new : room;
    const long long items = (long long)a.s.B * a.c.kv_heads * a.tiles, units = (keys + unit - 1) / unit + 1 + cost;
    const double most = std::min((double)items * std::sqrt((double)units), (double)items * units / min_units + 1.0);
    return most < (double)shares ? std::max((long long)most, 1LL) : shares;
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

// One warp: zeroes the rows [r0, r1) of a chunk of 128-byte rows.  Rows of V that
// hold no key of the sequence, or one before every window, count as 0: those of
// boxes that are not read before the boxes are, those inside a box after it has come.
// (Tested row by row this took 10 us of a tile; rows are taken by their range.)
__device__ __forceinline__ void zero_rows(unsigned char* chunk, int r0, int r1) {
    for (int i = r0 * 8 + (int)(threadIdx.x & 31); i < r1 * 8; i += 32)
        *reinterpret_cast<uint4*>(chunk + i * 16) = make_uint4(0, 0, 0, 0);
}
struct VRows {
    // [0, front) and [back_box, tile) are not read, [front, front_key) and [back, back_box) hold nothing seen
    int front, front_key, back, back_box;
    __device__ __forceinline__ VRows(int k0, int tile, int box_rows, int j0, int len) {
        front = max((j0 & ~(box_rows - 1)) - k0, 0);   // (box_rows is a power of two)
        front_key = max(j0 - k0, 0);
        back = min(len - k0, tile);
        back_box = min((back + box_rows - 1) & ~(box_rows - 1), tile);
    }
    // some row of a box that is read counts as 0
    __device__ __forceinline__ bool inside() const { return front < front_key || back < back_box; }
    __device__ __forceinline__ void zero_inside(unsigned char* chunk) const {
        zero_rows(chunk, front, front_key);
        zero_rows(chunk, back, back_box);
    }
};

// What a row's sum l of 2^(s - m) gives.  0: it saw no key (or none of more weight
// than 0), its output is 0 and its lse -inf; a sum that is not a number, of scores
// that are not, makes both NaN.
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
__device__ __forceinline__ float lse_of(float m2, float l) {
    return l == 0.0f ? -INFINITY : (m2 + log2f(l)) * 0.693147180559945309f;
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

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// two fp32 values in a register pair
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
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

// The heads of one token group as the TMA sees them: q as
// [d / 64][token][head][64 values], a box of one chunk of `tokens` tokens.
inline bool make_q_map(CUtensorMap* m, const __nv_bfloat16* q, long long q_stride, int q_heads, int T, int D, int group,
                       int tokens) {
    auto enc = get_encode();
    if (!enc) return false;
    const cuuint64_t dim[4] = {64, (cuuint64_t)q_heads, (cuuint64_t)T, (cuuint64_t)(D / 64)};
    const cuuint64_t stride[3] = {(cuuint64_t)D * 2, (cuuint64_t)q_stride * 2, 128};
    const cuuint32_t box[4] = {64, (cuuint32_t)group, (cuuint32_t)tokens, 1};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<__nv_bfloat16*>(q), dim, stride, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
__device__ __forceinline__ void tma_load_q(uint32_t dst, const CUtensorMap* m, int head, int token, int chunk,
                                           uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(0), "r"(head), "r"(token), "r"(chunk), "r"(bar)
        : "memory");
}

// Launchers of the kernels (each checks nothing: the entry point has).
// A row tile's results: parts are exchanged four columns at a time, [column /
// 4][row][4], then (m, l) by row.
constexpr int kTileRows = 128;
constexpr size_t part_floats(int D) { return (size_t)kTileRows * (D + 2); }

// The output of one row (a thread; `load(c, o)` gives 32 columns of its
// accumulator): to memory, divided by the sum, or into `part`.
template <int D, typename Load>
__device__ __forceinline__ void emit_row(const AttnArgs& a, bool whole, float* part, int row, bool live, long long orow,
                                         float m2, float l, Load load) {
    const float inv = inverse_sum(l);
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        __syncwarp();
        load(c, o);   // (a whole warp's)
        if (live && whole) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + orow * D + c);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    y[i] = pack_bf16(__uint_as_float(o[8 * e + 2 * i]) * inv, __uint_as_float(o[8 * e + 2 * i + 1]) * inv);
                dst[e] = make_uint4(y[0], y[1], y[2], y[3]);
            }
        } else if (live) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                __stcg(reinterpret_cast<uint4*>(part + ((size_t)(c / 4 + e) * kTileRows + row) * 4),
                       make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
        }
    }
    if (whole && live && a.lse) a.lse[orow] = lse_of(m2, l);
    if (!whole) __stcg(reinterpret_cast<float2*>(part + (size_t)D * kTileRows + 2 * row), make_float2(m2, l));
}

// A warp has stored its 32 rows' part and counts it into the item's counter:
// true if it was the last, which then adds the parts of all shares.  `counter`
// is that of the rows in share 0.
template <int COST>
__device__ __forceinline__ bool count_part(const Item& t, unsigned* counter, long long total, int P) {
    __threadfence();
    __syncwarp();
    const int c_lo = unit_owner(total, P, t.at + COST), c_hi = unit_owner(total, P, t.at + t.units - 1);
    unsigned last = 0;
    if ((threadIdx.x & 31) == 0)
        last = atomicInc(counter + 8 * c_lo, (unsigned)(c_hi - c_lo)) == (unsigned)(c_hi - c_lo);
    return __shfl_sync(0xffffffffu, last, 0) != 0;
}

// Adds the parts of all shares in their order, columns [c0, c1) of one row a
// thread; `first` is the row tile's part in share 0, a share has two, `stride`
// floats apart.
constexpr int join_columns(int D) { return D == 256 ? 64 : 32; }   // at a time
template <int D, int COST>
__device__ __forceinline__ void add_parts(const AttnArgs& a, const Item& t, const float* first, size_t stride, int row,
                                          bool live, long long orow, long long total, int P, int c0, int c1) {
    const int c_lo = unit_owner(total, P, t.at + COST), c_hi = unit_owner(total, P, t.at + t.units - 1);
    __threadfence();
    // (an item's first share may have begun before it: its part is then in its second slot)
    const int late = unit_begin(total, P, c_lo) >= t.at ? 0 : 1;
    auto part_of = [&](int x) { return first + (size_t)(2 * x + (x == c_lo ? late : 0)) * stride; };
    auto stat_of = [&](int x) {
        return __ldcg(reinterpret_cast<const float2*>(part_of(x) + (size_t)D * kTileRows + 2 * row));
    };
    // all loads in flight together; past the last part, its own again with no weight
    float mm = -INFINITY, ll = 0.0f;
    for (int x0 = c_lo; x0 <= c_hi; x0 += 4) {
        float2 st[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) st[i] = stat_of(min(x0 + i, c_hi));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float mn = fmaxf(mm, st[i].x), base = mn == -INFINITY ? 0.0f : mn;
            ll = ll * exp2_fast(mm - base) + (x0 + i <= c_hi ? st[i].y * exp2_fast(st[i].x - base) : 0.0f);
            mm = mn;
        }
    }
    const float base = mm == -INFINITY ? 0.0f : mm, inv = inverse_sum(ll);
    constexpr int W = D == 256 ? 2 : 3, COLS = join_columns(D);   // parts and columns in flight
#pragma unroll 1
    for (int c = c0; c < c1; c += COLS) {
        float4 y[COLS / 4];
#pragma unroll
        for (int e = 0; e < COLS / 4; ++e) y[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
        for (int x0 = c_lo; x0 <= c_hi; x0 += W) {
            float4 v[W][COLS / 4];
            float f[W];
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const int x = min(x0 + i, c_hi);
                const float* p = part_of(x) + ((size_t)(c / 4) * kTileRows + row) * 4;
                f[i] = stat_of(x).x;
#pragma unroll
                for (int e = 0; e < COLS / 4; ++e)
                    v[i][e] = __ldcg(reinterpret_cast<const float4*>(p + (size_t)e * kTileRows * 4));
            }
#pragma unroll
            for (int i = 0; i < W; ++i) {
                f[i] = x0 + i <= c_hi ? exp2_fast(f[i] - base) : 0.0f;
#pragma unroll
                for (int e = 0; e < COLS / 4; ++e) {
                    y[e].x = fmaf(v[i][e].x, f[i], y[e].x);
                    y[e].y = fmaf(v[i][e].y, f[i], y[e].y);
                    y[e].z = fmaf(v[i][e].z, f[i], y[e].z);
                    y[e].w = fmaf(v[i][e].w, f[i], y[e].w);
                }
            }
        }
        if (live) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + orow * D + c);
#pragma unroll
            for (int e = 0; e < COLS / 8; ++e)
                dst[e] = make_uint4(pack_bf16(y[2 * e].x * inv, y[2 * e].y * inv),
                                    pack_bf16(y[2 * e].z * inv, y[2 * e].w * inv),
                                    pack_bf16(y[2 * e + 1].x * inv, y[2 * e + 1].y * inv),
                                    pack_bf16(y[2 * e + 1].z * inv, y[2 * e + 1].w * inv));
        }
    }
    if (live && a.lse && c0 == 0) a.lse[orow] = lse_of(mm, ll);
}

struct MassArgs {
    const __nv_bfloat16* q;
    long long q_stride;
    CacheView c;
    SeqView s;
    int q_heads, group;
    int tiles;               // the tiles kernel: key tile pairs of the longest sequence
    float scale_log2;
    float lse_scale, nothing;   // the tiles kernel: -log2(e) / scale_log2; what a row that weighs nothing gets
    int window;
    const float* lse;
    float decay;
    const float* mass;       // may be out: plain loads, none that take it for read-only
    float* out;
};

cudaError_t launch_mass_rows(const MassArgs& a, const void* k, int sms, cudaStream_t stream);
cudaError_t launch_mass_tiles(const MassArgs& a, const void* k, int sms, cudaStream_t stream);
cudaError_t launch_attn_rows(const AttnArgs& a, const void* k, const void* v, int sms, cudaStream_t stream);
cudaError_t launch_attn_tiles(const AttnArgs& a, const void* k, const void* v, int sms, cudaStream_t stream);
cudaError_t launch_attn_chunk(const AttnArgs& a, const void* k, const void* v, int sms, cudaStream_t stream);
size_t attn_rows_workspace(int D);
size_t attn_tiles_workspace(int D);
size_t attn_chunk_workspace(int D);

}  // namespace tern
