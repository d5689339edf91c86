// tern_mass_tiles.cu -- the attention weight of many query rows a key head
// (prompt chunks), added to each key's running mass, on the tcgen05 tensor
// cores.
//
// The scores are computed transposed, S^T = K Q^T: a key is a row of the
// product, so a thread owns a key and its sum over the query rows is a sum of
// its own registers (no exchange, no atomics, a fixed order).  With the lse known
// a weight is exp2(S - lse) at once, and the lse, a constant of a column, is
// subtracted by the product itself: one more K = 16 step multiplies three ones
// on K's side with -lse / scale on Q's, as the sum of three bf16 values (24
// bits).  Reading it from shared memory instead, broadcast to every thread, cost
// four wavefronts a 16-byte load beside products that already take the whole
// bandwidth of shared memory (512 tokens over 16k keys, 32 heads of 128: 99 us then,
// 66 us, 1.03 PFLOP/s, now).
// An item is NS key tiles of 128 keys (two; one at D = 256) of one sequence and
// key head.  K's tiles are brought once and stay; the query rows that see them
// stream past in tiles of 128 packed rows (128 / group tokens, every head of
// the group), each used by both key tiles:
//   * a TMA warp fills K (double-buffered where it fits) and the ring of Q tiles;
//     another writes the lse step beside each;
//   * two threads issue S^T = K Q^T, for all key tiles, one for the even row tiles
//     and one for the odd, each into its own tensor-memory buffers: issuing is
//     nearly synchronous, and one thread's products cover the other's waits and
//     commits (a thread a key tile, with twice the commits: 1800 clocks a pair of
//     tiles against the products' 1152);
//   * a warpgroup a key tile reads S^T, exponentiates and adds.
// Items are whole and dealt out in equal contiguous shares of their row tiles;
// where a CTA has three or four, the fourth is what the others wait for.
#include <algorithm>
#include <type_traits>

#include "tern_attn.cuh"

namespace tern {
namespace {

using namespace sm100;

__device__ int g_mass_tiles_error;

constexpr int kKeys = 128, kRows = 128;
constexpr int kChunk = 64 * kKeys * 2;
// row tiles' time that an item costs besides its own (four prompts of up to 2000 tokens 59, 52, 66, 52 us
// and 2 x 300 tokens, window 4096, heads of 256 30, 35, 36, 36 us with 1, 2, 3, 5)
constexpr int kItemCost = 1;

template <int D>
struct Cfg {
    static constexpr int NC = D / 64;
    static constexpr int NS = D == 256 ? 1 : 2;
    static constexpr int kTile = NC * kChunk;
    static constexpr int KB = D == 256 ? 1 : 2;                 // buffers of K's tiles
    static constexpr int kSlots = D == 64 ? 6 : 2;              // Q tiles in flight
    static constexpr int kSoftWarps = 4 * NS;
    static constexpr int kThreads = 32 * (kSoftWarps + 4);
    static constexpr size_t kSmemRing = (size_t)KB * NS * kTile;
    static constexpr size_t kSmemLse = kSmemRing + (size_t)kSlots * kTile;        // [slot][128 rows][16] bf16
    static constexpr size_t kSmemOne = kSmemLse + (size_t)kSlots * kRows * 32;    // [128 keys][16]: 1, 1, 1, 0, ...
    static constexpr size_t kSmemBar = kSmemOne + (size_t)kKeys * 32;
    // barriers: q_full[slots], q_empty[slots], k_full[KB], k_empty[KB], s_full[2], s_empty[2], drain[2]
    static constexpr int kBars = 2 * kSlots + 2 * KB + 6;
    static constexpr size_t kSmemMisc = kSmemBar + kBars * 8;
    static constexpr size_t kSmem = kSmemMisc + 256 + 1024;
};
constexpr uint32_t kIdesc = idesc_bf16_f32(kKeys, kRows);

// A key tile pair against the row tiles that see any of its keys.
struct KeyTileExtent {
    int group, window, keys, tokens;   // keys of a pair, tokens of a row tile
    __device__ __forceinline__ void operator()(Item& t) const {
        t.j0 = t.rt * keys;
        t.j1 = min(t.j0 + keys, t.q.len);
        t.rows = t.q.n * group;
        if (t.j0 >= t.q.len) {
            t.units = 0;
            return;
        }
        int lo, hi;
        row_tiles(t, lo, hi);
        t.units = kItemCost + hi - lo;   // keys that nobody sees still decay
    }
    // row tiles [lo, hi): token i sees key j when j - (len - n) <= i (and i < that + window)
    __device__ __forceinline__ void row_tiles(const Item& t, int& lo, int& hi) const {
        const int first = max(t.j0 - (t.q.len - t.q.n), 0);
        const int end = window > 0 ? (int)min((long long)t.q.n, (long long)t.j1 - 1 - (t.q.len - t.q.n) + window) : t.q.n;
        lo = first / tokens;
        hi = end > first ? (end - 1) / tokens + 1 : lo;
    }
};

// Row r of a K = 16 step: x, y, z and thirteen zeros.
__device__ __forceinline__ void write_step(unsigned char* base, int r, float x, float y, float z) {
    const int flip = (r >> 2) & 1;
    *reinterpret_cast<uint4*>(base + r * 32 + 16 * flip) = make_uint4(pack_bf16(x, y), pack_bf16(z, 0.0f), 0, 0);
    *reinterpret_cast<uint4*>(base + r * 32 + 16 * (1 - flip)) = make_uint4(0, 0, 0, 0);
}

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
mass_tiles_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                  const MassArgs a, const int box_rows) {
    using C = Cfg<D>;
    constexpr int NC = C::NC, NS = C::NS, KB = C::KB, kSlots = C::kSlots;
    extern __shared__ __align__(1024) unsigned char smem_dyn[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem), bar0 = sbase + (uint32_t)C::kSmemBar;
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    enum { Q_FULL = 0, Q_EMPTY = kSlots, K_FULL = 2 * kSlots, K_EMPTY = K_FULL + KB, S_FULL = K_EMPTY + KB,
           S_EMPTY = S_FULL + 2, DRAIN = S_EMPTY + 2 };
    long long* sm_scan = reinterpret_cast<long long*>(smem + C::kSmemMisc);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm_scan + 8 + C::kThreads / 32);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kBars; ++i) {
            int count = 1;
            if (i >= K_EMPTY && i < K_EMPTY + KB) count = 2;
            if (i >= S_EMPTY && i < S_EMPTY + 2) count = 4 * NS;
            if (i < kSlots) count = 2;   // the copy, and the lse step
            mbar_init(bar(i), count);
        }
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmap_q);
        tma_prefetch_desc(&tmap_k);
    }
    for (int r = threadIdx.x; r < kKeys; r += C::kThreads)
        write_step(smem + C::kSmemOne, r, 1.0f, 1.0f, 1.0f);
    const int tokens = kRows / a.group, tile_rows = tokens * a.group;
    // the rows of a Q tile that no copy fills (a group that does not divide 128) are 0: finite scores, which the lse
    // step takes to no weight
    for (int i = threadIdx.x; i < kSlots * NC * (kRows - tile_rows) * 8; i += C::kThreads) {
        const int x = i / ((kRows - tile_rows) * 8), r = tile_rows + i / 8 % (kRows - tile_rows);
        *reinterpret_cast<uint4*>(smem + C::kSmemRing + x * kChunk + r * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    if (warp == C::kSoftWarps) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_dependents();
    pdl_wait();

    const KeyTileExtent extent{a.group, a.window, NS * kKeys, tokens};
    int P;
    long long total, w0, w1;
    Item t;
    const bool busy = find_share<C::kThreads>(a.s, a.c, extent, a.tiles, 1, (int)blockIdx.x, (int)gridDim.x, sm_scan, &g_mass_tiles_error, total, P, w0,
                                              w1, t);
    // whole items: those that begin in this CTA's share
    if (busy && t.at < w0) next_item(a.s, a.c, extent, a.tiles, t, &g_mass_tiles_error);
    auto fail = [&] {
        if (!*abort_flag) {
            *abort_flag = 1;
            report_device_error(&g_mass_tiles_error, TERN_DEVERR_ATTN_WAIT);
        }
    };
    auto wait = [&](uint32_t b, uint32_t parity) { return mbar_wait_bounded(b, parity, abort_flag, kAttnWaitNs); };

    if (!busy) {
    } else if (warp == C::kSoftWarps) {
        // ------------------------------ TMA ------------------------------
        uint32_t it = 0, kt = 0;
        bool ok = true;
        const int boxes = kKeys / box_rows;
        while (t.at < w1 && ok) {
            int lo, hi;
            extent.row_tiles(t, lo, hi);
            if (hi > lo) {
                const int* trow = a.s.table + (long long)t.b * a.s.width;
                const uint32_t kb = kt % KB;
                if (!__all_sync(0xffffffffu, wait(bar(K_EMPTY + (int)kb), ((kt / KB) & 1u) ^ 1u))) { ok = false; break; }
                // boxes of the pair that hold a key, for every chunk
                const int live = min(NS * boxes, (t.j1 - t.j0 + box_rows - 1) / box_rows);
                if (lane == 0) mbar_arrive_expect_tx(bar(K_FULL + (int)kb), (uint32_t)(live * NC * box_rows * 128));
                __syncwarp();
                for (int i = lane; i < live * NC; i += 32) {
                    const int x = i / NC, c = i % NC, key = t.j0 + x * box_rows;
                    const int page = checked_page(trow[key / a.c.page_size], a.c.pages, &g_mass_tiles_error);
                    tma_load_cache(sbase + (uint32_t)(((kb * NS + x / boxes) * NC + c) * kChunk + x % boxes * box_rows * 128),
                                   &tmap_k, key % a.c.page_size, c, t.hk, page, bar(K_FULL + (int)kb));
                }
                ++kt;
                for (int r = lo; r < hi; ++r, ++it) {
                    const uint32_t s = it % kSlots;
                    if (!__all_sync(0xffffffffu, wait(bar(Q_EMPTY + (int)s), ((it / kSlots) & 1u) ^ 1u))) { ok = false; break; }
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar(Q_FULL + (int)s), (uint32_t)(NC * tile_rows * 128));
                        for (int c = 0; c < NC; ++c)
                            tma_load_q(sbase + (uint32_t)(C::kSmemRing + s * C::kTile + c * kChunk), &tmap_q,
                                       t.hk * a.group, t.q.q0 + r * tokens, c, bar(Q_FULL + (int)s));
                    }
                }
            }
            next_item(a.s, a.c, extent, a.tiles, t, &g_mass_tiles_error);
            if (t.b >= a.s.B) break;
        }
        if (!ok && lane == 0) {
            fail();
            for (uint32_t i = it < (uint32_t)kSlots ? 0 : it - kSlots; i < it; ++i)
                (void)mbar_wait_drain(bar(Q_FULL + (int)(i % kSlots)), (i / kSlots) & 1u, 20000000ull);
            for (uint32_t i = kt < (uint32_t)KB ? 0 : kt - KB; i < kt; ++i)
                (void)mbar_wait_drain(bar(K_FULL + (int)(i % KB)), (i / KB) & 1u, 20000000ull);
        }
        __syncwarp();
    } else if (warp == C::kSoftWarps + 1) {
        // ------------------------------ the lse steps ------------------------------
        uint32_t it = 0;
        bool ok = true;
        while (t.at < w1 && ok) {
            int lo, hi;
            extent.row_tiles(t, lo, hi);
            // the lse of this lane's four rows of a row tile, fetched a tile ahead
            const float* lse[4];
            float z[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int row = lane + 32 * x;
                lse[x] = a.lse + (long long)(t.q.q0 + row / a.group) * a.q_heads + t.hk * a.group + row % a.group;
            }
            auto fetch = [&](int r) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int row = lane + 32 * x;
                    z[x] = row < tile_rows && r * tile_rows + row < t.rows ? lse[x][(long long)r * tokens * a.q_heads] : -INFINITY;
                }
            };
            if (hi > lo) fetch(lo);
            for (int r = lo; r < hi; ++r, ++it) {
                const uint32_t s = it % kSlots;
                if (!__all_sync(0xffffffffu, wait(bar(Q_EMPTY + (int)s), ((it / kSlots) & 1u) ^ 1u))) { ok = false; break; }
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    // a row that weighs nothing (lse -inf: it sees no key; +inf: exp(s - inf)) gets a finite value that
                    // leaves exp2 at 0: 0 * inf would be NaN
                    const float v = fabsf(z[x]) == INFINITY ? a.nothing : z[x] * a.lse_scale;
                    const float top = __bfloat162float(__float2bfloat16_rn(v));
                    const float mid = __bfloat162float(__float2bfloat16_rn(v - top));
                    write_step(smem + C::kSmemLse + s * (kRows * 32), lane + 32 * x, top, mid, v - top - mid);
                }
                if (r + 1 < hi) fetch(r + 1);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(Q_FULL + (int)s));
            }
            next_item(a.s, a.c, extent, a.tiles, t, &g_mass_tiles_error);
            if (t.b >= a.s.B) break;
        }
        if (!ok && lane == 0) fail();
        __syncwarp();
    } else if (warp > C::kSoftWarps) {
        // ------------------------------ MMA, one thread a parity of row tiles ------------------------------
        if (lane == 0) {
            const uint32_t me = (uint32_t)(warp - C::kSoftWarps - 2);
            uint32_t it = 0, kt = 0;
            bool ok = true, issued = false;
            while (t.at < w1 && ok) {
                int lo, hi;
                extent.row_tiles(t, lo, hi);
                if (hi > lo) {
                    const uint32_t kb = kt % KB;
                    ok = wait(bar(K_FULL + (int)kb), (kt / KB) & 1u);
                    for (int r = lo; r < hi && ok; ++r, ++it) {
                        if ((it & 1u) != me) continue;
                        const uint32_t s = it % kSlots;
                        ok = wait(bar(Q_FULL + (int)s), (it / kSlots) & 1u);
                        ok = ok && wait(bar(S_EMPTY + (int)me), ((it >> 1) & 1u) ^ 1u);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int x = 0; x < NS; ++x) {   // (a pair's second tile may hold no key: its sums are not stored)
#pragma unroll
                            for (int c = 0; c < NC; ++c) {
                                const uint64_t kd = smem_desc_k_sw128(sbase + (uint32_t)(((kb * NS + x) * NC + c) * kChunk));
                                const uint64_t qd = smem_desc_k_sw128(sbase + (uint32_t)(C::kSmemRing + s * C::kTile + c * kChunk));
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    mma_f16_ss(tmem + 256u * x + 128u * me, kd + 2 * kk, qd + 2 * kk, kIdesc, (c | kk) ? 1u : 0u);
                            }
                            mma_f16_ss(tmem + 256u * x + 128u * me, smem_desc_k_sw32(sbase + (uint32_t)C::kSmemOne),
                                       smem_desc_k_sw32(sbase + (uint32_t)(C::kSmemLse + s * (kRows * 32))), kIdesc, 1u);
                        }
                        issued = true;
                        mma_commit(bar(S_FULL + (int)me));
                        mma_commit(bar(Q_EMPTY + (int)s));
                    }
                    if (!ok) break;
                    mma_commit(bar(K_EMPTY + (int)kb));   // (at once where this thread had no product)
                    ++kt;
                }
                next_item(a.s, a.c, extent, a.tiles, t, &g_mass_tiles_error);
                if (t.b >= a.s.B) break;
            }
            if (!ok) {
                fail();
                if (issued) {
                    mma_commit(bar(DRAIN + (int)me));
                    (void)mbar_wait_drain(bar(DRAIN + (int)me), 0u, 100000000ull);
                }
            }
        }
        __syncwarp();
    } else {
        // ------------------------------ weights and sums ------------------------------
        const int me = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
        uint32_t it = 0;
        bool ok = true;
        const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2);
        const float skip = a.scale_log2 < 0.0f ? INFINITY : -INFINITY;   // times the scale: -inf
        while (t.at < w1 && ok) {
            int lo, hi;
            extent.row_tiles(t, lo, hi);
            const int key = t.j0 + me * kKeys + row;
            long long at = -1;   // where this key's mass is; -1: no key, or a bad page id
            float old = 0.0f;
            if (key < t.j1) {
                const int page = checked_page_to_write(a.s.table[(long long)t.b * a.s.width + key / a.c.page_size], a.c.pages, &g_mass_tiles_error);
                if (page >= 0) {
                    at = ((long long)page * a.c.kv_heads + t.hk) * a.c.page_size + key % a.c.page_size;
                    old = a.mass[at];
                }
            }
            // tokens [first, end) see this key
            const int first = key - (t.q.len - t.q.n);
            const int end = a.window > 0 ? (int)min((long long)t.q.n, (long long)first + a.window) : t.q.n;
            const int k_lo = t.j0 + me * kKeys - (t.q.len - t.q.n);   // of the tile's first key; its last is 127 above
            uint64_t sum[4] = {0, 0, 0, 0};
            for (int r = lo; r < hi; ++r, ++it) {
                const int odd = (int)(it & 1u);
                if (!__all_sync(0xffffffffu, wait(bar(S_FULL + odd), (it >> 1) & 1u))) { ok = false; break; }
                tc_fence_after();
                const uint32_t ts = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(256 * me + 128 * odd);
                const int tok0 = r * tokens;
                // some column of the tile may not see some key of it (or is no row of the sequence)
                const bool ends = (r + 1) * tile_rows > t.rows || (a.window > 0 && tok0 + tokens - 1 >= k_lo + a.window);
                const bool masked = ends || tok0 < k_lo + kKeys - 1;
                const int c0 = max(first - tok0, 0) * a.group, c1 = min(max(end - tok0, 0) * a.group, tile_rows);
                // 32 columns at a time, the next ones on their way meanwhile; tiles that all see apart,
                // without a branch between their exponentials (72 us -> 65)
                auto weigh = [&](auto some) {
                    uint32_t x[2][32];
                    tmem_ld_x32(ts, x[0]);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (i < 3) tmem_ld_x32(ts + 32u * (i + 1), x[(i + 1) & 1]);
                        float u[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) u[e] = __uint_as_float(x[i & 1][e]);
                        if constexpr (some.value) {
                            // (the lse step alone covers rows that weigh nothing, not scores that are not finite)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (32 * i + e < c0) u[e] = skip;
                            if (ends)
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (32 * i + e >= c1) u[e] = skip;
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += 2) unpack2(mul2(pack2(u[e], u[e + 1]), scale2), u[e], u[e + 1]);
#pragma unroll
                        for (int e = 0; e < 32; ++e) u[e] = exp2_fast(u[e]);
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
#pragma unroll
                            for (int y = 0; y < 4; ++y) sum[y] = add2(sum[y], pack2(u[e + 2 * y], u[e + 2 * y + 1]));
                        if (i < 3) tmem_ld_wait();
                        if (i == 2) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(bar(S_EMPTY + odd));
                        }
                    }
                };
                if (masked) weigh(std::true_type{});
                else weigh(std::false_type{});
            }
            if (!ok) break;
            if (at >= 0) {
                float x, y;
                unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), x, y);
                a.out[at] = fmaf(a.decay, old, x + y);
            }
            next_item(a.s, a.c, extent, a.tiles, t, &g_mass_tiles_error);
            if (t.b >= a.s.B) break;
        }
        if (!ok && lane == 0) fail();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == C::kSoftWarps) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D>
cudaError_t launch(MassArgs a, const void* k, int sms, cudaStream_t stream) {
    using C = Cfg<D>;
    int box = 128;
    while (a.c.page_size % box) box >>= 1;
    CUtensorMap mq, mk;
    if (!make_q_map(&mq, a.q, a.q_stride, a.q_heads, a.s.T, D, a.group, kRows / a.group) ||
        !make_cache_map(&mk, k, a.c, box, 1))
        return cudaErrorInvalidValue;
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(mass_tiles_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)C::kSmem);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    a.lse_scale = -1.44269504088896341f / a.scale_log2;
    a.nothing = a.scale_log2 < 0.0f ? 1e38f : -1e38f;   // times any scale a call may have: below every exponent
    a.tiles = (int)(((long long)a.s.width * a.c.page_size + C::NS * kKeys - 1) / (C::NS * kKeys));
    const long long items = (long long)a.s.B * a.c.kv_heads * a.tiles;
    return launch_pdl(mass_tiles_kernel<D>, dim3((unsigned)std::min<long long>(sms, items)), dim3(C::kThreads), C::kSmem,
                      stream, true, mq, mk, a, box);
}

}  // namespace

cudaError_t launch_mass_tiles(const MassArgs& a, const void* k, int sms, cudaStream_t stream) {
    switch (a.c.head_dim) {
        case 64: return launch<64>(a, k, sms, stream);
        case 128: return launch<128>(a, k, sms, stream);
        default: return launch<256>(a, k, sms, stream);
    }
}

cudaError_t read_mass_tiles_device_error(int* code) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_mass_tiles_error, sizeof(int));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_mass_tiles_error, &zero, sizeof(int));
}

}  // namespace tern
