// tern_attn_tiles.cu -- attention of query rows that fill one row tile a key
// head or less (verify steps, short chunks), and of any number at heads of 256
// values, on the tcgen05 tensor cores.
//
// A row tile is 128 packed rows (128 / group tokens, every head of the group),
// so one K and V tile serves all the heads that share it.  A CTA takes a row tile
// through a run of 128-key tiles:
//   * a TMA warp brings Q once and then K, another V, in chunks of 64 head
//     values x 128 keys (16 KB of 128-byte swizzled rows), through one ring; a
//     page gives boxes of up to 128 slots, one lane a box.  A copy takes a warp
//     about 110 clocks to issue, and a page id some 700 to look up (one warp
//     for both, without looking ahead, took 2000 to 3000 a tile and bound every
//     call), hence two warps, and ids fetched 32 boxes ahead;
//   * two threads issue S = Q K^T (both operands in shared memory, K-major) and
//     O += P V (P in tensor memory, V MN-major) with M = 128;
//   * warpgroups, one thread a row, read S, take the running maximum, write P =
//     exp2(S - m) as bf16 over S's own columns and keep the sum in fp32.  O is
//     only rescaled when a score passes the maximum in use by 2^8, so P and the
//     sums stay below 2^8 of their largest term.
// At D <= 128 two streams, each with an MMA thread, a warpgroup, an S and an O,
// take the even and the odd key tiles; the first one's warpgroup then adds both
// (tensor memory is open to it).  Such calls are bound by reading the cache, and
// warps without a live row do no arithmetic.  At D = 256, where one O takes half
// of tensor memory, there is one stream with two S buffers: one thread issues QK,
// ahead by a tile, the other PV.  Row tiles that read the same keys are then
// bound by L2's rate, 8.5 TB/s (2 x 300 tokens, window of 4096: 61 us), and a
// verify step by the cache's (4 x 5 tokens over 32k keys, 8 key heads of 128: 94 us,
// 5.6 TB/s, the last 8 us the joins).
// Slots past a sequence's last key and before its windows may hold anything: scores are masked before
// the exponential and V's rows are zeroed in shared memory by the TMA warp
// before the tile is handed on (a row of P is 0 there, and 0 * NaN is not).
// Work is shared out as in the rows kernel: equal contiguous shares of all
// (sequence, row tile, key head) items' 128-key tiles; parts meet in the
// workspace, and the warp that counts last for its 32 rows adds them in order.
#include "tern_attn.cuh"

namespace tern {
namespace {

using namespace sm100;

__device__ int g_attn_tiles_error;

constexpr int kKeys = 128, kRows = kTileRows;
constexpr int kChunk = 64 * kKeys * 2;      // 16 KB: 64 head values of 128 keys (or rows)
constexpr int kItemCost = 3;                // key tiles' time that an item costs besides its own (2 and 4: within 3 %)
constexpr int kMinTiles = 4;                // key tiles a share holds at least

template <int D>
struct Cfg {
    static constexpr int NC = D / 64;                       // chunks of a K, V or Q tile
    static constexpr int NS = D == 256 ? 1 : 2;             // streams: every NS-th key tile each
    static constexpr int CG = D == 64 ? 1 : 2;             // chunks of a ring slot
    static constexpr int NG = NC / CG;                      // slots of a K or V tile
    static constexpr int kSlots = D == 64 ? 10 : D == 128 ? 5 : 4;
    static constexpr int kSoftWarps = 4 * NS;
    // two streams: a third warpgroup (two TMA and two MMA warps) gives registers
    // to the softmax warps, which hold a row of S each: 256 x 208 + 128 x 88 =
    // 384 x 168, what the CTA was launched with
    static constexpr int kThreads = NS == 2 ? 384 : 256;
    static constexpr uint32_t kS = 0, kO = 256;             // tensor memory: S (and P) at 128 b, O at kO + D s
    static constexpr size_t kSmemRing = (size_t)NC * kChunk;
    static constexpr size_t kSmemBar = kSmemRing + (size_t)kSlots * CG * kChunk;
    // barriers: full[slots], empty[slots], then pairs: q_full, q_empty, s_full,
    // s_empty, p_full, o_full, o_empty, drain; tail, merge, join
    static constexpr int kBars = 2 * kSlots + 19;
    static constexpr size_t kSmemMisc = kSmemBar + kBars * 8;
    static constexpr size_t kSmemStat = kSmemMisc + 256;              // the second stream's (m, l)
    static constexpr size_t kSmem = kSmemStat + (NS == 2 ? kRows * 8 : 0) + 1024;
};
constexpr uint32_t kIdescQK = idesc_bf16_f32(kRows, kKeys);

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
attn_tiles_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                  const __grid_constant__ CUtensorMap tmap_v, const AttnArgs a, const int box_rows) {
    using C = Cfg<D>;
    constexpr int NC = C::NC, NS = C::NS, CG = C::CG, NG = C::NG, kSlots = C::kSlots;
    constexpr bool kWide = D == 256;   // one row tile, two S buffers
    extern __shared__ __align__(1024) unsigned char smem_dyn[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem), bar0 = sbase + (uint32_t)C::kSmemBar;
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    auto full_bar = [&](uint32_t i) { return bar((int)(i % kSlots)); };
    auto empty_bar = [&](uint32_t i) { return bar(kSlots + (int)(i % kSlots)); };
    auto slot_phase = [&](uint32_t i) { return (i / kSlots) & 1u; };
    auto slot_addr = [&](uint32_t i) { return sbase + (uint32_t)C::kSmemRing + (i % kSlots) * (uint32_t)(CG * kChunk); };
    enum { Q_FULL = 2 * kSlots, Q_EMPTY = Q_FULL + 2, S_FULL = Q_EMPTY + 2, S_EMPTY = S_FULL + 2, P_FULL = S_EMPTY + 2,
           O_FULL = P_FULL + 2, O_EMPTY = O_FULL + 2, DRAIN = O_EMPTY + 2, TAIL = DRAIN + 2, MERGE = TAIL + 1, JOIN };
    long long* sm_scan = reinterpret_cast<long long*>(smem + C::kSmemMisc);   // [8 + warps]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm_scan + 8 + C::kThreads / 32);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* join_flag = const_cast<volatile int*>(abort_flag) + 1;      // [2][4]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kBars; ++i) {
            const bool by_warps = (i >= P_FULL && i < P_FULL + 2) || (i >= O_EMPTY && i < O_EMPTY + 2) || i == MERGE ||
                                  i == JOIN;
            const bool by_threads = NS == 2 && ((i >= kSlots && i < 2 * kSlots) || i == Q_EMPTY);   // both MMA threads
            mbar_init(bar(i), by_warps ? 4 : by_threads ? 2 : 1);
        }
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmap_q);
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
    }
    if (warp == C::kSoftWarps + 1) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_dependents();
    pdl_wait();

    const int tile_rows = kRows / a.group * a.group;   // whole tokens
    int P;
    long long total, w0, w1;
    Item t;
    const RowTileExtent<kKeys, kItemCost> extent{tile_rows, a.group, a.window};
    const bool busy = find_share<C::kThreads>(a.s, a.c, extent, a.tiles, kMinTiles, (int)blockIdx.x, (int)gridDim.x,
                                              sm_scan, &g_attn_tiles_error, total, P, w0, w1, t);
    auto fail = [&] {
        if (!*abort_flag) {
            *abort_flag = 1;
            report_device_error(&g_attn_tiles_error, TERN_DEVERR_ATTN_WAIT);
        }
    };
    auto wait = [&](uint32_t b, uint32_t parity) { return mbar_wait_bounded(b, parity, abort_flag, kAttnWaitNs); };

    if (!busy) {
        // no share: straight to the end
    } else if (warp >= C::kSoftWarps) {
      if constexpr (NS == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
      if (warp == C::kSoftWarps || warp == C::kSoftWarps + 3) {
        // ------------------------------ TMA: Q and K, or V ------------------------------
        const bool is_v = warp != C::kSoftWarps;
        const CUtensorMap* map = is_v ? &tmap_v : &tmap_k;
        uint32_t it = is_v ? NG : 0, used = 0, tails = 0;   // slots: K(0), V(0), K(1), ...
        bool ok = true;
        const int boxes = kKeys / box_rows, c = lane / boxes, box = lane - c * boxes;   // this lane's piece of a tile
        for (long long w = w0; w < w1 && ok;) {
            const Segment seg = segment_of(extent, t, w, w1);
            const int nt = seg.n, key0 = seg.first * kKeys;
            const int* trow = a.s.table + (long long)t.b * a.s.width;
            // lane i: the page of box i of the current 32 boxes of this segment, and of the next 32
            auto raw_id = [&](int x) {
                const int k = key0 + x * box_rows;
                return x < nt * boxes && k < t.q.len && k + box_rows > t.j0 ? trow[(unsigned)k / (unsigned)a.c.page_size] : 0;
            };
            int ids = 0, ahead = raw_id(lane);
            if (!is_v && nt > 0) {
                if (!__all_sync(0xffffffffu, wait(bar(Q_EMPTY), (used & 1u) ^ 1u))) { ok = false; break; }
                ++used;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar(Q_FULL), (uint32_t)(NC * tile_rows * 128));
                    const int tok = t.q.q0 + t.rt * (tile_rows / a.group);
                    for (int x = 0; x < NC; ++x)
                        tma_load_q(sbase + (uint32_t)(x * kChunk), &tmap_q, t.hk * a.group, tok, x, bar(Q_FULL));
                }
            }
            for (int j = 0; j < nt && ok; ++j) {
                if (((j * boxes) & 31) == 0) {
                    ids = checked_page(ahead, a.c.pages, &g_attn_tiles_error);
                    ahead = raw_id(j * boxes + 32 + lane);
                }
                const int page = __shfl_sync(0xffffffffu, ids, (j * boxes + box) & 31);
                const int k0 = key0 + j * kKeys, k = k0 + box * box_rows;
                // boxes that hold no key of these rows are not read; V's rows there count as 0
                const bool use = c < NC && k < t.q.len && k + box_rows > t.j0;
                const VRows rows(k0, kKeys, box_rows, t.j0, t.q.len);
                const bool part = is_v && rows.inside(), unread = is_v && (rows.front > 0 || rows.back_box < kKeys);
                const uint32_t mine = __ballot_sync(0xffffffffu, use);
                const uint32_t bytes = (uint32_t)__popc(mine & ((1u << boxes) - 1u)) * box_rows * 128u;   // a chunk's
                const int slot = (unsigned)k % (unsigned)a.c.page_size;
                if (part && lane == 0) mbar_arrive_expect_tx(bar(TAIL), bytes * NC);
                for (int g = 0; g < NG; ++g) {
                    if (!__all_sync(0xffffffffu, wait(empty_bar(it + g), slot_phase(it + g) ^ 1u))) {
                        ok = false;
                        break;
                    }
                    unsigned char* chunks = smem + C::kSmemRing + ((it + g) % kSlots) * (CG * kChunk);
                    if (unread) {
                        for (int x = 0; x < CG; ++x) {
                            zero_rows(chunks + x * kChunk, 0, rows.front);
                            zero_rows(chunks + x * kChunk, rows.back_box, kKeys);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (!part && lane == 0) mbar_arrive_expect_tx(full_bar(it + g), bytes * CG);
                    __syncwarp();
                    if (use && c / CG == g)
                        tma_load_cache(slot_addr(it + g) + (uint32_t)((c % CG) * kChunk + box * box_rows * 128), map,
                                       slot, c, t.hk, page, part ? bar(TAIL) : full_bar(it + g));
                }
                if (!ok) break;
                if (part) {
                    if (!__all_sync(0xffffffffu, wait(bar(TAIL), tails & 1u))) {
                        ok = false;
                        break;
                    }
                    ++tails;
                    for (int x = 0; x < NC; ++x)
                        rows.zero_inside(smem + C::kSmemRing + (((it + x / CG) % kSlots) * CG + x % CG) * kChunk);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        for (int g = 0; g < NG; ++g) mbar_arrive(full_bar(it + g));
                }
                it += 2 * NG;
            }
            w = seg.we;
            if (w < w1) next_item(a.s, a.c, extent, a.tiles, t, &g_attn_tiles_error);
        }
        if (!ok && lane == 0) {
            fail();
            // copies in flight land before the CTA goes away
            for (uint32_t i = it < 2 * kSlots ? (is_v ? NG : 0) : it - 2 * kSlots; i <= it; i += 2 * NG)
                for (int g = 0; g < NG; ++g) (void)mbar_wait_drain(full_bar(i + g), slot_phase(i + g), 20000000ull);
            if (used) (void)mbar_wait_drain(bar(Q_FULL), (used - 1u) & 1u, 20000000ull);
            if (is_v) (void)mbar_wait_drain(bar(TAIL), tails & 1u, 20000000ull);
        }
        __syncwarp();
      } else if (warp <= C::kSoftWarps + 2) {
        // ------------------------------ MMA ------------------------------
        if (lane == 0) {
            constexpr uint32_t kIdescPV = idesc_bf16_f32(kRows, D) | kIdescBMnMajor;
            const int me = warp - C::kSoftWarps - 1;
            uint32_t it = 0, used = 0, jobs = 0;
            bool ok = true, issued = false;
            auto need = [&](uint32_t b, uint32_t parity) {
                if (ok && !wait(b, parity)) ok = false;
                return ok;
            };
            auto qk = [&](uint32_t buf, int c, uint32_t addr) {   // S(buf) (+)= chunk c of Q K^T
                const uint64_t qd = smem_desc_k_sw128(sbase + (uint32_t)(c * kChunk));
                const uint64_t kd = smem_desc_k_sw128(addr);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_f16_ss(tmem + C::kS + 128u * buf, qd + 2 * kk, kd + 2 * kk, kIdescQK, (c | kk) ? 1u : 0u);
                issued = true;
            };
            auto pv = [&](int s, uint32_t buf, uint32_t addr, bool acc) {   // O(s) (+)= P(buf) V
                const uint64_t vd = smem_desc_mn_sw128(addr, kChunk);
#pragma unroll
                for (int kk = 0; kk < kKeys / 16; ++kk)
                    mma_f16_ts(tmem + C::kO + (uint32_t)(D * s), tmem + C::kS + 128u * buf + 8u * kk,
                               vd + (uint64_t)(kk * (2048 >> 4)), kIdescPV, (acc || kk) ? 1u : 0u);
                issued = true;
            };
            for (long long w = w0; w < w1 && ok;) {
                const Segment seg = segment_of(extent, t, w, w1);
                const int nt = seg.n;
                if constexpr (NS == 2) {
                    // QK(j), PV(j) of every second key tile; of the others only the slots are released
                    if (nt > 0) need(bar(Q_FULL), used & 1u);
                    for (int j = 0; j < nt && ok; ++j) {
                        const bool mine = (j & 1) == me;
                        if (!need(full_bar(it), slot_phase(it))) break;
                        if (mine) {
                            tc_fence_after();
#pragma unroll
                            for (int c = 0; c < NC; ++c) qk(me, c, slot_addr(it) + (uint32_t)(c * kChunk));
                            mma_commit(bar(S_FULL + me));
                            mma_commit(empty_bar(it));
                            if (j + 2 >= nt) mma_commit(bar(Q_EMPTY));   // its last use: the next may come
                        } else {
                            mbar_arrive(empty_bar(it));
                        }
                        ++it;
                        if (!need(full_bar(it), slot_phase(it))) break;
                        if (mine) {
                            if (!need(bar(P_FULL + me), jobs++ & 1u)) break;
                            // the previous item's output has been read
                            if (j == me && !need(bar(O_EMPTY + me), (used & 1u) ^ 1u)) break;
                            tc_fence_after();
                            pv(me, me, slot_addr(it), j != me);
                            mma_commit(empty_bar(it));
                        } else {
                            mbar_arrive(empty_bar(it));
                        }
                        ++it;
                    }
                    if (nt > 0 && ok) {
                        // a stream without a tile of this item says nothing of its O: no P of its warpgroup
                        // came first, so the barrier could run two phases ahead of that warpgroup
                        if (me < nt) mma_commit(bar(O_FULL + me));
                        else mbar_arrive(bar(Q_EMPTY));
                        ++used;
                    }
                } else if (me == 0) {
                    if (nt > 0) need(bar(Q_FULL), used & 1u);
                    for (int j = 0; j < nt && ok; ++j, ++jobs) {
                        // the P that was over this S, two tiles back, has been used
                        if (!need(bar(S_EMPTY + (int)(jobs & 1u)), ((jobs >> 1) & 1u) ^ 1u)) break;
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            if (!need(full_bar(it + g), slot_phase(it + g))) break;
                            tc_fence_after();
#pragma unroll
                            for (int c = 0; c < CG; ++c) qk(jobs & 1u, g * CG + c, slot_addr(it + g) + (uint32_t)(c * kChunk));
                            if (g == NG - 1) mma_commit(bar(S_FULL + (int)(jobs & 1u)));
                            mma_commit(empty_bar(it + g));
                        }
                        it += 2 * NG;
                    }
                    if (nt > 0 && ok) {
                        mma_commit(bar(Q_EMPTY));
                        ++used;
                    }
                } else {
                    for (int j = 0; j < nt && ok; ++j, ++jobs) {
                        it += NG;
#pragma unroll
                        for (int g = 0; g < NG; ++g) need(full_bar(it + g), slot_phase(it + g));
                        need(bar(P_FULL + (int)(jobs & 1u)), (jobs >> 1) & 1u);
                        if (j == 0) need(bar(O_EMPTY), (used & 1u) ^ 1u);
                        if (!ok) break;
                        tc_fence_after();
                        pv(0, jobs & 1u, slot_addr(it), j > 0);   // (its slots lie one behind the other)
                        mma_commit(bar(O_FULL));
                        mma_commit(bar(S_EMPTY + (int)(jobs & 1u)));
#pragma unroll
                        for (int g = 0; g < NG; ++g) mma_commit(empty_bar(it + g));
                        it += NG;
                    }
                    if (nt > 0) ++used;
                }
                w = seg.we;
                if (w < w1) next_item(a.s, a.c, extent, a.tiles, t, &g_attn_tiles_error);
            }
            if (!ok) {
                fail();
                if (issued) {
                    mma_commit(bar(DRAIN + me));
                    (void)mbar_wait_drain(bar(DRAIN + me), 0u, 100000000ull);
                }
            }
        }
        __syncwarp();
      }
    } else {
        // ------------------------------ softmax, output ------------------------------
        if constexpr (NS == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int s = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t to = tmem + lanes + C::kO + (uint32_t)(D * s);
        // S tiles and finished O's of this stream, items with keys, merged and joined items
        uint32_t sc = 0, oc = 0, items = 0, merges = 0, joins = 0;
        const bool flip = a.scale_log2 < 0.0f;
        const float scale = fabsf(a.scale_log2);
        bool ok = true;
        for (long long w = w0; w < w1 && ok;) {
            const Segment seg = segment_of(extent, t, w, w1);
            const int nt = seg.n;
            if (!seg.skip) {
                const int rows = t.rows, r = t.rt * tile_rows + row;   // packed row of the sequence
                const bool live = row < rows, idle = quad * 32 >= rows;
                const int p = t.q.len - t.q.n + r / a.group;
                const int hi = live ? p : -1, lo = a.window > 0 ? p - a.window : -1;
                const int p_lo = t.q.len - t.q.n + t.rt * tile_rows / a.group;
                const int p_hi = t.q.len - t.q.n + (t.rt * tile_rows + rows - 1) / a.group;
                const int key0 = seg.first * kKeys;
                float m = -INFINITY, l = 0.0f;
                for (int j = s; j < nt && ok; j += NS, ++sc) {
                    const uint32_t buf = kWide ? sc & 1u : (uint32_t)s;
                    const uint32_t ph = kWide ? (sc >> 1) & 1u : sc & 1u;
                    if (!__all_sync(0xffffffffu, wait(bar(S_FULL + (int)buf), ph))) { ok = false; break; }
                    if (idle) {
                        if (lane == 0) mbar_arrive(bar(P_FULL + (int)buf));
                        continue;
                    }
                    tc_fence_after();
                    const uint32_t ts = tmem + lanes + C::kS + 128u * buf;
                    uint32_t x[4][32];
#pragma unroll
                    for (int i = 0; i < 4; ++i) tmem_ld_x32(ts + 32u * i, x[i]);
                    tmem_ld_wait();
                    if (flip)
#pragma unroll
                        for (int i = 0; i < 128; ++i) x[i >> 5][i & 31] ^= 0x80000000u;
                    const int k0 = key0 + j * kKeys;
                    if (k0 + kKeys - 1 > p_lo || (a.window > 0 && k0 <= p_hi - a.window)) {
#pragma unroll
                        for (int i = 0; i < 128; ++i)
                            if (i > hi - k0) x[i >> 5][i & 31] = 0xff800000u;
                        if (a.window > 0)   // (apart: both in one test took whole prompts 153 us, not 142)
#pragma unroll
                            for (int i = 0; i < 128; ++i)
                                if (i <= lo - k0) x[i >> 5][i & 31] = 0xff800000u;
                    }
                    float mx[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        mx[i] = __uint_as_float(x[i][0]);
#pragma unroll
                        for (int e = 1; e < 31; e += 2)
                            mx[i] = max3(mx[i], __uint_as_float(x[i][e]), __uint_as_float(x[i][e + 1]));
                    }
                    const float top = max3(fmaxf(mx[0], __uint_as_float(x[0][31])), fmaxf(mx[1], __uint_as_float(x[1][31])),
                                           max3(mx[2], __uint_as_float(x[2][31]), fmaxf(mx[3], __uint_as_float(x[3][31]))));
                    // (rows of no query of the sequence hold what the copies left: they have no vote)
                    if (__any_sync(0xffffffffu, live && (top - m) * scale > 8.0f)) {
                        const float mn = fmaxf(m, top);
                        const float f = m == -INFINITY ? 0.0f : exp2_fast((m - mn) * scale);
                        m = mn;
                        l *= f;
                        if (j > s) {
                            if (kWide) {
                                // the product before this one is still adding into O
                                if (!__all_sync(0xffffffffu, wait(bar(O_FULL), (oc + (uint32_t)j - 1u) & 1u))) {
                                    ok = false;
                                    break;
                                }
                                tc_fence_after();
                            }
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                uint32_t o[16];
                                tmem_ld_x16(to + c, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tmem_st_x16(to + c, o);
                            }
                        }
                    }
                    const float mb = m == -INFINITY ? 0.0f : m * scale;
                    const uint64_t sc2 = pack2(scale, scale), mb2 = pack2(-mb, -mb);
                    uint64_t sum[2] = {0, 0};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float u, v;
                            unpack2(fma2(pack2(__uint_as_float(x[i][2 * e]), __uint_as_float(x[i][2 * e + 1])), sc2, mb2), u, v);
                            u = exp2_fast(u);
                            v = exp2_fast(v);
                            sum[e & 1] = add2(sum[e & 1], pack2(u, v));
                            pk[e] = pack_bf16(u, v);
                        }
                        tmem_st_x16(ts + 16u * i, pk);
                    }
                    float su, sv;
                    unpack2(add2(sum[0], sum[1]), su, sv);
                    l += su + sv;
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(P_FULL + (int)buf));
                }
                if (!ok) break;
                const long long orow = (long long)(t.q.q0 + r / a.group) * a.q_heads + t.hk * a.group + r % a.group;
                if (nt > 0) ++items;
                if (nt > s) {
                    oc += kWide ? (uint32_t)nt : 1u;
                    // (with two S buffers the product before the last may be running too)
                    bool done = !kWide || nt < 2 || wait(bar(O_FULL + s), (oc - 2u) & 1u);
                    done = done && wait(bar(O_FULL + s), (oc - 1u) & 1u);
                    if (!__all_sync(0xffffffffu, done)) { ok = false; break; }
                    tc_fence_after();
                }
                float m2 = m * scale;   // -inf stays
                float f0 = 1.0f, f1 = 0.0f;
                if (NS == 2 && nt > 0) {
                    float2* stat = reinterpret_cast<float2*>(smem + C::kSmemStat);
                    if (s == 1) {
                        // the first stream has read what the last item left here
                        if (items > 1 && !__all_sync(0xffffffffu, wait(bar(O_EMPTY + 1), items & 1u))) { ok = false; break; }
                        stat[row] = make_float2(m2, l);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(MERGE));
                    } else {
                        if (!__all_sync(0xffffffffu, wait(bar(MERGE), merges++ & 1u))) { ok = false; break; }
                        tc_fence_after();   // (the second stream waited for its last product)
                        const float2 o = stat[row];
                        const float mm = fmaxf(m2, o.x), base = mm == -INFINITY ? 0.0f : mm;
                        f0 = exp2_fast(m2 - base);
                        f1 = exp2_fast(o.x - base);
                        l = l * f0 + o.y * f1;
                        m2 = mm;
                    }
                }
                if (s == 0) {
                    float* part = a.partial + (size_t)(2 * blockIdx.x + (w == w0 ? 0 : 1)) * part_floats(D);
                    if (!idle)
                        emit_row<D>(a, seg.whole, part, row, live, orow, m2, l, [&](int c, uint32_t (&o)[32]) {
                            if (nt == 0) {
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = 0u;
                                return;
                            }
                            tmem_ld_x32(to + c, o);
                            if constexpr (NS == 2) {
                                uint32_t o1[32];   // (an accumulator that no product reached holds anything)
                                tmem_ld_x32(to + (uint32_t)D + c, o1);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 32; ++e) {
                                    const float x = f0 > 0.0f ? __uint_as_float(o[e]) * f0 : 0.0f;
                                    o[e] = __float_as_uint(f1 > 0.0f ? fmaf(__uint_as_float(o1[e]), f1, x) : x);
                                }
                            }
                            tmem_ld_wait();
                        });
                    if (nt > 0) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(bar(O_EMPTY));
                            if (NS == 2) mbar_arrive(bar(O_EMPTY + 1));
                        }
                    }
                    if (!seg.whole) {
                        // warps without rows take columns of those that have some (5 tokens over 32k keys of one
                        // head, 16 parts: 37.6 -> 34.6 us)
                        const int quads = rows > 64 ? 4 : rows > 32 ? 2 : 1, to_quad = quad & (quads - 1);
                        bool last = !idle && count_part<kItemCost>(t, a.counters + quad, total, P);
                        if (quads < 4) {
                            if (!idle && lane == 0) join_flag[(joins & 1u) * 4 + quad] = last;
                            __syncwarp();
                            if (lane == 0) mbar_arrive(bar(JOIN));
                            if (!__all_sync(0xffffffffu, wait(bar(JOIN), joins & 1u))) { ok = false; break; }
                            last = join_flag[(joins & 1u) * 4 + to_quad];
                            ++joins;
                        }
                        constexpr int kMost = D / join_columns(D);   // warps of a quad
                        const int of = min(4 / quads, kMost), mine = quad / quads, row2 = to_quad * 32 + lane;
                        const int r2 = t.rt * tile_rows + row2;
                        const long long orow2 = (long long)(t.q.q0 + r2 / a.group) * a.q_heads + t.hk * a.group + r2 % a.group;
                        if (last && mine < of)
                            add_parts<D, kItemCost>(a, t, a.partial, part_floats(D), row2, row2 < rows, orow2, total, P,
                                                    mine * (D / of), (mine + 1) * (D / of));
                    }
                }
            }
            w = seg.we;
            if (w < w1) next_item(a.s, a.c, extent, a.tiles, t, &g_attn_tiles_error);
        }
        if (!ok && lane == 0) fail();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == C::kSoftWarps + 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D>
cudaError_t launch(AttnArgs a, const void* k, const void* v, int sms, cudaStream_t stream) {
    using C = Cfg<D>;
    int box = 128;
    while (a.c.page_size % box) box >>= 1;   // page_size is a multiple of 16
    CUtensorMap mq, mk, mv;
    if (!make_q_map(&mq, a.q, a.q_stride, a.q_heads, a.s.T, D, a.group, kRows / a.group) || !make_cache_map(&mk, k, a.c, box, 1) || !make_cache_map(&mv, v, a.c, box, 1))
        return cudaErrorInvalidValue;
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(attn_tiles_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)C::kSmem);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    const int R = kRows / a.group * a.group;
    a.tiles = (int)(((long long)a.s.max_new * a.group + R - 1) / R);
    const long long P = most_shares(a, kKeys, kItemCost, kMinTiles, sms);
    return launch_pdl(attn_tiles_kernel<D>, dim3((unsigned)P), dim3(C::kThreads), C::kSmem, stream, true, mq, mk, mv, a,
                      box);
}

}  // namespace

size_t attn_tiles_workspace(int D) { return (size_t)kMaxSms * 2 * 4 * part_floats(D); }

cudaError_t launch_attn_tiles(const AttnArgs& a, const void* k, const void* v, int sms, cudaStream_t stream) {
    switch (a.c.head_dim) {
        case 64: return launch<64>(a, k, v, sms, stream);
        case 128: return launch<128>(a, k, v, sms, stream);
        default: return launch<256>(a, k, v, sms, stream);
    }
}

cudaError_t read_attn_tiles_device_error(int* code) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_attn_tiles_error, sizeof(int));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_attn_tiles_error, &zero, sizeof(int));
}

}  // namespace tern
