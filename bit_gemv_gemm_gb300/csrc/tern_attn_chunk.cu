// tern_attn_chunk.cu -- attention of many query rows a key head (prompt chunks,
// more than one row tile, heads of 64 and 128) on the tcgen05 tensor cores.
//
// A row tile is 128 packed rows (128 / group tokens, every head of the group),
// so one K and V tile serves all the heads that share it.  A CTA takes a row tile
// through a run of 128-key tiles:
//   * a TMA warp brings Q and K, another V, in chunks of 64 head values x 128
//     keys, through one ring.  A copy takes a warp about 110 clocks to issue and a
//     page id some 700 to look up, hence two warps, and ids fetched 32 boxes ahead;
//   * one thread issues S = Q K^T (both operands in shared memory, K-major),
//     another O += P V (P in tensor memory, V MN-major).  Issuing is nearly
//     synchronous (a wait or a commit between products costs the thread about
//     150 and 57 clocks that its own products do not cover: 110 clocks a 64-clock
//     product from one thread), so each covers the other's;
//   * S has three buffers, so QK runs ahead, and two softmax warpgroups take the
//     tiles in turn, one thread a row: read S, exponentiate, write P as bf16 over
//     S's own columns.
// The two warpgroups share a row's maximum in use: each hands it on as soon as
// it has looked at its tile's scores, well before it has exponentiated them.  It
// only moves when a score passes it by 2^8 (then O is rescaled, after the product
// before has been added), so P and the sums stay below 2^8 of their largest term.
// Each warpgroup keeps its own sum, in fp32; they meet at the item's end.
// Two neighbouring row tiles are one item, taken by a pair of CTAs that start
// together and go through the same key tiles at the same pace, each with its own
// loads and waits: what one has just read is in L2 for the other.  A pair is
// launched as a cluster, which puts it on neighbouring SMs, and shares nothing
// else (single CTAs with a row tile each, 512 tokens over 32k keys 226 us and whole
// prompts 188; pairs without the cluster 213 and 192; pairs 214 and 148).
// 512 tokens over 32k keys, 32 heads of 128: 214 us, 1.27 PFLOP/s, 10 TB/s from L2
// (195 us, 1.39 PFLOP/s, where three inputs take turns).  TMA multicast of each
// half to both CTAs took 202 (191), but a library that programs of several GPUs
// load has no multicast loads.  The tiles kernel's two streams take 243 there and
// 176 for the prompts.
// Slots past a sequence's last key and before its windows may hold anything: scores are masked before
// the exponential and V's rows are zeroed in shared memory by the TMA warp
// before the tile is handed on (a row of P is 0 there, and 0 * NaN is not).
// Work is shared out as in the rows kernel: equal contiguous shares of all
// (sequence, pair of row tiles, key head) items' 128-key tiles, a share a pair; parts
// meet in the workspace, and the warp that counts last for its 32 rows adds them in
// order.
#include "tern_attn.cuh"

namespace tern {
namespace {

using namespace sm100;

__device__ int g_attn_chunk_error;

constexpr int kKeys = 128, kRows = kTileRows;
constexpr int kChunk = 64 * kKeys * 2;      // 16 KB: 64 head values of 128 keys (or rows)
// key tiles' time that an item costs besides its own (four prompts of up to 4000
// tokens, whose items are of unlike length: 155, 148, 151 us with 4, 5, 7; four of up
// to 2000, heads of 128: 76, 77, 80)
constexpr int kItemCost = 5;
constexpr int kMinTiles = 4;                // key tiles a share holds at least
constexpr int kSoftWarps = 8;
// a third warpgroup (two TMA and two MMA warps) gives registers to the softmax
// warps, which hold a row of S each: 256 x 208 + 128 x 88 = 384 x 168, what the
// CTA was launched with
constexpr int kThreads = 384;

template <int D>
struct Cfg {
    static constexpr int NC = D / 64;                       // chunks of a K, V or Q tile
    static constexpr int kTile = NC * kChunk;
    static constexpr int kSlots = D == 64 ? 12 : 6;         // K and V tiles, in turn
    // K and V have a warp each that waits for its own slots alone: a slot has to be always the same one's
    static_assert(kSlots % 2 == 0, "K's slots and V's");
    static constexpr int NB = 3;                            // buffers of S
    static constexpr uint32_t kS = 0, kO = 128 * NB;        // tensor memory: S (and P) at 128 b, then O
    static constexpr size_t kSmemRing = (size_t)kTile;
    static constexpr size_t kSmemBar = kSmemRing + (size_t)kSlots * kTile;
    static constexpr int kBars = 2 * kSlots + 2 + 3 * NB + 1 + 8 + 1 + 1 + 2;
    static constexpr size_t kSmemMisc = (kSmemBar + kBars * 8 + 15) / 16 * 16;
    static constexpr size_t kSmemM = kSmemMisc + 256;       // a row's maximum in use, and a warpgroup's sums
    static constexpr size_t kSmem = kSmemM + 2 * kRows * 4 + 1024;
    static_assert(kSmem <= 232448, "shared memory of one CTA");
};
constexpr uint32_t kIdescQK = idesc_bf16_f32(kRows, kKeys);

// Where one role is in a ring of N slots.
template <int N>
struct Ring {
    uint32_t slot, phase = 0;
    __device__ __forceinline__ explicit Ring(uint32_t first) : slot(first) {}
    __device__ __forceinline__ void skip(uint32_t n) {
        slot += n;
        if (slot >= N) slot -= N, phase ^= 1u;
    }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_chunk_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                  const __grid_constant__ CUtensorMap tmap_v, const AttnArgs a, const int box_rows) {
    using C = Cfg<D>;
    constexpr int NC = C::NC, NB = C::NB, kSlots = C::kSlots, kTile = C::kTile;
    extern __shared__ __align__(1024) unsigned char smem_dyn[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem), bar0 = sbase + (uint32_t)C::kSmemBar;
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    enum { Q_FULL = 2 * kSlots, Q_EMPTY, S_FULL, S_EMPTY = S_FULL + NB, P_FULL = S_EMPTY + NB, O_EMPTY = P_FULL + NB, HAND, MERGE = HAND + 8, TAIL, DRAIN };   // DRAIN: two
    static_assert(DRAIN + 2 == C::kBars, "barriers");
    long long* sm_scan = reinterpret_cast<long long*>(smem + C::kSmemMisc);   // [8 + warps]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm_scan + 8 + kThreads / 32);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    float* sm_m = reinterpret_cast<float*>(smem + C::kSmemM);
    float* sm_l = sm_m + kRows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kBars; ++i) {
            int count = 1;
            if ((i >= P_FULL && i < P_FULL + NB) || i == O_EMPTY || i == MERGE) count = 4;
            mbar_init(bar(i), count);
        }
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmap_q);
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
    }
    if (warp == kSoftWarps + 1) {
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
    const int R = 2 * tile_rows;                       // rows of an item: this CTA's row tile and its neighbour's
    const int rank = (int)blockIdx.x & 1, share = (int)blockIdx.x / 2;
    const RowTileExtent<kKeys, kItemCost> extent{R, a.group, a.window};
    int P;
    long long total, w0, w1;
    Item t;
    const bool busy = find_share<kThreads>(a.s, a.c, extent, a.tiles, kMinTiles, share, (int)gridDim.x / 2,
                                           sm_scan, &g_attn_chunk_error, total, P, w0, w1, t);
    auto fail = [&] {
        if (!*abort_flag) {
            *abort_flag = 1;
            report_device_error(&g_attn_chunk_error, TERN_DEVERR_ATTN_WAIT);
        }
    };
    auto wait = [&](uint32_t b, uint32_t parity) { return mbar_wait_bounded(b, parity, abort_flag, kAttnWaitNs); };

    if (!busy) {
        // no share: straight to the end
    } else if (warp >= kSoftWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == kSoftWarps || warp == kSoftWarps + 3) {
            // ------------------------------ TMA: Q and K, or V ------------------------------
            const bool is_v = warp != kSoftWarps;
            const CUtensorMap* map = is_v ? &tmap_v : &tmap_k;
            uint32_t n = 0, used = 0, tails = 0;   // key tiles, items, tiles with rows to zero so far
            bool ok = true;
            const int boxes = kKeys / box_rows;                        // of a chunk
            const int c = lane / boxes, box = lane - c * boxes;        // this lane's piece of a tile
            const uint32_t piece = (uint32_t)(c * kChunk + box * box_rows * 128);   // in its slot
            const bool page_boxes = box_rows == a.c.page_size;         // a box is a whole page
            Ring<kSlots> ring(is_v ? 1 : 0);   // K(0), V(0), K(1), ...
            for (long long w = w0; w < w1 && ok;) {
                const Segment seg = segment_of(extent, t, w, w1);
                // (an item's second row tile may be absent)
                const int nt = t.rows > rank * tile_rows ? seg.n : 0, key0 = seg.first * kKeys;
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
                        const int tok = t.q.q0 + (t.rt * R + rank * tile_rows) / a.group;
                        for (int x = 0; x < NC; ++x)
                            tma_load_q(sbase + (uint32_t)(x * kChunk), &tmap_q, t.hk * a.group, tok, x, bar(Q_FULL));
                    }
                }
                for (int j = 0; j < nt; ++j, ++n, ring.skip(2)) {
                    if (((j * boxes) & 31) == 0) {
                        ids = checked_page(ahead, a.c.pages, &g_attn_chunk_error);
                        ahead = raw_id(j * boxes + 32 + lane);
                    }
                    const int page = __shfl_sync(0xffffffffu, ids, (j * boxes + box) & 31);
                    const int k0 = key0 + j * kKeys, k = k0 + box * box_rows;
                    const int slot = page_boxes ? 0 : (unsigned)k % (unsigned)a.c.page_size;
                    bool use = c < NC, part = false, unread = false;
                    uint32_t bytes = kKeys * 128u;   // a chunk's
                    const VRows rows(k0, kKeys, box_rows, t.j0, t.q.len);
                    if (k0 < t.j0 || k0 + kKeys > t.q.len) {
                        // boxes that hold no key of these rows are not read; V's rows there count as 0
                        use = use && k < t.q.len && k + box_rows > t.j0;
                        bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, use) & ((1u << boxes) - 1u)) * box_rows * 128u;
                        part = is_v && rows.inside();
                        unread = is_v && (rows.front > 0 || rows.back_box < kKeys);
                    }
                    const uint32_t full = part ? bar(TAIL) : bar((int)ring.slot);
                    unsigned char* chunks = smem + C::kSmemRing + ring.slot * (uint32_t)kTile;
                    if (!__all_sync(0xffffffffu, wait(bar(kSlots + (int)ring.slot), ring.phase ^ 1u))) {
                        ok = false;
                        break;
                    }
                    if (unread) {
                        for (int x = 0; x < NC; ++x) {
                            zero_rows(chunks + x * kChunk, 0, rows.front);
                            zero_rows(chunks + x * kChunk, rows.back_box, kKeys);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (lane == 0) mbar_arrive_expect_tx(full, bytes * NC);
                    __syncwarp();
                    if (use) tma_load_cache(smem_u32(chunks) + piece, map, slot, c, t.hk, page, full);
                    if (part) {
                        if (!__all_sync(0xffffffffu, wait(full, tails & 1u))) {
                            ok = false;
                            break;
                        }
                        ++tails;
                        for (int x = 0; x < NC; ++x) rows.zero_inside(chunks + x * kChunk);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar((int)ring.slot));
                    }
                }
                w = seg.we;
                if (w < w1) next_item(a.s, a.c, extent, a.tiles, t, &g_attn_chunk_error);
            }
            if (!ok && lane == 0) {
                fail();
                // copies in flight land before the CTA goes away
                constexpr uint32_t kTiles = kSlots / 2;
                for (uint32_t x = n < kTiles ? 0 : n - kTiles; x <= n; ++x) {
                    const uint32_t r = 2 * x + (is_v ? 1 : 0);
                    (void)mbar_wait_drain(bar((int)(r % kSlots)), (r / kSlots) & 1u, 20000000ull);
                }
                if (used) (void)mbar_wait_drain(bar(Q_FULL), (used - 1u) & 1u, 20000000ull);
                if (is_v) (void)mbar_wait_drain(bar(TAIL), tails & 1u, 20000000ull);
            }
            __syncwarp();
        } else {
            // ------------------------------ MMA: QK, or PV ------------------------------
            if (lane == 0) {
                const bool is_pv = warp != kSoftWarps + 1;
                constexpr uint32_t kIdescPV = idesc_bf16_f32(kRows, D) | kIdescBMnMajor;
                uint32_t used = 0;
                Ring<kSlots> ring(is_pv ? 1 : 0);   // the next key tile's slot
                Ring<NB> sb(0);                     // ... and its S
                // between one tile's products and the next this thread spends some 600 of a tile's 1600
                // clocks, waits that are over and commits; slots are counted along, not divided out, and
                // both barriers are asked at once (heads of 64, 512 tokens over 32k: 173 -> 168 us)
                const uint64_t qd0 = smem_desc_k_sw128(sbase), kd0 = smem_desc_k_sw128(sbase + (uint32_t)C::kSmemRing);
                const uint64_t vd0 = smem_desc_mn_sw128(sbase + (uint32_t)C::kSmemRing, kChunk);
                bool ok = true, issued = false;
                auto need = [&](uint32_t b, uint32_t parity) {
                    if (ok && !wait(b, parity)) ok = false;
                    return ok;
                };
                auto need2 = [&](uint32_t b, uint32_t parity, uint32_t b2, uint32_t parity2) {
                    const bool r = mbar_try_wait(b, parity), r2 = mbar_try_wait(b2, parity2);
                    if (!r) need(b, parity);
                    if (!r2) need(b2, parity2);
                    return ok;
                };
                for (long long w = w0; w < w1 && ok;) {
                    const Segment seg = segment_of(extent, t, w, w1);
                    if (seg.n > 0 && t.rows > rank * tile_rows) {
                        if (!is_pv) need(bar(Q_FULL), used & 1u);
                        for (int j = 0; j < seg.n && ok; ++j, ring.skip(2), sb.skip(1)) {
                            const uint32_t s_tmem = tmem + C::kS + 128u * sb.slot, o_tmem = tmem + C::kO;
                            const uint64_t at = (uint64_t)(ring.slot * (uint32_t)(kTile >> 4));
                            if (!is_pv) {
                                // the P that was over this S has been used
                                if (!need2(bar((int)ring.slot), ring.phase, bar(S_EMPTY + (int)sb.slot), sb.phase ^ 1u)) break;
                                tc_fence_after();
#pragma unroll
                                for (int c = 0; c < NC; ++c)
#pragma unroll
                                    for (int kk = 0; kk < 4; ++kk)
                                        mma_f16_ss(s_tmem, qd0 + (uint64_t)(c * (kChunk >> 4) + 2 * kk),
                                                   kd0 + at + (uint64_t)(c * (kChunk >> 4) + 2 * kk), kIdescQK,
                                                   (c | kk) ? 1u : 0u);
                                mma_commit(bar(S_FULL + (int)sb.slot));
                            } else {
                                if (!need2(bar((int)ring.slot), ring.phase, bar(P_FULL + (int)sb.slot), sb.phase)) break;
                                if (j == 0 && !need(bar(O_EMPTY), (used & 1u) ^ 1u)) break;   // the previous item's output has been read
                                tc_fence_after();
#pragma unroll
                                for (int kk = 0; kk < kKeys / 16; ++kk)
                                    mma_f16_ts(o_tmem, s_tmem + 8u * kk, vd0 + at + (uint64_t)(kk * (2048 >> 4)), kIdescPV,
                                               (j || kk) ? 1u : 0u);
                                mma_commit(bar(S_EMPTY + (int)sb.slot));
                            }
                            mma_commit(bar(kSlots + (int)ring.slot));
                            issued = true;
                        }
                        if (ok) {
                            if (!is_pv) mma_commit(bar(Q_EMPTY));
                            ++used;
                        }
                    }
                    w = seg.we;
                    if (w < w1) next_item(a.s, a.c, extent, a.tiles, t, &g_attn_chunk_error);
                }
                if (!ok) {
                    fail();
                    if (issued) {
                        mma_commit(bar(DRAIN + (is_pv ? 1 : 0)));
                        (void)mbar_wait_drain(bar(DRAIN + (is_pv ? 1 : 0)), 0u, 100000000ull);
                    }
                }
            }
            __syncwarp();
        }
    } else {
        // ------------------------------ softmax, output ------------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int wg = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t to = tmem + lanes + C::kO;
        uint32_t first_tile = 0, merges = 0;   // key tiles and merged items so far
        const bool flip = a.scale_log2 < 0.0f;
        const float scale = fabsf(a.scale_log2);
        bool ok = true;
        auto all_wait = [&](int i, uint32_t parity) {
            if (ok && !__all_sync(0xffffffffu, wait(bar(i), parity))) ok = false;
            return ok;
        };
        // the maximum in use after key tile n, from the warpgroup that took it
        auto handed = [&](uint32_t n) { return all_wait(HAND + (int)(n & 1u) * 4 + quad, (n >> 1) & 1u); };
        for (long long w = w0; w < w1 && ok;) {
            const Segment seg = segment_of(extent, t, w, w1);
            const int nt = seg.n, rows = min(tile_rows, t.rows - rank * tile_rows);   // of this CTA's row tile
            if (!seg.skip && rows > 0) {
                const int r = t.rt * R + rank * tile_rows + row;   // packed row of the sequence
                const bool live = row < rows, idle = quad * 32 >= rows;
                const int p = t.q.len - t.q.n + r / a.group;
                const int hi = live ? p : -1, lo = a.window > 0 ? p - a.window : -1;
                const int p_lo = t.q.len - t.q.n + (t.rt * R + rank * tile_rows) / a.group;
                const int p_hi = t.q.len - t.q.n + (t.rt * R + rank * tile_rows + rows - 1) / a.group;
                const int key0 = seg.first * kKeys;
                float m = -INFINITY, l = 0.0f;   // l is relative to m, the maximum in use when this warpgroup last looked
                for (int j = 0; j < nt && ok; ++j) {
                    const uint32_t n = first_tile + (uint32_t)j, buf = n % NB, ph = (n / NB) & 1u;
                    if ((int)(n & 1u) != wg) continue;
                    if (!all_wait(S_FULL + (int)buf, ph)) break;
                    if (idle) {
                        if (n > 0 && !handed(n - 1)) break;
                        if (lane == 0) {
                            mbar_arrive(bar(HAND + wg * 4 + quad));
                            mbar_arrive(bar(P_FULL + (int)buf));
                        }
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
                    // (the tile before, of the last item too: the hand-overs stay in step)
                    if (n > 0 && !handed(n - 1)) break;
                    float now = j > 0 ? sm_m[row] : -INFINITY;
                    // (rows of no query of the sequence hold what the copies left: they have no vote)
                    const bool move = __any_sync(0xffffffffu, live && (top - now) * scale > 8.0f);
                    const float before = now;
                    if (move) now = fmaxf(now, top);
                    sm_m[row] = now;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(HAND + wg * 4 + quad));
                    l *= m == -INFINITY ? 0.0f : exp2_fast((m - now) * scale);
                    m = now;
                    if (move && j > 0) {
                        // the product before has been added
                        if (!all_wait(S_EMPTY + (int)((n - 1u) % NB), ((n - 1u) / NB) & 1u)) break;
                        tc_fence_after();
                        const float f = before == -INFINITY ? 0.0f : exp2_fast((before - now) * scale);
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
                // the warpgroup of the last tile writes the rows (the first one, where there is no tile)
                const uint32_t last = first_tile + (uint32_t)nt - 1u;
                const bool writer = nt > 0 ? (int)(last & 1u) == wg : wg == 0;
                if (nt > 1) {
                    if (!writer) {
                        // (idle warps wait, too: one that ran on into the next item would count itself in for this one)
                        if (!handed(last)) break;
                        // (a sum that is not a number stays one, whatever its weight)
                        const float top = sm_m[row];
                        if (!idle) sm_l[row] = l * (top == -INFINITY ? 1.0f : exp2_fast((m - top) * scale));
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(MERGE));
                    } else {
                        if (!all_wait(MERGE, merges & 1u)) break;
                        l += sm_l[row];
                    }
                    ++merges;
                }
                if (writer) {
                    if (nt > 0) {
                        if (!all_wait(S_EMPTY + (int)(last % NB), (last / NB) & 1u)) break;
                        tc_fence_after();
                    }
                    const float m2 = m * scale;   // -inf stays
                    const long long orow = (long long)(t.q.q0 + r / a.group) * a.q_heads + t.hk * a.group + r % a.group;
                    constexpr size_t kPart = 2 * part_floats(D);   // both row tiles
                    float* part = a.partial + (size_t)(2 * share + (w == w0 ? 0 : 1)) * kPart + rank * part_floats(D);
                    if (!idle)
                        emit_row<D>(a, seg.whole, part, row, live, orow, m2, l, [&](int c, uint32_t (&o)[32]) {
                            if (nt > 0) {
                                tmem_ld_x32(to + c, o);
                                tmem_ld_wait();
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = 0u;
                            }
                        });
                    if (nt > 0) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(O_EMPTY));
                    }
                    if (!seg.whole && !idle &&
                        count_part<kItemCost>(t, a.counters + 4 * rank + quad, total, P))
                        add_parts<D, kItemCost>(a, t, a.partial + rank * part_floats(D), kPart, row, live, orow, total, P, 0,
                                                D);
                }
                first_tile += (uint32_t)nt;
            }
            w = seg.we;
            if (w < w1) next_item(a.s, a.c, extent, a.tiles, t, &g_attn_chunk_error);
        }
        if (!ok && lane == 0) fail();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kSoftWarps + 1) {
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
    if (!make_q_map(&mq, a.q, a.q_stride, a.q_heads, a.s.T, D, a.group, kRows / a.group) ||
        !make_cache_map(&mk, k, a.c, box, 1) || !make_cache_map(&mv, v, a.c, box, 1))
        return cudaErrorInvalidValue;
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(attn_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)C::kSmem);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    const int R = 2 * (kRows / a.group * a.group);
    a.tiles = (int)(((long long)a.s.max_new * a.group + R - 1) / R);
    const long long P = most_shares(a, kKeys, kItemCost, kMinTiles, sms / 2);
    return launch_pdl_clusters(attn_chunk_kernel<D>, 2, dim3((unsigned)(2 * P)), dim3(kThreads), C::kSmem, stream, mq, mk,
                               mv, a, box);
}

}  // namespace

size_t attn_chunk_workspace(int D) { return (size_t)kMaxSms * 2 * 4 * part_floats(D); }

cudaError_t launch_attn_chunk(const AttnArgs& a, const void* k, const void* v, int sms, cudaStream_t stream) {
    switch (a.c.head_dim) {
        case 64: return launch<64>(a, k, v, sms, stream);
        default: return launch<128>(a, k, v, sms, stream);
    }
}

cudaError_t read_attn_chunk_device_error(int* code) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_attn_chunk_error, sizeof(int));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_attn_chunk_error, &zero, sizeof(int));
}

}  // namespace tern
