// tern_attn_rows.cu -- attention of few query rows a key head (decode, verify):
// bound by reading the cache once.
//
// One item is up to 16 packed rows (token, head of the group) of one sequence
// and key head; its keys are read in strips of 16.  All strips of all
// items are cut into one equal contiguous share a CTA (no CTA idles behind a
// long sequence), two CTAs an SM.  In a CTA every warp takes every fourth strip of a
// segment for itself: its lane 0 fetches the strip's K and V by TMA into the
// warp's own ring (three strips of 8 KB at D = 128: 192 KB in flight an SM),
// so warps never wait for one another inside a segment.  Per strip a warp
// does S = Q K^T and O += P V with mma.sync (m16n8k16, bf16 in, fp32 out)
// with a running maximum that only moves when a score passes it by 2^8: the
// sums stay below 2^8 times their largest term, far inside fp32.
// At a segment's end the four warps' (O, m, l) meet in shared memory in a
// fixed order.  A segment that is the whole item is written out; a part goes to
// the workspace, and the CTA that counts itself last into the item's counter
// adds the parts in their order, so results do not depend on which CTA is last.
// 32 sequences of up to 16k keys, 8 key heads of 128: 207 us, 6.4 TB/s; one token
// over 500 keys is a chain of dependent reads, some 8 us.
#include <algorithm>

#include "tern_attn.cuh"

namespace tern {
namespace {

__device__ int g_attn_rows_error;

constexpr int kWarps = 4, kThreads = kWarps * 32, kStrip = 16;
constexpr int R = 16;                          // query rows of an item
constexpr int kItemCost = 4;                   // strips' time that an item costs besides its own
constexpr int kMinUnits = 2 * kWarps;         // strips a share holds at least (two a warp)

template <int D>
struct Cfg {
    static constexpr int kStage = kStrip * D * 4;                 // K and V of one strip
    static constexpr int kStages = D == 64 ? 6 : 3;
    static constexpr int kRing = kStages * kStage;                // one warp's
    static constexpr int kQ = R * D * 2;
    static constexpr int kCtas = D == 256 ? 1 : 2;                // an SM
    static constexpr int kPart = R * (D + 2);                     // floats of a part
    static constexpr size_t kSmemQ = (size_t)kWarps * kRing;
    static constexpr size_t kSmemBar = kSmemQ + kQ;
    static constexpr size_t kSmemStat = kSmemBar + kWarps * kStages * 8;
    static constexpr size_t kSmemMisc = kSmemStat + (size_t)kWarps * R * 8;
    static constexpr size_t kSmem = kSmemMisc + 128 + 1024;       // + alignment slack
    static_assert(kRing >= R * D * 4, "a warp's rows are merged through its ring");
};

__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <int D>
__global__ void __launch_bounds__(kThreads, Cfg<D>::kCtas)
attn_rows_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                 const AttnArgs a) {
    using namespace sm100;
    using C = Cfg<D>;
    extern __shared__ __align__(1024) unsigned char smem_dyn[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = sbase + (uint32_t)(warp * C::kRing), qs = sbase + (uint32_t)C::kSmemQ;
    const uint32_t bars = sbase + (uint32_t)C::kSmemBar + (uint32_t)(warp * C::kStages * 8);
    float* sm_m = reinterpret_cast<float*>(smem + C::kSmemStat);             // [warp][R]
    float* sm_l = sm_m + kWarps * R;
    long long* sm_scan = reinterpret_cast<long long*>(smem + C::kSmemMisc);   // [8 + kWarps]
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm_scan + 8 + kWarps);
    int* sm_last = reinterpret_cast<int*>(sm_scan + 8 + kWarps) + 1;

    if (lane == 0) {
        for (int s = 0; s < C::kStages; ++s) mbar_init(bars + 8u * s, 1);
        fence_barrier_init();
        if (warp == 0) {
            *abort_flag = 0;
            tma_prefetch_desc(&tmap_k);
            tma_prefetch_desc(&tmap_v);
        }
    }
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();

    const int cta = blockIdx.x;
    int P;
    long long total, w0, w1;
    Item t;
    const RowTileExtent<kStrip, kItemCost> extent{R, a.group, a.window};
    if (!find_share<kThreads>(a.s, a.c, extent, a.tiles, kMinUnits, (int)blockIdx.x, (int)gridDim.x, sm_scan, &g_attn_rows_error, total, P, w0, w1, t))
        return;

    uint32_t it = 0;   // strips this warp has fetched and used, over all segments
    for (long long w = w0; w < w1;) {
        // ---- one segment of the item ----
        const Seq q = t.q;
        const int rows = t.rows, units = t.units, j0 = t.j0, j1 = t.j1, r0 = t.rt * R, hk = t.hk, b = t.b;
        const Segment seg = segment_of(extent, t, w, w1);
        const long long at = t.at, we = seg.we;
        const int first = seg.first, strips = seg.n;
        if (!seg.skip) {
        const int my = strips > warp ? (strips - warp + kWarps - 1) / kWarps : 0;
        // page ids: lane i holds the one of this warp's strip i of the current 32
        const int* trow = a.s.table + (long long)b * a.s.width;
        int ids = 0;
        auto fetch_ids = [&](int base) {
            const int k = base + lane;
            ids = 0;
            if (k < my) ids = checked_page(trow[(unsigned)((first + warp + kWarps * k) * kStrip) / (unsigned)a.c.page_size], a.c.pages, &g_attn_rows_error);
        };
        auto issue = [&](int k) {   // strip k of this warp, into slot (it + k) mod stages
            const int page = __shfl_sync(0xffffffffu, ids, k & 31);
            if (lane == 0) {
                const uint32_t s = (it + (uint32_t)k) % C::kStages;
                const int slot = (unsigned)((first + warp + kWarps * k) * kStrip) % (unsigned)a.c.page_size;
                mbar_arrive_expect_tx(bars + 8u * s, C::kStage);
                tma_load_cache(ring + s * C::kStage, &tmap_k, slot, 0, hk, page, bars + 8u * s);
                tma_load_cache(ring + s * C::kStage + C::kStage / 2, &tmap_v, slot, 0, hk, page, bars + 8u * s);
            }
        };
        fetch_ids(0);
        for (int k = 0; k < C::kStages && k < my; ++k) issue(k);
        // the rows of Q, in the layout of the A fragments' loads
        for (int i = threadIdx.x; i < R * (D / 8); i += kThreads) {
            const int r = i / (D / 8), c = i % (D / 8);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < rows) {
                const int tok = (r0 + r) / a.group, g = (r0 + r) % a.group;
                v = *reinterpret_cast<const uint4*>(a.q + (long long)(q.q0 + tok) * a.q_stride +
                                                    (long long)(hk * a.group + g) * D + c * 8);
            }
            *reinterpret_cast<uint4*>(smem + C::kSmemQ + (c >> 3) * (R * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
        }
        // the keys that each of this thread's rows sees: (lo, hi]
        int hi[2], lo[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = i * 8 + (lane >> 2);
            const int p = q.len - q.n + (r0 + min(r, rows - 1)) / a.group;
            hi[i] = r < rows ? p : -1;
            lo[i] = a.window > 0 ? p - a.window : -1;
        }
        const int p_lo = q.len - q.n + r0 / a.group, p_hi = q.len - q.n + (r0 + rows - 1) / a.group;
        __syncthreads();

        float o[D / 8][4] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {};
        for (int k = 0; k < my; ++k) {
            const uint32_t slot = (it + (uint32_t)k) % C::kStages, phase = ((it + (uint32_t)k) / C::kStages) & 1u;
            const int key0 = (first + warp + kWarps * k) * kStrip;
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(bars + 8u * slot, phase, abort_flag, kAttnWaitNs))) {
                if (!*abort_flag) {
                    *abort_flag = 1;
                    if (lane == 0) report_device_error(&g_attn_rows_error, TERN_DEVERR_ATTN_WAIT);
                }
                if (lane == 0)   // the copies in flight land before the CTA goes away
                    for (int x = k; x < my && x < k + C::kStages; ++x)
                        (void)mbar_wait_drain(bars + 8u * ((it + (uint32_t)x) % C::kStages),
                                              ((it + (uint32_t)x) / C::kStages) & 1u, 100000000ull);
                break;
            }
            const uint32_t ks = ring + slot * C::kStage, vs = ks + C::kStage / 2;
            // S = Q K^T
            float s[2][4] = {};
            const int mi = lane >> 3, l7 = lane & 7;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t kb[4], qa[4];
                const int krow = (mi >> 1) * 8 + l7, kc = (kk & 3) * 2 + (mi & 1);
                ldsm4(kb, ks + (kk >> 2) * (kStrip * 128) + krow * 128 + ((kc ^ l7) << 4));
                const int qrow = (mi & 1) * 8 + l7, qc = (kk & 3) * 2 + (mi >> 1);
                ldsm4(qa, qs + (kk >> 2) * (R * 128) + qrow * 128 + ((qc ^ l7) << 4));
                mma_bf16(s[0], qa, kb[0], kb[1]);
                mma_bf16(s[1], qa, kb[2], kb[3]);
            }
            // scores in powers of two; a strip that some row does not see whole is masked
            const bool masked = key0 + kStrip - 1 > p_lo || (a.window > 0 && key0 <= p_hi - a.window);
            bool grow = false;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x = s[n][e] * a.scale_log2;
                    if (masked) {
                        const int key = key0 + n * 8 + (lane & 3) * 2 + (e & 1);
                        if (key > hi[e >> 1] || key <= lo[e >> 1]) x = -INFINITY;
                    }
                    s[n][e] = x;
                    grow |= x > m[e >> 1] + 8.0f;
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                    if (x > m[h]) {
                        const float f = exp2_fast(m[h] - x);   // 0 from -inf
                        m[h] = x;
                        l[h] *= f;
#pragma unroll
                        for (int n = 0; n < D / 8; ++n) {
                            o[n][2 * h] *= f;
                            o[n][2 * h + 1] *= f;
                        }
                    }
                }
            }
            uint32_t pa[4];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // a row that has seen nothing keeps m = -inf: its probabilities are 0
                    const float mm = m[h] == -INFINITY ? 0.0f : m[h];
                    const float x = exp2_fast(s[n][2 * h] - mm), y = exp2_fast(s[n][2 * h + 1] - mm);
                    l[h] += x + y;
                    pa[2 * n + h] = pack_bf16(x, y);
                }
            // slots before the first visible key and past the last may hold anything: their V counts as 0
            uint32_t z0 = 0xffffffffu, z1 = 0xffffffffu;
            if (key0 + kStrip > j1 || key0 < j0) {
                const int k0 = key0 + (lane & 3) * 2;
                auto seen = [&](int k) { return k >= j0 && k < j1; };
                z0 = (seen(k0) ? 0xffffu : 0u) | (seen(k0 + 1) ? 0xffff0000u : 0u);
                z1 = (seen(k0 + 8) ? 0xffffu : 0u) | (seen(k0 + 9) ? 0xffff0000u : 0u);
            }
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
                uint32_t vb[4];
                const int vrow = (mi & 1) * 8 + l7, vc = (n & 3) * 2 + (mi >> 1);
                ldsm4_t(vb, vs + (n >> 2) * (kStrip * 128) + vrow * 128 + ((vc ^ l7) << 4));
                vb[0] &= z0;
                vb[1] &= z1;
                vb[2] &= z0;
                vb[3] &= z1;
                mma_bf16(o[2 * n], pa, vb[0], vb[1]);
                mma_bf16(o[2 * n + 1], pa, vb[2], vb[3]);
            }
            __syncwarp();
            if (((k + C::kStages) & 31) == 0) fetch_ids(k + C::kStages);
            if (k + C::kStages < my) issue(k + C::kStages);
        }
        it += (uint32_t)my;

        // ---- the four warps' rows meet ----
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float x = l[h];
            x += __shfl_xor_sync(0xffffffffu, x, 1);
            x += __shfl_xor_sync(0xffffffffu, x, 2);
            const int r = h * 8 + (lane >> 2);
            if ((lane & 3) == 0) {
                sm_m[warp * R + r] = m[h];
                sm_l[warp * R + r] = x;
            }
            // [R][D] fp32 over the warp's own ring; columns rotated by row against bank conflicts
            float* mo = reinterpret_cast<float*>(smem + warp * C::kRing) + r * D;
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
                *reinterpret_cast<float2*>(mo + ((n * 8 + (lane & 3) * 2 + r * 8) & (D - 1))) =
                    make_float2(o[n][2 * h], o[n][2 * h + 1]);
        }
        __syncthreads();
        if (*abort_flag) return;

        const bool whole = seg.whole;
        float* part = a.partial + (size_t)(2 * cta + (w == w0 ? 0 : 1)) * C::kPart;
        auto store_row = [&](int r, int c, const float (&y)[4], float mm, float ll) {
            // columns c .. c + 3 of row r, divided by the sum
            const int tok = (r0 + r) / a.group, g = (r0 + r) % a.group;
            const long long row = (long long)(q.q0 + tok) * a.q_heads + hk * a.group + g;
            const float inv = inverse_sum(ll);
            *reinterpret_cast<uint2*>(a.out + row * D + c) =
                make_uint2(pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv));
            if (c == 0 && a.lse) a.lse[row] = lse_of(mm, ll);
        };
        for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = i % (D / 4) * 4;
            float mm = -INFINITY, ll = 0.0f, y[4] = {};
#pragma unroll
            for (int x = 0; x < kWarps; ++x) mm = fmaxf(mm, sm_m[x * R + r]);
#pragma unroll
            for (int x = 0; x < kWarps; ++x) {
                const float f = sm_m[x * R + r] == -INFINITY ? 0.0f : exp2_fast(sm_m[x * R + r] - mm);
                ll += sm_l[x * R + r] * f;
                const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + x * C::kRing) +
                                                                  r * D + ((c + r * 8) & (D - 1)));
                y[0] += v.x * f;
                y[1] += v.y * f;
                y[2] += v.z * f;
                y[3] += v.w * f;
            }
            if (whole) {
                store_row(r, c, y, mm, ll);
            } else {
                __stcg(reinterpret_cast<float4*>(part + r * D + c), make_float4(y[0], y[1], y[2], y[3]));
                if (c == 0) __stcg(reinterpret_cast<float2*>(part + R * D + 2 * r), make_float2(mm, ll));
            }
        }
        if (!whole) {
            // count into the item's counter (its first CTA's); the last one adds the parts
            const int c_lo = unit_owner(total, P, at + kItemCost), c_hi = unit_owner(total, P, at + units - 1);
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) *sm_last = atomicInc(a.counters + c_lo, (unsigned)(c_hi - c_lo)) == (unsigned)(c_hi - c_lo);
            __syncthreads();
            if (*sm_last) {
                __threadfence();
                // an item's first CTA may have begun before it: the part is then in its second slot
                const int late = unit_begin(total, P, c_lo) >= at ? 0 : 1;
                for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
                    const int r = i / (D / 4), c = i % (D / 4) * 4;
                    float mm = -INFINITY, ll = 0.0f, y[4] = {};
                    // eight parts' loads in flight together; past the last, its own again with no weight
                    for (int x0 = c_lo; x0 <= c_hi; x0 += 8) {
                        float2 st[8];
                        float4 v[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int x = min(x0 + k, c_hi);
                            const float* px = a.partial + (size_t)(2 * x + (x == c_lo ? late : 0)) * C::kPart;
                            st[k] = __ldcg(reinterpret_cast<const float2*>(px + R * D + 2 * r));
                            v[k] = __ldcg(reinterpret_cast<const float4*>(px + r * D + c));
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float mn = fmaxf(mm, st[k].x), base = mn == -INFINITY ? 0.0f : mn;
                            const float f0 = exp2_fast(mm - base), f1 = x0 + k <= c_hi ? exp2_fast(st[k].x - base) : 0.0f;
                            mm = mn;
                            ll = ll * f0 + st[k].y * f1;
                            y[0] = y[0] * f0 + v[k].x * f1;
                            y[1] = y[1] * f0 + v[k].y * f1;
                            y[2] = y[2] * f0 + v[k].z * f1;
                            y[3] = y[3] * f0 + v[k].w * f1;
                        }
                    }
                    store_row(r, c, y, mm, ll);
                }
            }
        }
        // the ring was written as ordinary memory: order that before the next copies into it
        fence_proxy_async_smem();
        __syncthreads();
        }

        w = we;
        if (w < w1) next_item(a.s, a.c, extent, a.tiles, t, &g_attn_rows_error);
    }
}

template <int D>
cudaError_t launch(AttnArgs a, const void* k, const void* v, int sms, cudaStream_t stream) {
    using C = Cfg<D>;
    CUtensorMap mk, mv;
    if (!make_cache_map(&mk, k, a.c, kStrip, D / 64) || !make_cache_map(&mv, v, a.c, kStrip, D / 64))
        return cudaErrorInvalidValue;
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(attn_rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)C::kSmem);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    a.tiles = (int)(((long long)a.s.max_new * a.group + R - 1) / R);
    const long long P = most_shares(a, kStrip, kItemCost, kMinUnits, (long long)sms * C::kCtas);
    return launch_pdl(attn_rows_kernel<D>, dim3((unsigned)P), dim3(kThreads), C::kSmem, stream, true, mk, mv, a);
}

}  // namespace

template <int D>
constexpr size_t parts_bytes() { return (size_t)kMaxSms * Cfg<D>::kCtas * 2 * Cfg<D>::kPart * 4; }
size_t attn_rows_workspace(int D) {
    return D == 64 ? parts_bytes<64>() : D == 128 ? parts_bytes<128>() : parts_bytes<256>();
}

cudaError_t launch_attn_rows(const AttnArgs& a, const void* k, const void* v, int sms,
                             cudaStream_t stream) {
    switch (a.c.head_dim) {
        case 64: return launch<64>(a, k, v, sms, stream);
        case 128: return launch<128>(a, k, v, sms, stream);
        default: return launch<256>(a, k, v, sms, stream);
    }
}

cudaError_t read_attn_rows_device_error(int* code) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_attn_rows_error, sizeof(int));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_attn_rows_error, &zero, sizeof(int));
}

}  // namespace tern
