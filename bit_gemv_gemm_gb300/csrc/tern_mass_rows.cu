// tern_mass_rows.cu -- the attention weight of few query rows a key head
// (decode, verify), added to each key's running mass: bound by reading K once.
//
// As in the attention's rows kernel the keys go in strips of 16, all strips
// of all (sequence, key head) items cut into equal contiguous shares, and
// every warp brings its strips into a ring of its own by TMA.  A strip's
// scores are one S = Q K^T by mma.sync per 16 query rows; with the lse known
// the weights are exp2(S - lse) at once, and a key's sum is a sum down its
// column of S: over a thread's rows, then over the eight lanes that hold the
// column.  A strip belongs to one warp, so a key's sum has a fixed order.
// 8 sequences of up to 16k keys, 8 key heads of 128: 39 us, 4.7 TB/s (some 5 us to
// find the shares and fill the rings).
#include <algorithm>

#include "tern_attn.cuh"

namespace tern {
namespace {

__device__ int g_mass_rows_error;

constexpr int kStrip = 16, kRows = 64;

// A strip is little work in a long chain (wait, loads, products, exponentials,
// shuffles: about 2000 clocks), so an SM needs many warps to keep its copies
// coming: 16, with three strips each in flight.
template <int D>
struct Cfg {
    static constexpr int kWarps = D == 256 ? 8 : 16, kThreads = kWarps * 32;
    static constexpr int kMinUnits = kWarps;           // strips a share holds at least
    static constexpr int kStage = kStrip * D * 2;      // K of one strip
    static constexpr int kStages = D == 64 ? 6 : 3;
    static constexpr size_t kSmemQ = (size_t)kWarps * kStages * kStage;
    static constexpr size_t kSmemBar = kSmemQ + (size_t)kRows * D * 2;
    static constexpr size_t kSmemLse = kSmemBar + kWarps * kStages * 8;
    static constexpr size_t kSmemMisc = kSmemLse + kRows * 4;
    static constexpr size_t kSmem = kSmemMisc + 256 + 1024;
};

template <int UNIT>
struct AllKeysExtent {   // every key of the sequence, against all its rows
    int group;
    __device__ __forceinline__ void operator()(Item& t) const {
        t.rows = t.q.n * group;
        t.j0 = 0;
        t.j1 = t.q.len;
        t.units = (t.q.len + UNIT - 1) / UNIT;
    }
};

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
mass_rows_kernel(const __grid_constant__ CUtensorMap tmap_k, const MassArgs a) {
    using namespace sm100;
    using C = Cfg<D>;
    constexpr int kWarps = C::kWarps, kThreads = C::kThreads;
    extern __shared__ __align__(1024) unsigned char smem_dyn[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = sbase + (uint32_t)(warp * C::kStages * C::kStage), qs = sbase + (uint32_t)C::kSmemQ;
    const uint32_t bars = sbase + (uint32_t)C::kSmemBar + (uint32_t)(warp * C::kStages * 8);
    float* sm_lse = reinterpret_cast<float*>(smem + C::kSmemLse);
    long long* sm_scan = reinterpret_cast<long long*>(smem + C::kSmemMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm_scan + 8 + kWarps);

    if (lane == 0) {
        for (int s = 0; s < C::kStages; ++s) mbar_init(bars + 8u * s, 1);
        fence_barrier_init();
        if (warp == 0) {
            *abort_flag = 0;
            tma_prefetch_desc(&tmap_k);
        }
    }
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();

    int P;
    long long total, w0, w1;
    Item t;
    const AllKeysExtent<kStrip> extent{a.group};
    if (!find_share<kThreads>(a.s, a.c, extent, 1, C::kMinUnits, (int)blockIdx.x, (int)gridDim.x, sm_scan, &g_mass_rows_error, total, P, w0, w1, t)) return;

    uint32_t it = 0;
    for (long long w = w0; w < w1;) {
        const Seq q = t.q;
        const int rows = t.rows, hk = t.hk, tiles = (rows + 15) / 16;
        const long long we = min(w1, t.at + t.units);
        const int first = (int)(w - t.at), strips = (int)(we - w);
        const int my = strips > warp ? (strips - warp + kWarps - 1) / kWarps : 0;
        const int* trow = a.s.table + (long long)t.b * a.s.width;
        int ids = 0;
        auto fetch_ids = [&](int base) {
            const int k = base + lane;
            ids = 0;
            if (k < my)
                ids = checked_page_to_write(trow[(unsigned)((first + warp + kWarps * k) * kStrip) / (unsigned)a.c.page_size], a.c.pages, &g_mass_rows_error);
        };
        auto issue = [&](int k) {
            const int page = __shfl_sync(0xffffffffu, ids, k & 31);
            if (lane == 0) {
                const uint32_t s = (it + (uint32_t)k) % C::kStages;
                const int slot = (unsigned)((first + warp + kWarps * k) * kStrip) % (unsigned)a.c.page_size;
                mbar_arrive_expect_tx(bars + 8u * s, C::kStage);
                tma_load_cache(ring + s * C::kStage, &tmap_k, slot, 0, hk, max(page, 0), bars + 8u * s);
            }
        };
        // the mass of strip k, lane (lane & 15)'s key; -1: none.  Its page id is still in the lanes: in the block of
        // 32 that the ring is being filled from, or in the one before
        int before = 0;
        auto mass_at = [&](int k, int filled) -> long long {
            const int now = __shfl_sync(0xffffffffu, ids, k & 31), old = __shfl_sync(0xffffffffu, before, k & 31);
            const int strip = first + warp + kWarps * k, key = strip * kStrip + (lane & 15);
            if (k >= my || key >= q.len || lane >= 16) return -1;
            const int page = (k >> 5) == (filled >> 5) ? now : old;
            if (page < 0) return -1;   // (a bad id)
            return ((long long)page * a.c.kv_heads + hk) * a.c.page_size + (unsigned)key % (unsigned)a.c.page_size;
        };
        fetch_ids(0);
        for (int k = 0; k < C::kStages && k < my; ++k) issue(k);
        for (int i = threadIdx.x; i < tiles * 16 * (D / 8); i += kThreads) {
            const int r = i / (D / 8), c = i % (D / 8);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < rows)
                v = *reinterpret_cast<const uint4*>(a.q + (long long)(q.q0 + r / a.group) * a.q_stride +
                                                    (long long)(hk * a.group + r % a.group) * D + c * 8);
            *reinterpret_cast<uint4*>(smem + C::kSmemQ + (c >> 3) * (kRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
        }
        for (int r = threadIdx.x; r < tiles * 16; r += kThreads) {
            // a row without keys (lse = -inf) and a row past the last weigh nothing
            float x = INFINITY;
            if (r < rows) {
                x = a.lse[(long long)(q.q0 + r / a.group) * a.q_heads + hk * a.group + r % a.group];
                x = x == -INFINITY ? INFINITY : x * 1.44269504088896341f;
            }
            sm_lse[r] = x;
        }
        const int p_lo = q.len - q.n, p_hi = q.len - 1;
        __syncthreads();

        long long at = mass_at(0, 0);
        float old = at >= 0 ? a.mass[at] : 0.0f;
        for (int k = 0; k < my; ++k) {
            const uint32_t slot = (it + (uint32_t)k) % C::kStages, phase = ((it + (uint32_t)k) / C::kStages) & 1u;
            const int key0 = (first + warp + kWarps * k) * kStrip;
            // (the block of strip k + stages is in ids from the end of step k on, that of strip k + stages - 1 now)
            const long long next_at = mass_at(k + 1, k + C::kStages - 1);
            const float next_old = next_at >= 0 ? a.mass[next_at] : 0.0f;
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(bars + 8u * slot, phase, abort_flag, kAttnWaitNs))) {
                if (!*abort_flag) {
                    *abort_flag = 1;
                    if (lane == 0) report_device_error(&g_mass_rows_error, TERN_DEVERR_ATTN_WAIT);
                }
                if (lane == 0)
                    for (int x = k; x < my && x < k + C::kStages; ++x)
                        (void)mbar_wait_drain(bars + 8u * ((it + (uint32_t)x) % C::kStages),
                                              ((it + (uint32_t)x) / C::kStages) & 1u, 100000000ull);
                break;
            }
            const uint32_t ks = ring + slot * C::kStage;
            const int mi = lane >> 3, l7 = lane & 7;
            float sum[2][2] = {};   // keys key0 + 8 n + 2 (lane & 3) + e
            const bool masked = key0 + kStrip - 1 > p_lo || (a.window > 0 && key0 <= p_hi - a.window);
            for (int i = 0; i < tiles; ++i) {
                // two accumulators a column tile, fragments loaded four steps ahead: the products are a short chain
                float s2[2][2][4] = {};
#pragma unroll
                for (int k4 = 0; k4 < D / 64; ++k4) {
                    uint32_t kb[4][4], qa[4][4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int krow = (mi >> 1) * 8 + l7, kc = x * 2 + (mi & 1);
                        ldsm4(kb[x], ks + k4 * (kStrip * 128) + krow * 128 + ((kc ^ l7) << 4));
                        const int qrow = i * 16 + (mi & 1) * 8 + l7, qc = x * 2 + (mi >> 1);
                        ldsm4(qa[x], qs + k4 * (kRows * 128) + qrow * 128 + ((qc ^ l7) << 4));
                    }
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        mma_bf16(s2[x & 1][0], qa[x], kb[x][0], kb[x][1]);
                        mma_bf16(s2[x & 1][1], qa[x], kb[x][2], kb[x][3]);
                    }
                }
                float s[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[n][e] = s2[0][n][e] + s2[1][n][e];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = i * 16 + h * 8 + (lane >> 2);
                    const float z = sm_lse[r];
                    const int p = q.len - q.n + r / a.group;
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float x = exp2_fast(fmaf(s[n][2 * h + e], a.scale_log2, -z));
                            if (masked) {
                                const int key = key0 + n * 8 + (lane & 3) * 2 + e;
                                if (key > p || (a.window > 0 && key <= p - a.window) || r >= rows) x = 0.0f;
                            }
                            sum[n][e] += x;
                        }
                }
            }
            __syncwarp();
            if (((k + C::kStages) & 31) == 0) {
                before = ids;
                fetch_ids(k + C::kStages);
            }
            if (k + C::kStages < my) issue(k + C::kStages);
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sum[n][e] += __shfl_xor_sync(0xffffffffu, sum[n][e], 4);
                    sum[n][e] += __shfl_xor_sync(0xffffffffu, sum[n][e], 8);
                    sum[n][e] += __shfl_xor_sync(0xffffffffu, sum[n][e], 16);
                }
            // lane i < 16 writes key i: its sum lies with lane (i % 8) / 2, half i / 8, element i % 2
            const int from = (lane & 7) >> 1;
            const float a0 = __shfl_sync(0xffffffffu, sum[0][0], from), a1 = __shfl_sync(0xffffffffu, sum[0][1], from);
            const float b0 = __shfl_sync(0xffffffffu, sum[1][0], from), b1 = __shfl_sync(0xffffffffu, sum[1][1], from);
            const float got = (lane & 8) ? ((lane & 1) ? b1 : b0) : ((lane & 1) ? a1 : a0);
            if (at >= 0) a.out[at] = fmaf(a.decay, old, got);
            at = next_at;
            old = next_old;
        }
        it += (uint32_t)my;
        __syncthreads();   // the rows of Q are replaced next
        if (*abort_flag) return;
        w = we;
        if (w < w1) next_item(a.s, a.c, extent, 1, t, &g_mass_rows_error);
    }
}

template <int D>
cudaError_t launch(const MassArgs& a, const void* k, int sms, cudaStream_t stream) {
    using C = Cfg<D>;
    CUtensorMap mk;
    if (!make_cache_map(&mk, k, a.c, kStrip, D / 64)) return cudaErrorInvalidValue;
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(mass_rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)C::kSmem);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    const long long strips = (long long)a.s.B * a.c.kv_heads * ((long long)a.s.width * a.c.page_size / kStrip);
    const long long P = std::min<long long>(sms, (strips + C::kMinUnits - 1) / C::kMinUnits);
    return launch_pdl(mass_rows_kernel<D>, dim3((unsigned)P), dim3(C::kThreads), C::kSmem, stream, true, mk, a);
}

}  // namespace

cudaError_t launch_mass_rows(const MassArgs& a, const void* k, int sms, cudaStream_t stream) {
    switch (a.c.head_dim) {
        case 64: return launch<64>(a, k, sms, stream);
        case 128: return launch<128>(a, k, sms, stream);
        default: return launch<256>(a, k, sms, stream);
    }
}

cudaError_t read_mass_rows_device_error(int* code) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_mass_rows_error, sizeof(int));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_mass_rows_error, &zero, sizeof(int));
}

}  // namespace tern
