// tern_delta_chunk.cu -- the gated delta rule over prompts, 64 tokens at a time,
// on the tcgen05 tensor cores.
//
// With G the running sum of the decays' logs in a chunk and S the state before it,
//   A_ij = beta_i e^(G_i - G_j) k_i.k_j (j < i),   T = (I + A)^-1 diag(beta),
//   U = T (V - e^G K S^T),
//   O = scale e^G Q S^T + P U,   P_ij = scale e^(G_i - G_j) q_i.k_j (j <= i),
//   S <- e^(G_last) S + sum_j e^(G_last - G_j) u_j k_j^T.
// A CTA takes 128 rows of one head's S through its sequence.  Everything with rows
// of S (S itself, X = V - e^G K S^T, U, O) is kept transposed, a thread a row, so
// those products have M = 128 and their left operand in tensor memory, and what
// passes from one product to the next never leaves its row.
//
// The chain from chunk to chunk, four phases of eight warps (two threads a row)
// between three products:
//   S = e^G_last S + D, its parts to tensor memory  ->  K S^T
//   X = V - e^G K S^T                               ->  U = T X
//   e^(G_last - G) U                                ->  D = U^T K
// and beside it, in the gaps of the tensor pipe: Q S^T and P U, the output, and the
// Gram matrices [K; Q] K^T of the chunk after the next, from which four warps make T
// (forward substitution, a thread a column) and P, two warps the decays and the
// lengths of q and k from the tiles themselves.
//
// Rounding.  q, k, v are exact as bf16.  S, X, U and T are fp32 cut into two bf16
// values, which carry 2^-17 of each (one would lose 2^-8 of the state a chunk);
// lengths and decays are applied in fp32, to rows and columns of results.  P is one
// bf16: it only reaches the output, which is rounded to that.
// Exponents are differences of G, at most 0, and G is a sum in 64 bits kept as two
// fp32: a long or strong decay before a pair of tokens does not blur theirs.
#include "tern_delta.cuh"
#include "tern_sm100.cuh"

namespace tern {
namespace {

using namespace sm100;

__device__ int g_delta_chunk_error;

constexpr int kDiagRow = 20;                          // floats of a row of a 16 x 16 block of A
constexpr int kTok = 64, kRows = 128;                 // tokens of a chunk, rows of S
constexpr int kKqStages = 3, kVStages = 3, kCoefStages = 4, kTpStages = 2;
constexpr uint64_t kDeltaWaitNs = 1000000000ull;      // 1 s: far beyond any real wait

// What one chunk's tokens are scaled by.
struct alignas(16) Coef {
    float beta[kTok], minus_near[kTok];   // beta; -beta e^G |k|^-1
    float left[kTok];                     // e^(G_last - G) |k|^-1
    float near_q[kTok];                   // scale e^G |q|^-1
    float beta_k[kTok], scale_q[kTok], k[kTok];   // beta |k|^-1; scale |q|^-1; |k|^-1
    float to_end[kTok];                   // |k|^-1 e^(G at its 16's last token - G)
    float2 G[kTok];                       // G in powers of two, two parts
    float2 end[4];                        // that of each 16's last token
    float last, unused[3];                // e^G_last
};

template <int DK>
struct Cfg {
    static constexpr int NC = DK / 64;                          // chunks of 64 values of a K or Q row
    static constexpr int HALF = DK / 2;                         // columns of S that a thread holds
    static constexpr int kKqBytes = NC * 2 * kTok * 128;        // K over Q, 128-byte swizzled rows
    static constexpr int kVBytes = 2 * kTok * 128;
    static constexpr int kTpBytes = 3 * kTok * 128;             // T's two parts, P
    static constexpr size_t kKq = 0, kV = kKq + (size_t)kKqStages * kKqBytes, kTp = kV + (size_t)kVStages * kVBytes,
                            kA = kTp + (size_t)kTpStages * kTpBytes, kDiag = kA + 2 * kTok * 128,
                            kCoef = kDiag + kTok * kDiagRow * 4,
                            kBar = kCoef + kCoefStages * sizeof(Coef), kMisc = kBar + 48 * 8, kSmem = kMisc + 64 + 1024;
};
constexpr int kThreads = 512;

// tensor memory columns: D over the parts of S; K S^T, then U; Q S^T; parts of X, then
// of U; parts of the scaled U; P U; Gram matrices
enum { T_S = 0, T_KS = 128, T_QS = 192, T_X = 256, T_UP = 320, T_O = 384, T_GRAM = 448 };

enum {
    KQ_FULL = 0, KQ_EMPTY = KQ_FULL + kKqStages, V_FULL = KQ_EMPTY + kKqStages, V_EMPTY = V_FULL + kVStages,
    COEF_FULL = V_EMPTY + kVStages, COEF_EMPTY = COEF_FULL + kCoefStages, TP_FULL = COEF_EMPTY + kCoefStages,
    TP_EMPTY = TP_FULL + kTpStages, GRAM_FULL = TP_EMPTY + kTpStages, GRAM_EMPTY, S_FULL, KS_FULL, X_FULL, U_FULL,
    UP_FULL, U2_FULL, D_FULL, O_FULL, O_EMPTY, PREP, TAIL, DRAIN, BARS
};
static_assert(BARS <= 48, "barriers");

__device__ __forceinline__ int bar_count(int i) {
    if (i >= V_EMPTY && i < V_EMPTY + kVStages) return 8;
    if (i >= COEF_FULL && i < COEF_EMPTY) return 2;
    if (i >= COEF_EMPTY && i < TP_FULL) return 8;
    if ((i >= TP_FULL && i < TP_EMPTY) || i == GRAM_EMPTY || i == PREP) return 4;
    if (i == S_FULL || i == X_FULL || i == UP_FULL || i == U2_FULL || i == O_EMPTY) return 8;
    return 1;
}

// Two neighbours as a bf16 pair and what it leaves of them as another.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = pack_bf16(a, b);
    float x, y;
    unpack2(add2(pack2(a, b), pack2(-__uint_as_float(hi << 16), -__uint_as_float(hi & 0xFFFF0000u))), x, y);
    lo = pack_bf16(x, y);
}

// A 16-byte unit of a row of a [64][64] bf16 tile with 128-byte swizzled rows.
__device__ __forceinline__ uint32_t tile_at(uint32_t tile, int row, int unit) {
    return tile + (uint32_t)(row * 128 + ((unit ^ (row & 7)) << 4));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm2_t(uint32_t& a, uint32_t& b, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr) : "memory");
}
// an 8 x 8 bf16 matrix, a row over four lanes, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Column `col` of the inverse of a 16 x 16 unit lower triangle, whose strict part is at A.
__device__ __forceinline__ void solve16(const float* A, int col, float (&t)[16]) {
    uint64_t pair[8];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        uint64_t s0 = 0, s1 = 0;
#pragma unroll
        for (int k = 0; k < i; k += 4) {
            const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(A + i * kDiagRow + k);
            s0 = fma2(a.x, pair[k / 2], s0);
            if (k + 2 < i) s1 = fma2(a.y, pair[k / 2 + 1], s1);
        }
        float x, y;
        unpack2(add2(s0, s1), x, y);
        t[i] = (i == col ? 1.0f : 0.0f) - (x + y);
        pair[i / 2] = (i & 1) ? pack2(t[i - 1], t[i]) : pack2(t[i], 0.0f);
    }
}
// Rows R.., columns C.. of T below its diagonal blocks, 8 columns `n8` of it a warp:
//   -T22 (A21 T11),  T11 and T22 the 16 B rows from C and R on, every product of two
// parts each without the smallest (lo lo).
template <int B>
__device__ __forceinline__ void join_blocks(uint32_t A, uint32_t T, int R, int C, int n8, int lane) {
    constexpr uint32_t kPart = kTok * 128;
    float m[B][4];
#pragma unroll
    for (int i = 0; i < B; ++i) m[i][0] = m[i][1] = m[i][2] = m[i][3] = 0.0f;
#pragma unroll
    for (int kb = 0; kb < B; ++kb) {
        uint32_t bh[2], bl[2];
        const uint32_t at = tile_at(T, C + 16 * kb + (lane & 15), C / 8 + n8);
        ldsm2_t(bh[0], bh[1], at);
        ldsm2_t(bl[0], bl[1], at + kPart);
#pragma unroll
        for (int i = 0; i < B; ++i) {
            uint32_t ah[4], al[4];
            const uint32_t from = tile_at(A, R + 16 * i + (lane & 15), C / 8 + 2 * kb + (lane >> 4));
            ldsm4(ah, from);
            ldsm4(al, from + kPart);
            mma_bf16(m[i], ah, bh[0], bh[1]);
            mma_bf16(m[i], ah, bl[0], bl[1]);
            mma_bf16(m[i], al, bh[0], bh[1]);
        }
    }
    uint32_t mh[B][2], ml[B][2];
#pragma unroll
    for (int i = 0; i < B; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            uint32_t hi, lo;
            split2(-m[i][2 * x], -m[i][2 * x + 1], hi, lo);
            mh[i][x] = transpose8(hi);
            ml[i][x] = transpose8(lo);
        }
#pragma unroll
    for (int i = 0; i < B; ++i) {
        float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kb = 0; kb <= i; ++kb) {
            uint32_t ah[4], al[4];
            const uint32_t from = tile_at(T, R + 16 * i + (lane & 15), R / 8 + 2 * kb + (lane >> 4));
            ldsm4(ah, from);
            ldsm4(al, from + kPart);
            mma_bf16(t, ah, mh[kb][0], mh[kb][1]);
            mma_bf16(t, ah, ml[kb][0], ml[kb][1]);
            mma_bf16(t, al, mh[kb][0], mh[kb][1]);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            uint32_t hi, lo;
            split2(t[2 * x], t[2 * x + 1], hi, lo);
            const uint32_t to = tile_at(T, R + 16 * i + 8 * x + lane / 4, C / 8 + n8) + 4u * (lane & 3);
            sts32(to, hi);
            sts32(to + kPart, lo);
        }
    }
}

// The log of a decay in powers of two, times 2^40: |g| is at most 200 here.
__device__ __forceinline__ long long fixed_log2(float g) {
    g = g > 200.0f ? 200.0f : g;
    const float p = g * 1.44269502162933349609f, e = fmaf(g, 1.44269502162933349609f, -p) + g * 1.92596299e-8f;
    return __float2ll_rn(p * 1099511627776.0f) + __float2ll_rn(e * 1099511627776.0f);
}
__device__ __forceinline__ float unfixed(long long x) { return __ll2float_rn(x) * 9.094947017729282379e-13f; }

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, uint32_t src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(m)), "r"(src), "r"(c0), "r"(c1), "r"(c2) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// the stores of this thread have read their shared memory; have been carried out
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

template <int DK>
__global__ void __launch_bounds__(kThreads, 1)
delta_chunk_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                   const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_out,
                   const DeltaArgs a) {
    using C = Cfg<DK>;
    constexpr int NC = C::NC, HALF = C::HALF;
    extern __shared__ __align__(1024) unsigned char smem_dyn[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) { return sbase + (uint32_t)C::kBar + 8u * (uint32_t)i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    Coef* const coefs = reinterpret_cast<Coef*>(smem + C::kCoef);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < BARS; ++i) mbar_init(bar(i), (uint32_t)bar_count(i));
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmap_q);
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
        tma_prefetch_desc(&tmap_out);
    }
    // T and P above their diagonal 16 x 16 blocks stay 0
    for (int i = threadIdx.x; i < kTpStages * C::kTpBytes / 16; i += kThreads)
        reinterpret_cast<uint4*>(smem + C::kTp)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    if (warp == 12) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_dependents();
    pdl_wait();

    const int h = blockIdx.x % a.v_heads, row0 = blockIdx.x / a.v_heads * kRows, hk = h / a.group;
    const StateSeq s = load_state_seq(a.s, blockIdx.y, &g_delta_chunk_error);
    const int chunks = (s.n + kTok - 1) / kTok;
    auto fail = [&] {
        if (!*abort_flag) {
            *abort_flag = 1;
            report_device_error(&g_delta_chunk_error, TERN_DEVERR_DELTA_WAIT);
        }
    };
    auto wait = [&](int b, uint32_t parity) { return mbar_wait_bounded(bar(b), parity, abort_flag, kDeltaWaitNs); };
    auto wait_warp = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)) != 0; };
    auto arrive = [&](int b) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(b));
    };

    if (warp < 8) {
        // ------------------------------ the chain ------------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        const int half = warp >> 2, row = (warp & 3) * 32 + lane;
        const bool live = row0 + row < a.dv;
        const uint32_t mine = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t ts = mine + T_S + (uint32_t)(HALF * half);
        float S[HALF];
        {
            const float4* from = reinterpret_cast<const float4*>(
                a.state + (((long long)s.src * a.v_heads + h) * a.dv + row0 + row) * DK + HALF * half);
#pragma unroll
            for (int i = 0; i < HALF / 4; ++i) {
                const float4 x = s.src >= 0 && live ? from[i] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                S[4 * i] = x.x;
                S[4 * i + 1] = x.y;
                S[4 * i + 2] = x.z;
                S[4 * i + 3] = x.w;
            }
        }
        auto v_tile = [&](int c) {   // this warp's 32 rows of S: [token][32 values]
            return reinterpret_cast<__nv_bfloat16*>(smem + C::kV + (c % kVStages) * C::kVBytes + (warp & 3) * (kTok * 64) +
                                                    half * (32 * 64)) + lane;
        };
        // S = e^G_last S + D of a chunk, and its parts to where D was: 16 columns each of 32 values
        auto next_state = [&](int c, bool more) {
            float last = 1.0f;
            if (c >= 0) {
                if (!wait_warp(D_FULL, (uint32_t)c & 1u)) return false;
                tc_fence_after();
                last = coefs[c % kCoefStages].last;
            }
            const uint64_t last2 = pack2(last, last);
#pragma unroll
            for (int i = 0; i < HALF; i += 32) {
                if (c >= 0) {
                    uint32_t d[32];
                    tmem_ld_x32(ts + (uint32_t)i, d);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        unpack2(fma2(last2, pack2(S[i + e], S[i + e + 1]),
                                     pack2(__uint_as_float(d[e]), __uint_as_float(d[e + 1]))), S[i + e], S[i + e + 1]);
                }
                if (!more) continue;
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) split2(S[i + 2 * e], S[i + 2 * e + 1], hi[e], lo[e]);
                tmem_st_x16(ts + (uint32_t)i, hi);
                tmem_st_x16(ts + (uint32_t)i + 16u, lo);
            }
            return true;
        };
        // the output of a chunk: this thread's row, 32 of its tokens
        auto output = [&](int c) {
            if (!wait_warp(O_FULL, (uint32_t)c & 1u)) return false;
            tc_fence_after();
            const Coef& k = coefs[c % kCoefStages];
            uint32_t x[32], y[32];
            tmem_ld_x32(mine + T_QS + 32u * half, x);
            tmem_ld_x32(mine + T_O + 32u * half, y);
            tmem_ld_wait();
            tc_fence_before();
            arrive(O_EMPTY);
            // over the values that this thread read there, and out of shared memory in one piece
            __nv_bfloat16* const o = v_tile(c);
#pragma unroll
            for (int i = 0; i < 32; ++i)
                o[32 * i] = __float2bfloat16(fmaf(k.near_q[32 * half + i], __uint_as_float(x[i]), __uint_as_float(y[i])));
            const int first = c * kTok + 32 * half, n = s.n - first;
            if (n >= 32) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && row0 + row < a.dv) {
                    tma_store_3d(&tmap_out, smem_u32(o), row0 + row, h, s.t0 + first);
                    bulk_commit();
                }
            } else if (live) {   // the sequence ends among these tokens
                const long long step = (long long)a.v_heads * a.dv;
                __nv_bfloat16* to = a.out + (s.t0 + first) * step + (long long)h * a.dv + row0 + row;
                for (int i = 0; i < n; ++i) to[i * step] = o[32 * i];
            }
            arrive(COEF_EMPTY + c % kCoefStages);
            return true;
        };
        auto stored = [&](int c) {   // the stores of a chunk's output have left its place in shared memory
            if (lane == 0) {
                bulk_wait_read();
                mbar_arrive(bar(V_EMPTY + c % kVStages));
            }
        };
        bool ok = true;
        for (int c = 0; c < chunks; ++c) {
            const uint32_t ph = (uint32_t)c & 1u;
            if (!next_state(c - 1, true)) { ok = false; break; }
            tmem_st_wait();
            tc_fence_before();
            arrive(S_FULL);
            if (c > 1) stored(c - 2);
            if (c > 0 && !output(c - 1)) { ok = false; break; }

            const Coef& k = coefs[c % kCoefStages];
            if (!wait_warp(COEF_FULL + c % kCoefStages, (uint32_t)(c / kCoefStages) & 1u) ||
                !wait_warp(V_FULL + c % kVStages, (uint32_t)(c / kVStages) & 1u) || !wait_warp(KS_FULL, ph)) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t x[32], hi[16], lo[16];
            tmem_ld_x32(mine + T_KS + 32u * half, x);
            const __nv_bfloat16* v = v_tile(c);
            float vx[32];   // then what the parts of X leave of it: T's diagonal is 1
#pragma unroll
            for (int i = 0; i < 32; ++i) vx[i] = __bfloat162float(v[32 * i]) * k.beta[32 * half + i];
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float2 near = *reinterpret_cast<const float2*>(&k.minus_near[32 * half + 2 * e]);
                float p, q;
                unpack2(fma2(pack2(near.x, near.y), pack2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])),
                             pack2(vx[2 * e], vx[2 * e + 1])), p, q);
                split2(p, q, hi[e], lo[e]);
                unpack2(add2(pack2(p, q), pack2(-__uint_as_float(hi[e] << 16), -__uint_as_float(hi[e] & 0xFFFF0000u))), p, q);
                unpack2(add2(pack2(p, q), pack2(-__uint_as_float(lo[e] << 16), -__uint_as_float(lo[e] & 0xFFFF0000u))),
                        vx[2 * e], vx[2 * e + 1]);
            }
            tmem_st_x16(mine + T_X + 16u * half, hi);
            tmem_st_x16(mine + T_X + 32u + 16u * half, lo);
            tmem_st_wait();
            tc_fence_before();
            arrive(X_FULL);

            if (!wait_warp(U_FULL, ph)) { ok = false; break; }
            tc_fence_after();
            tmem_ld_x32(mine + T_KS + 32u * half, x);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) + vx[i]);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float2 left = *reinterpret_cast<const float2*>(&k.left[32 * half + 2 * e]);
                float p, q;
                unpack2(mul2(pack2(left.x, left.y), pack2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]))), p, q);
                split2(p, q, hi[e], lo[e]);
            }
            tmem_st_x16(mine + T_UP + 16u * half, hi);
            tmem_st_x16(mine + T_UP + 32u + 16u * half, lo);
            tmem_st_wait();
            tc_fence_before();
            arrive(UP_FULL);
#pragma unroll
            for (int e = 0; e < 16; ++e) split2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]), hi[e], lo[e]);
            tmem_st_x16(mine + T_X + 16u * half, hi);
            tmem_st_x16(mine + T_X + 32u + 16u * half, lo);
            tmem_st_wait();
            tc_fence_before();
            arrive(U2_FULL);
        }
        if (ok && chunks > 0) ok = next_state(chunks - 1, false) && output(chunks - 1);
        if (lane == 0) bulk_wait();
        if (!ok) {
            if (lane == 0) fail();
        } else if (s.dst >= 0 && live && (s.n > 0 || s.dst != s.src)) {
            float4* to = reinterpret_cast<float4*>(
                a.state + (((long long)s.dst * a.v_heads + h) * a.dv + row0 + row) * DK + HALF * half);
#pragma unroll
            for (int i = 0; i < HALF / 4; ++i) to[i] = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
        }
        __syncwarp();
    } else if (warp < 12) {
        // ------------------------------ T and P from the Gram matrices ------------------------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
        // warps 8 and 9: K K^T, rows 0-31 and 32-63; 10 and 11: Q K^T
        const int part = (warp - 8) & 1, i = 32 * part + lane, me = warp - 8;
        const bool is_k = warp < 10, low = lane < 16;
        const uint32_t gram = tmem + ((uint32_t)((warp - 8) * 32) << 16) + T_GRAM;
        const uint32_t A = sbase + (uint32_t)C::kA;
        float* const diag = reinterpret_cast<float*>(smem + C::kDiag);
        uint32_t syncs = 0;
        auto sync_warps = [&] {   // the four of them
            arrive(PREP);
            return wait_warp(PREP, syncs++ & 1u);
        };
        // 16 values as bf16 to two units of a row of a tile (and what that leaves of them to the next tile)
        auto put16 = [&](uint32_t tile, int unit, const float (&z)[16], bool both) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) split2(z[8 * u + 2 * e], z[8 * u + 2 * e + 1], hi[e], lo[e]);
                const uint32_t at = tile_at(tile, i, unit + u);
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3]) : "memory");
                if (both)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + kTok * 128), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3]) : "memory");
            }
        };
        bool ok = true;
        for (int c = 0; c < chunks && ok; ++c) {
            const Coef& k = coefs[c % kCoefStages];
            const uint32_t T = sbase + (uint32_t)(C::kTp + (c % kTpStages) * C::kTpBytes);
            if (!wait_warp(COEF_FULL + c % kCoefStages, (uint32_t)(c / kCoefStages) & 1u) ||
                !wait_warp(GRAM_FULL, (uint32_t)c & 1u) ||
                !wait_warp(TP_EMPTY + c % kTpStages, ((uint32_t)(c / kTpStages) & 1u) ^ 1u) ||
                (c > 0 && !wait_warp(TP_FULL + (c - 1) % kTpStages, (uint32_t)((c - 1) / kTpStages) & 1u))) {
                ok = false;   // (the last: all four are done with the last chunk's A)
                break;
            }
            tc_fence_after();
            const float mul = is_k ? k.beta_k[i] : k.scale_q[i];
            const uint64_t G = pack2(k.G[i].x, k.G[i].y);
            auto decay_to = [&](float2 g) {   // e^(G_i - g)
                float x, y;
                unpack2(add2(G, pack2(-g.x, -g.y)), x, y);
                return exp2_fast(x + y);
            };
            const uint32_t to = is_k ? A : T + 2 * kTok * 128;
            // tokens of the 16s before this row's: through the last token of their 16, so that no factor is above 1
            auto before = [&](int b, const uint32_t* x) {
                const float f = decay_to(k.end[b]) * mul;
                float z[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) z[e] = f * k.to_end[16 * b + e] * __uint_as_float(x[e]);
                put16(to, 2 * b, z, is_k);
            };
            uint32_t x[32];
            if (part) {
                tmem_ld_x32(gram, x);
                tmem_ld_wait();
                before(0, x);
                before(1, x + 16);
            }
            __syncwarp();
            tmem_ld_x32(gram + 32u * part, x);
            tmem_ld_wait();
            tc_fence_before();
            arrive(GRAM_EMPTY);
            if (!low) before(2 * part, x);
            {   // this row's own 16: the difference itself, 0 right of the diagonal
                const int j0 = 32 * part + (lane & 16);
                float z[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float f = decay_to(k.G[j0 + e]) * k.k[j0 + e] * mul;
                    const int over = e - (lane & 15);
                    z[e] = over < (is_k ? 0 : 1) ? f * __uint_as_float(low ? x[e] : x[16 + e]) : 0.0f;
                }
                if (is_k) {
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        *reinterpret_cast<float4*>(diag + i * kDiagRow + e) = make_float4(z[e], z[e + 1], z[e + 2], z[e + 3]);
                } else {
                    put16(to, j0 / 8, z, false);
                }
            }
            if (!sync_warps()) { ok = false; break; }
            {   // the diagonal blocks of T, one a warp, a column a lane; the upper lanes keep the lower parts
                float t[16];
                solve16(diag + 16 * me * kDiagRow, lane & 15, t);
                const int col = 16 * me + (lane & 15);
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const __nv_bfloat16 hi = __float2bfloat16(t[r]), lo = __float2bfloat16(t[r] - __bfloat162float(hi));
                    const uint32_t at = tile_at(T, 16 * me + r, col / 8) + 2u * (col & 7) + (low ? 0u : (uint32_t)(kTok * 128));
                    const __nv_bfloat16 w = low ? hi : lo;
                    asm volatile("st.shared.b16 [%0], %1;" ::"r"(at), "h"(*reinterpret_cast<const unsigned short*>(&w)) : "memory");
                }
            }
            if (!sync_warps()) { ok = false; break; }
            join_blocks<1>(A, T, 32 * (me >> 1) + 16, 32 * (me >> 1), me & 1, lane);
            if (!sync_warps()) { ok = false; break; }
            join_blocks<2>(A, T, 32, 0, me, lane);
            fence_proxy_async_smem();
            arrive(TP_FULL + c % kTpStages);
        }
        if (!ok && lane == 0) fail();
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 12) {
            // ------------------------------ MMA ------------------------------
            if (lane == 0) {
                constexpr uint32_t kIdesc = idesc_bf16_f32(kRows, kTok);
                constexpr uint32_t kIdescD = idesc_bf16_f32(kRows, DK) | kIdescBMnMajor;
                bool ok = true, issued = false;
                auto need = [&](int b, uint32_t parity) {
                    if (ok && !wait(b, parity)) ok = false;
                    return ok;
                };
                auto kq = [&](int c) { return sbase + (uint32_t)(C::kKq + (c % kKqStages) * C::kKqBytes); };
                auto gram = [&](int c) {
                    if (!need(KQ_FULL + c % kKqStages, (uint32_t)(c / kKqStages) & 1u) ||
                        !need(GRAM_EMPTY, ((uint32_t)c & 1u) ^ 1u))
                        return;
                    tc_fence_after();
                    const uint64_t d = smem_desc_k_sw128(kq(c));
#pragma unroll
                    for (int kk = 0; kk < DK / 16; ++kk) {
                        const uint64_t at = d + (uint64_t)((kk / 4) * ((2 * kTok * 128) >> 4) + 2 * (kk % 4));
                        mma_f16_ss(tmem + T_GRAM, at, at, kIdesc, kk > 0);
                    }
                    issued = true;
                    mma_commit(bar(GRAM_FULL));
                };
                // (+)= parts of S times K (first = 0) or Q (1) rows
                auto with_state = [&](int c, uint32_t to, int first) {
                    const uint64_t d = smem_desc_k_sw128(kq(c) + (uint32_t)(first * kTok * 128));
#pragma unroll
                    for (int p = 0; p < 2; ++p)
#pragma unroll
                        for (int kk = 0; kk < DK / 16; ++kk) {
                            const uint32_t left = tmem + T_S + (uint32_t)(32 * (kk / 2) + 16 * p + 8 * (kk % 2));
                            mma_f16_ts(tmem + to, left, d + (uint64_t)((kk / 4) * ((2 * kTok * 128) >> 4) + 2 * (kk % 4)),
                                       kIdesc, (p | kk) ? 1u : 0u);
                        }
                };
                // (+)= 64 tokens in tensor memory times a [64][64] tile
                auto with_tile = [&](uint32_t to, uint32_t left, uint32_t tile, bool more) {
                    const uint64_t d = smem_desc_k_sw128(tile);
#pragma unroll
                    for (int kk = 0; kk < kTok / 16; ++kk)
                        mma_f16_ts(tmem + to, tmem + left + 8u * kk, d + 2 * kk, kIdesc, (more || kk) ? 1u : 0u);
                };
                if (chunks > 0) gram(0);
                if (chunks > 1) gram(1);
                for (int c = 0; c < chunks && ok; ++c) {
                    const uint32_t ph = (uint32_t)c & 1u;
                    const uint32_t tp = sbase + (uint32_t)(C::kTp + (c % kTpStages) * C::kTpBytes);
                    if (!need(S_FULL, ph)) break;
                    tc_fence_after();
                    with_state(c, T_KS, 0);
                    mma_commit(bar(KS_FULL));
                    if (c > 0 && !need(O_EMPTY, ph ^ 1u)) break;
                    tc_fence_after();
                    with_state(c, T_QS, 1);
                    if (!need(TP_FULL + c % kTpStages, (uint32_t)(c / kTpStages) & 1u) || !need(X_FULL, ph)) break;
                    tc_fence_after();
                    with_tile(T_KS, T_X, tp, false);
                    with_tile(T_KS, T_X + 32, tp, true);
                    with_tile(T_KS, T_X, tp + kTok * 128, true);
                    mma_commit(bar(U_FULL));
                    if (c + 2 < chunks) gram(c + 2);
                    if (!need(UP_FULL, ph)) break;
                    tc_fence_after();
                    {
                        const uint64_t d = smem_desc_mn_sw128(kq(c), 2 * kTok * 128);
#pragma unroll
                        for (int p = 0; p < 2; ++p)
#pragma unroll
                            for (int kk = 0; kk < kTok / 16; ++kk)
                                mma_f16_ts(tmem + T_S, tmem + T_UP + 32u * p + 8u * kk, d + (uint64_t)(kk * (2048 >> 4)),
                                           kIdescD, (p | kk) ? 1u : 0u);
                    }
                    mma_commit(bar(D_FULL));
                    mma_commit(bar(KQ_EMPTY + c % kKqStages));
                    if (!need(U2_FULL, ph)) break;
                    tc_fence_after();
                    with_tile(T_O, T_X, tp + 2 * kTok * 128, false);
                    with_tile(T_O, T_X + 32, tp + 2 * kTok * 128, true);
                    mma_commit(bar(TP_EMPTY + c % kTpStages));
                    mma_commit(bar(O_FULL));   // (the last: the CTA ends after it)
                }
                if (!ok) {
                    fail();
                    if (issued) {
                        mma_commit(bar(DRAIN));
                        (void)mbar_wait_drain(bar(DRAIN), 0u, 100000000ull);
                    }
                }
            }
            __syncwarp();
        } else if (warp == 13) {
            // ------------------------------ TMA ------------------------------
            // V comes a chunk behind K and Q, which are wanted two chunks ahead
            const int v_chunks = min(4, (a.dv - row0 + 31) / 32);
            const uint32_t kq_bytes = (uint32_t)C::kKqBytes, v_bytes = (uint32_t)(v_chunks * kTok * 64);
            // rows past the sequence's end count as 0
            auto zero = [&](unsigned char* rows, int from, int row_bytes) {
                for (int i = from * (row_bytes / 16) + lane; i < kTok * (row_bytes / 16); i += 32)
                    *reinterpret_cast<uint4*>(rows + i * 16) = make_uint4(0, 0, 0, 0);
            };
            bool ok = true;
            int kqs = 0, vs = 0;   // copies begun
            for (int c = 0; c <= chunks && ok; ++c) {
                if (c < chunks) {
                    const int st = c % kKqStages, left = s.n - c * kTok;
                    if (!wait_warp(KQ_EMPTY + st, ((uint32_t)(c / kKqStages) & 1u) ^ 1u)) { ok = false; break; }
                    const uint32_t at = sbase + (uint32_t)(C::kKq + st * C::kKqBytes), to = left < kTok ? bar(TAIL) : bar(KQ_FULL + st);
                    if (lane == 0) {
                        mbar_arrive_expect_tx(to, kq_bytes);
                        for (int x = 0; x < NC; ++x) {
                            tma_load_2d(at + (uint32_t)(2 * x * kTok * 128), &tmap_k, hk * DK + 64 * x, s.t0 + c * kTok, to);
                            tma_load_2d(at + (uint32_t)((2 * x + 1) * kTok * 128), &tmap_q, hk * DK + 64 * x, s.t0 + c * kTok, to);
                        }
                    }
                    ++kqs;
                    __syncwarp();
                    if (left < kTok) {
                        if (!wait_warp(TAIL, 0u)) { ok = false; break; }
                        for (int x = 0; x < NC; ++x) zero(smem + C::kKq + st * C::kKqBytes + 2 * x * kTok * 128, left, 128);
                        fence_proxy_async_smem();
                        arrive(KQ_FULL + st);
                    }
                }
                if (c > 0) {
                    const int b = c - 1, st = b % kVStages, left = s.n - b * kTok;
                    if (!wait_warp(V_EMPTY + st, ((uint32_t)(b / kVStages) & 1u) ^ 1u)) { ok = false; break; }
                    const uint32_t at = sbase + (uint32_t)(C::kV + st * C::kVBytes), to = left < kTok ? bar(TAIL) : bar(V_FULL + st);
                    if (lane == 0) {
                        mbar_arrive_expect_tx(to, v_bytes);
                        for (int x = 0; x < v_chunks; ++x)
                            tma_load_2d(at + (uint32_t)(x * kTok * 64), &tmap_v, h * a.dv + row0 + 32 * x, s.t0 + b * kTok, to);
                    }
                    ++vs;
                    __syncwarp();
                    if (left < kTok) {
                        if (!wait_warp(TAIL, 1u)) { ok = false; break; }
                        for (int x = 0; x < v_chunks; ++x) zero(smem + C::kV + st * C::kVBytes + x * kTok * 64, left, 64);
                        fence_proxy_async_smem();
                        arrive(V_FULL + st);
                    }
                }
            }
            if (!ok && lane == 0) {
                fail();
                // copies in flight land before the CTA goes away
                const bool tail = s.n % kTok != 0;
                for (int i = max(0, kqs - kKqStages); i < kqs; ++i)
                    (void)mbar_wait_drain(tail && i == chunks - 1 ? bar(TAIL) : bar(KQ_FULL + i % kKqStages),
                                          tail && i == chunks - 1 ? 0u : (uint32_t)(i / kKqStages) & 1u, 20000000ull);
                for (int i = max(0, vs - kVStages); i < vs; ++i)
                    (void)mbar_wait_drain(tail && i == chunks - 1 ? bar(TAIL) : bar(V_FULL + i % kVStages),
                                          tail && i == chunks - 1 ? 1u : (uint32_t)(i / kVStages) & 1u, 20000000ull);
            }
            __syncwarp();
        } else {
            // ------------------------------ decays, steps and lengths ------------------------------
            const int part = warp - 14, i = 32 * part + lane;
            auto gates = [&](int c, int token) {
                const int t = c * kTok + token;
                return t < s.n ? delta_gates(a, s.t0 + t, h) : make_float2(0.0f, 0.0f);
            };
            float2 now = make_float2(0.0f, 0.0f);
            float beside = 0.0f;   // the other half's token's
            if (chunks > 0) {
                now = gates(0, i);
                beside = gates(0, i ^ 32).x;
            }
            bool ok = true;
            for (int c = 0; c < chunks; ++c) {
                const float2 gate = now;
                long long other = fixed_log2(beside);
                if (c + 1 < chunks) {
                    now = gates(c + 1, i);
                    beside = gates(c + 1, i ^ 32).x;
                }
                const int ks = c % kKqStages, cs = c % kCoefStages;
                if (!wait_warp(COEF_EMPTY + cs, ((uint32_t)(c / kCoefStages) & 1u) ^ 1u) ||
                    !wait_warp(KQ_FULL + ks, (uint32_t)(c / kKqStages) & 1u)) {
                    ok = false;
                    break;
                }
                float ik = 1.0f, iq = 1.0f;
                if (a.norm) {
                    float kk = 0.0f, qq = 0.0f;
                    const unsigned char* at = smem + C::kKq + ks * C::kKqBytes + i * 128;
                    uint64_t k2 = 0, q2 = 0;
                    for (int x = 0; x < NC; ++x, at += 2 * kTok * 128)
#pragma unroll 2
                        for (int u = 0; u < 8; ++u) {
                            const uint4 kv = *reinterpret_cast<const uint4*>(at + ((u ^ (i & 7)) << 4));
                            const uint4 qv = *reinterpret_cast<const uint4*>(at + kTok * 128 + ((u ^ (i & 7)) << 4));
                            const uint32_t kw[4] = {kv.x, kv.y, kv.z, kv.w}, qw[4] = {qv.x, qv.y, qv.z, qv.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint64_t kp = pack2(__uint_as_float(kw[e] << 16), __uint_as_float(kw[e] & 0xFFFF0000u));
                                const uint64_t qp = pack2(__uint_as_float(qw[e] << 16), __uint_as_float(qw[e] & 0xFFFF0000u));
                                k2 = fma2(kp, kp, k2);
                                q2 = fma2(qp, qp, q2);
                            }
                        }
                    float x, y;
                    unpack2(k2, x, y);
                    kk = x + y;
                    unpack2(q2, x, y);
                    qq = x + y;
                    ik = 1.0f / sqrtf(kk + kDeltaNormEps);
                    iq = 1.0f / sqrtf(qq + kDeltaNormEps);
                }
                // the running sum, in 64 bits of which 40 stand behind the point
                long long G = fixed_log2(gate.x);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long x = __shfl_up_sync(0xffffffffu, G, o);
                    if (lane >= o) G += x;
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) other += __shfl_xor_sync(0xffffffffu, other, o);
                if (part) G += other;
                const long long end = __shfl_sync(0xffffffffu, G, lane | 15);
                const long long all = __shfl_sync(0xffffffffu, G, 31) + (part ? 0 : other);
                Coef& k = coefs[cs];
                const float hi = unfixed(G), near = exp2f(hi);
                const float2 both = make_float2(hi, unfixed(G - __float2ll_rn(hi * 1099511627776.0f)));
                const float beta = fmaf(gate.x, 0.0f, gate.y);   // (a decay that is no number makes the step none)
                k.beta[i] = beta;
                k.minus_near[i] = -beta * near * ik;
                k.left[i] = exp2f(unfixed(all - G)) * ik;
                k.near_q[i] = a.scale * iq * near;
                k.beta_k[i] = beta * ik;
                k.scale_q[i] = a.scale * iq;
                k.k[i] = ik;
                k.to_end[i] = exp2f(unfixed(end - G)) * ik;
                k.G[i] = both;
                if ((lane & 15) == 15) k.end[i / 16] = both;
                if (part && lane == 31) k.last = exp2f(unfixed(all));
                arrive(COEF_FULL + cs);
            }
            if (!ok && lane == 0) fail();
            __syncwarp();
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// [T][heads * dim] as the TMA sees it, a box of `box` values of 64 tokens.
bool make_token_map(CUtensorMap* m, const __nv_bfloat16* base, long long stride, int width, int T, int box_width) {
    auto enc = get_encode();
    if (!enc) return false;
    const cuuint64_t dim[2] = {(cuuint64_t)width, (cuuint64_t)T};
    const cuuint64_t step[1] = {(cuuint64_t)(stride > width ? stride : width) * 2};   // (one token: any stride)
    const cuuint32_t box[2] = {(cuuint32_t)box_width, kTok};
    const cuuint32_t es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<__nv_bfloat16*>(base), dim, step, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, box_width == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The output, [T][heads][dv]: a box of 32 values of one head and 32 tokens; what
// lies past a head's last value is not written.
bool make_out_map(CUtensorMap* m, __nv_bfloat16* base, int heads, int dv, int T) {
    auto enc = get_encode();
    if (!enc) return false;
    const cuuint64_t dim[3] = {(cuuint64_t)dv, (cuuint64_t)heads, (cuuint64_t)T};
    const cuuint64_t step[2] = {(cuuint64_t)dv * 2, (cuuint64_t)dv * heads * 2};
    const cuuint32_t box[3] = {32, 1, 32};
    const cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dim, step, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

template <int DK>
cudaError_t launch(const DeltaArgs& a, cudaStream_t stream) {
    using C = Cfg<DK>;
    CUtensorMap mq, mk, mv, mo;
    if (!make_token_map(&mq, a.q, a.q_token, a.k_heads * DK, a.s.T, 64) ||
        !make_token_map(&mk, a.k, a.k_token, a.k_heads * DK, a.s.T, 64) ||
        !make_token_map(&mv, a.v, a.v_token, a.v_heads * a.dv, a.s.T, 32) || !make_out_map(&mo, a.out, a.v_heads, a.dv, a.s.T))
        return cudaErrorInvalidValue;
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev]) {
        const cudaError_t e =
            cudaFuncSetAttribute(delta_chunk_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    return launch_pdl(delta_chunk_kernel<DK>, dim3((unsigned)((a.dv + kRows - 1) / kRows * a.v_heads), (unsigned)a.s.B),
                      dim3(kThreads), C::kSmem, stream, true, mq, mk, mv, mo, a);
}

}  // namespace

cudaError_t launch_delta_chunk(const DeltaArgs& a, cudaStream_t stream) {
    return a.dk == 128 ? launch<128>(a, stream) : launch<64>(a, stream);
}

cudaError_t read_delta_chunk_device_error(int* code) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_delta_chunk_error, sizeof(int));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_delta_chunk_error, &zero, sizeof(int));
}

}  // namespace tern
