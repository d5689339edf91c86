// tern_delta_join.cu -- sequences of the gated delta rule that went in pieces, joined.
//
// Of each piece behind the first there are B, its last state from S = 0, M, what it does
// to any state (a row of it for each row of the unit matrix), and the outputs of both.
// One kind of CTA makes the states between the pieces, S <- S M + B one after the other,
// another the outputs, out = out_B + S out_M, chunk by chunk.  Both are tcgen05 products of
// 128 rows of S, a tensor memory lane a row; S, M and out_M are two bf16 parts each (2^-17),
// taken without the smallest product, and lie in memory as shared memory wants them, so
// that a bulk copy brings each.
//
// What bounds it is latency: a copy, a product and its rows' way out for a CTA's first chunk,
// then the copies of 64 KB a chunk and the products' issue; 32 heads, 16 chunks each: 13 us
// (40 MB from L2), of which the states, on CTAs of their own, are hidden but for the last.
#include "tern_delta.cuh"
#include "tern_sm100.cuh"

namespace tern {
namespace {

using namespace sm100;

__device__ int g_delta_join_error;

// 16 warps for rows and values, four a row, and one for copies and products
constexpr int kJoinThreads = 17 * 32, kRows = kDeltaRows, kTok = kDeltaChunk;

// Shared memory: parts of S; two stages, each of either a chunk's out_M and out_B or of M
template <int DK>
struct Shared {
    static constexpr uint32_t kS = delta_parts_bytes(kRows, DK), kO = delta_parts_bytes(kTok, DK), kLocal = kRows * kTok * 4;
    static constexpr uint32_t kStage = kO + kLocal, kBar = kS + 2 * kStage, kSmem = kBar + 64 + 1024;
    static_assert(delta_parts_bytes(DK, DK) <= kStage, "M in a stage");
};

// What both kinds of CTA have.
template <int DK>
struct Join {
    using L = Shared<DK>;
    const DeltaArgs& a;
    const StateSeq& s;
    unsigned char* smem;
    uint32_t base;
    int b, h, tile, warp, lane, per, used;   // per: tokens of a piece, used: pieces of this sequence
    bool ok = true;
    int begun = 0;   // copies to the stages, one after the other (in the warp that waits for them)

    __device__ __forceinline__ uint32_t copied(int stage) const { return base + L::kBar + 8 * stage; }
    __device__ __forceinline__ uint32_t done(int stage) const { return base + L::kBar + 16 + 8 * stage; }
    __device__ __forceinline__ uint32_t read(int stage) const { return base + L::kBar + 32 + 8 * stage; }
    __device__ __forceinline__ uint32_t stage(int i) const { return base + L::kS + (i & 1) * L::kStage; }
    __device__ __forceinline__ uint32_t drained() const { return base + L::kBar + 56; }
    // A role that gives up goes to close(): nothing is copied or issued after it.
    __device__ __forceinline__ bool need(uint32_t bar, int i) { return ok = wait_warp(bar, (uint32_t)(i >> 1) & 1u); }
    __device__ __forceinline__ void arrive(uint32_t bar) const {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    }
    __device__ __forceinline__ const unsigned char* parts(int piece) const {
        return delta_parts(a.p, b, a.v_heads, h, DK, (a.dv + kRows - 1) / kRows, tile, piece);
    }
    // Barriers and `cols` columns of tensor memory for the CTA; `first` begins its copies.
    template <class F>
    __device__ __forceinline__ uint32_t open(F first) {
        if (threadIdx.x == 0) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(copied(i), 1);
                mbar_init(done(i), 1);
                mbar_init(read(i), 16);
            }
            mbar_init(drained(), 1);
            fence_barrier_init();
            first();
        }
        if (warp == 0) {
            __syncwarp();
            tmem_alloc(base + L::kBar + 48, 128);
            tmem_relinquish();
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        pdl_launch_dependents();   // (the next kernel may want tensor memory: not before this one has its own)
        return *reinterpret_cast<volatile uint32_t*>(smem + L::kBar + 48);
    }
    __device__ __forceinline__ void close(uint32_t tmem) {
        if (!ok && lane == 0) report_device_error(&g_delta_join_error, TERN_DEVERR_DELTA_WAIT);
        tc_fence_before();
        if (!__syncthreads_and(ok)) {   // a wait gave up: what is on its way ends before the CTA does
            if (warp == 16 && elect_one()) {
                for (int i = max(0, begun - 2); i < begun; ++i)
                    (void)mbar_wait_drain(copied(i & 1), (uint32_t)(i >> 1) & 1u, 20000000ull);
                mma_commit(drained());
                (void)mbar_wait_drain(drained(), 0u, 100000000ull);
            }
            __syncthreads();
        }
        if (warp == 0) {
            tc_fence_after();
            tmem_dealloc(tmem, 128);
        }
    }
    // The three products of the parts of S with those of a [N][DK] or, MN, [DK][N] matrix.
    template <int N, bool MN>
    __device__ __forceinline__ void product(uint32_t to, uint32_t with) {
        constexpr uint32_t kIdesc = idesc_bf16_f32(kRows, N) | (MN ? kIdescBMnMajor : 0u), kPart = (uint32_t)N * DK * 2;
#pragma unroll 1
        for (int part = 0; part < 3; ++part) {   // hi hi, lo hi, hi lo
            const uint32_t x = base + (part == 1 ? L::kS / 2 : 0u), y = with + (part == 2 ? kPart : 0u);
#pragma unroll
            for (int k = 0; k < DK / 16; ++k)
                mma_f16_ss(to, smem_desc_k_sw128(x + (k / 4) * (kRows * 128)) + 2 * (k % 4),
                           MN ? smem_desc_mn_sw128(y + 2048u * k, DK * 128) : smem_desc_k_sw128(y + (k / 4) * (N * 128)) + 2 * (k % 4),
                           kIdesc, part > 0 || k > 0);
        }
    }

    // The states behind the pieces, 128 rows; the last goes to the pool.
    __device__ __forceinline__ void states() {
        const long long at = (long long)b * a.v_heads + h;
        const unsigned char* move = a.p.move + at * (a.p.count - 1) * delta_parts_bytes(DK, DK);
        constexpr uint32_t kM = delta_parts_bytes(DK, DK);
        const uint32_t tmem = open([&] {
            mbar_arrive_expect_tx(copied(0), L::kS + kM);
            bulk_load(base, parts(0), L::kS, copied(0));
            bulk_load(stage(0), move, kM, copied(0));
        });
        if (warp == 16) {
            begun = 1;
#pragma unroll 1
            for (int i = 0; i + 1 < used; ++i) {
                // S is there, the columns are free, and M before the last is done with
                if (i > 0 && !need(read(i - 1 & 1), i - 1)) break;
                if (i + 2 < used) {
                    if (lane == 0) {
                        mbar_arrive_expect_tx(copied(i + 1 & 1), kM);
                        bulk_load(stage(i + 1), move + (i + 1) * (long long)kM, kM, copied(i + 1 & 1));
                    }
                    ++begun;
                    __syncwarp();
                }
                if (!need(copied(i & 1), i)) break;
                tc_fence_after();
                if (elect_one()) {
                    product<DK, true>(tmem, stage(i));
                    mma_commit(done(i & 1));
                }
                __syncwarp();
            }
        } else {
            constexpr int kCols = DK / 4, kAt = 16;   // of a thread; at once
            const int row = 32 * (warp & 3) + lane, col0 = kCols * (warp >> 2);
            const bool live = kRows * tile + row < a.dv;
#pragma unroll 1
            for (int i = 0; i + 1 < used; ++i) {
                const float* from = a.p.state + ((at * a.p.count + i + 1) * a.dv + kRows * tile + row) * DK + col0;
                const bool last = i + 2 == used;
                float* to = a.state + (((long long)max(s.dst, 0) * a.v_heads + h) * a.dv + kRows * tile + row) * DK + col0;
                float v[kCols];
#pragma unroll
                for (int e = 0; e < kCols; e += 4) {
                    const float4 x = live ? *reinterpret_cast<const float4*>(from + e) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    v[e] = x.x, v[e + 1] = x.y, v[e + 2] = x.z, v[e + 3] = x.w;
                }
                if (!need(done(i & 1), i)) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < kCols; c += kAt) {
                    uint32_t d[kAt];
                    tmem_ld_x16(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)(col0 + c), d);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < kAt; ++e) v[c + e] += __uint_as_float(d[e]);
                }
                if (last) {
                    if (live && s.dst >= 0)
#pragma unroll
                        for (int e = 0; e < kCols; e += 4) *reinterpret_cast<float4*>(to + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                } else {
#pragma unroll
                    for (int e = 0; e < kCols; e += 8) put_parts8(smem, kRows, DK, row, col0 + e, v + e);
                    fence_proxy_async_smem();
                    tc_fence_before();
                    arrive(read(i & 1));
                    if (live)
#pragma unroll
                        for (int e = 0; e < kCols; e += 8)
                            put_parts8(const_cast<unsigned char*>(parts(i + 1)), kRows, DK, row, col0 + e, v + e);
                }
            }
        }
        close(tmem);
    }

    // The outputs of up to `count` chunks of a piece from its chunk `chunk` on, 128 rows.
    __device__ __forceinline__ void outs(int piece, int chunk, int count) {
        const int first = per * piece + kTok * chunk, left = min(per * (piece + 1), s.n) - first;   // this CTA's tokens
        const int chunks = min(count, (left + kTok - 1) / kTok), width = min(kRows, a.dv - kRows * tile);
        if (chunks <= 0) return;
        const long long at = (delta_piece_chunk(a.p.count, s.t0, b) + (first - per) / kTok) * a.v_heads + h;
        auto copy = [&](int i) {
            const uint32_t bar = copied(i & 1);
            mbar_arrive_expect_tx(bar, L::kO + (uint32_t)(width * kTok * 4) + (i == 0 ? L::kS : 0u));
            if (i == 0) bulk_load(base, parts(piece - 1), L::kS, bar);
            const long long x = at + (long long)i * a.v_heads;
            bulk_load(stage(i), a.p.out_move + x * L::kO, L::kO, bar);
            bulk_load(stage(i) + L::kO, a.p.out + (x * a.dv + kRows * tile) * kTok, (uint32_t)(width * kTok * 4), bar);
        };
        const uint32_t tmem = open([&] {
            copy(0);
            if (chunks > 1) copy(1);
        });
        if (warp == 16) {
            begun = min(2, chunks);
#pragma unroll 1
            for (int i = 0; i < chunks; ++i) {
                if (!need(copied(i & 1), i)) break;
                tc_fence_after();
                if (elect_one()) {
                    product<kTok, false>(tmem + kTok * (i & 1), stage(i));
                    mma_commit(done(i & 1));
                }
                __syncwarp();
                if (i > 0 && i + 1 < chunks) {   // the chunk before has left its stage and its columns
                    if (!need(read(i - 1 & 1), i - 1)) break;
                    if (lane == 0) copy(i + 1);
                    ++begun;
                    __syncwarp();
                }
            }
        } else {
            // this thread's row of S and quarter of a chunk's tokens
            const int row = 32 * (warp & 3) + lane, quarter = 16 * (warp >> 2);
            const long long step = (long long)a.v_heads * a.dv;
#pragma unroll 1
            for (int i = 0; i < chunks; ++i) {
                if (!need(copied(i & 1), i)) break;   // (for out_B)
                const float* local = reinterpret_cast<const float*>(smem + (stage(i) - base) + L::kO) + quarter * width + min(row, width - 1);
                float v[16];
#pragma unroll
                for (int t = 0; t < 16; ++t) v[t] = local[t * width];
                if (!need(done(i & 1), i)) break;
                tc_fence_after();
                uint32_t d[16];
                tmem_ld_x16(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)(kTok * (i & 1) + quarter), d);
                tmem_ld_wait();
                tc_fence_before();
                arrive(read(i & 1));
                const int n = row < width ? left - kTok * i - quarter : 0;
                __nv_bfloat16* to = a.out + (s.t0 + first + kTok * i + quarter) * step + (long long)h * a.dv + kRows * tile + row;
#pragma unroll
                for (int t = 0; t < 16; ++t, to += step)
                    if (t < n) *to = __float2bfloat16(__uint_as_float(d[t]) + v[t]);
            }
        }
        close(tmem);
    }
};

// Along x stand the CTAs of the states (`states`: one or none), then `ctas` of the outputs of each piece
// behind the first, `count` chunks each.  Both at once where neither waits for the other: with two
// pieces, whose only state between them is the first's own.
template <int DK>
__global__ void __launch_bounds__(kJoinThreads, 1)
delta_join_kernel(const DeltaArgs a, int states, int ctas, int count) {
    extern __shared__ __align__(1024) unsigned char smem_dyn[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
    pdl_wait();
    const StateSeq s = load_state_seq(a.s, blockIdx.z, &g_delta_join_error);
    const int per = delta_piece_chunks(a.p, s.n) * kTok, x = (int)blockIdx.x - states;
    if (s.n <= per) return;   // one piece: nothing to join
    Join<DK> join{a, s, smem, smem_u32(smem), (int)blockIdx.z, (int)blockIdx.y % a.v_heads, (int)blockIdx.y / a.v_heads,
                  (int)threadIdx.x >> 5, (int)threadIdx.x & 31, per, (s.n + per - 1) / per};
    if (x < 0) join.states();
    else join.outs(1 + x / ctas, x % ctas * count, count);
}

template <int DK>
cudaError_t launch(const DeltaArgs& a, int sms, cudaStream_t stream) {
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    constexpr uint32_t kSmem = Shared<DK>::kSmem;
    if (!attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(delta_join_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    const int y = (a.dv + kRows - 1) / kRows * a.v_heads, z = a.s.B, pieces = a.p.count - 1;
    const int chunks = (a.s.max_new + kTok - 1) / kTok, per = (chunks + pieces) / a.p.count;
    // as many CTAs for the outputs as are on the SMs at once
    const int room = sms - (pieces == 1 ? y * z : 0), most = room / (y * z * pieces);
    const int count = most > 0 ? (per + most - 1) / most : per, ctas = (per + count - 1) / count;
    if (pieces > 1) {
        const cudaError_t e = launch_pdl(delta_join_kernel<DK>, dim3(1, y, z), dim3(kJoinThreads), kSmem, stream, true, a, 1, ctas, count);
        if (e != cudaSuccess) return e;
    }
    const int states = pieces == 1 ? 1 : 0;
    return launch_pdl(delta_join_kernel<DK>, dim3(states + ctas * pieces, y, z), dim3(kJoinThreads), kSmem, stream, true, a, states, ctas, count);
}

}  // namespace

cudaError_t launch_delta_join(const DeltaArgs& a, int sms, cudaStream_t stream) {
    return a.dk == 128 ? launch<128>(a, sms, stream) : launch<64>(a, sms, stream);
}

cudaError_t read_delta_join_device_error(int* code) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_delta_join_error, sizeof(int));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_delta_join_error, &zero, sizeof(int));
}

}  // namespace tern
