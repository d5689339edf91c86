// tern_norm.cu -- the norms before and after a block, fused with the residual
// stream and the block's gate.
//
//   before:  h = residual + s x,   y = h / sqrt(mean h^2 + eps) (w + c) [act(gate)]
//   after:   y = residual + s (x / sqrt(mean x^2 + eps) (w + c) [act(gate)])
//
// A row's values stay in the registers of a team of threads between the sum of
// squares and the output: every input is read once, every output written once,
// and the weight stays in registers over all rows of a team.  Bound by those
// bytes: 4096 rows of 5120 with a residual, all in bf16, 27.7 us, 6.1 TB/s, 89 % of the
// copy bandwidth; 777 rows of 4104, fp32 after a block, 7.4 us.  A call of a few rows is
// bound by its latency, 2.9 us.
#include <math.h>

#include <algorithm>

#include "tern_sm100.cuh"
#include "tern_state.cuh"

namespace tern {
namespace {

__device__ int g_norm_error;

constexpr int kMaxDim = 32768;

struct NormArgs {
    const void *x, *residual, *gate;
    const float* weight;
    void *out, *residual_out;
    long long x_token, x_head, r_token, r_head, g_token, g_head;   // strides in elements
    int x_f32, r_f32, g_f32, out_f32;
    int heads, dim, rows, after, sigmoid_gate;
    unsigned div, shift;   // row / heads = umulhi(row, div) >> shift
    float scale, eps, offset, part, whole;   // part: 2^-k >= 1 / (2 dim); whole: 2^k / dim
};

// The types and forms that a kernel is made for, with which its loops have no choices left: heads'
// outputs in bf16 with a gate of 16 or 32 bits or none; before a block, ungated, all in bf16
// or from fp32; after one, in fp32; everything else as the arguments say.  2048 x 48 heads of
// 128 under a bf16 gate 10.5 us so, 14.4 by kAny; 4096 rows of 5120 before a block 27.4
// and 28.9, 777 of 4104 after one 7.2 and 7.7.
enum NormKind { kAny, kHeads, kHeadsGate16, kHeadsGate32, kBefore16, kBefore32, kAfter32 };
template <int KIND>
__device__ __forceinline__ NormArgs made_for(NormArgs a) {
    if (KIND == kHeads || KIND == kHeadsGate16 || KIND == kHeadsGate32) {
        a.x_f32 = a.out_f32 = a.after = 0;
        a.residual = nullptr;
        a.residual_out = nullptr;
        if (KIND == kHeads) a.gate = nullptr;
        a.g_f32 = KIND == kHeadsGate32;
    }
    if (KIND == kBefore16 || KIND == kBefore32) {
        a.x_f32 = a.r_f32 = KIND == kBefore32;
        a.out_f32 = a.after = 0;
        a.gate = nullptr;
    }
    if (KIND == kAfter32) {
        a.x_f32 = a.r_f32 = a.out_f32 = a.after = 1;
        a.residual_out = nullptr;
    }
    return a;
}
inline NormKind norm_kind(const NormArgs& a) {
    if (a.after) return a.x_f32 && a.residual && a.r_f32 && a.out_f32 ? kAfter32 : kAny;
    if (a.out_f32) return kAny;
    if (a.residual) return a.gate || a.x_f32 != a.r_f32 ? kAny : a.x_f32 ? kBefore32 : kBefore16;
    return a.x_f32 ? kAny : !a.gate ? kHeads : a.g_f32 ? kHeadsGate32 : kHeadsGate16;
}

__device__ __forceinline__ float act(float z, int only_sigmoid) {
    const float s = sigmoid(z);
    return only_sigmoid ? s : z * s;
}

struct NormRow {
    long long x, r, g;
};
__device__ __forceinline__ NormRow norm_row(const NormArgs& a, int row) {
    const int t = a.heads == 1 ? row : (int)(__umulhi((unsigned)row, a.div) >> a.shift), h = row - t * a.heads;
    return NormRow{t * a.x_token + h * a.x_head, t * a.r_token + h * a.r_head, t * a.g_token + h * a.g_head};
}

// One piece of 8 values of one row.
struct NormPiece {
    Raw8 x, r, g;
};
__device__ __forceinline__ void load_piece(const NormArgs& a, const NormRow& at, int d, NormPiece& p) {
    p.x = load_raw8(a.x, at.x + d, a.x_f32);
    if (a.residual) p.r = load_raw8(a.residual, at.r + d, a.r_f32);
    if (a.gate) p.g = load_raw8(a.gate, at.g + d, a.g_f32);
}
// The values that the norm is taken of, and their squares added to `sum`, each
// times a.part, the power of two next to 1 / dim: a sum overflows only where the
// mean does.
__device__ __forceinline__ void open_piece(const NormArgs& a, const NormPiece& p, float (&h)[8], float& sum) {
    widen8(p.x, a.x_f32, h);
    if (!a.after && a.residual) {
        float r[8];
        widen8(p.r, a.r_f32, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = fmaf(a.scale, h[e], r[e]);
    }
    uint64_t s = pack2(sum, 0.0f);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const uint64_t v = pack2(h[e], h[e + 1]);
        s = fma2(mul2(v, pack2(a.part, a.part)), v, s);
    }
    float odd;
    unpack2(s, sum, odd);
    sum += odd;
}
__device__ __forceinline__ void close_piece(const NormArgs& a, const NormPiece& p, long long out, float inv,
                                            const float (&w)[8], float (&h)[8]) {
    if (a.residual_out) store_raw8(a.residual_out, out, a.r_f32, h);
#pragma unroll
    for (int e = 0; e < 8; e += 2)
        unpack2(mul2(mul2(pack2(h[e], h[e + 1]), pack2(inv, inv)), pack2(w[e], w[e + 1])), h[e], h[e + 1]);
    if (a.gate) {
        float z[8];
        widen8(p.g, a.g_f32, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] *= act(z[e], a.sigmoid_gate);
    }
    if (a.after) {
        float r[8] = {};
        if (a.residual) widen8(p.r, a.r_f32, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = fmaf(a.scale, h[e], r[e]);
    }
    store_raw8(a.out, out, a.out_f32, h);
}
__device__ __forceinline__ void load_weight(const NormArgs& a, int d, float (&w)[8]) {
    widen8(load_raw8(a.weight, d, 1), 1, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] += a.offset;
}

// Rows of up to 512 values: a team of TEAM lanes of a warp holds ROWS rows at a
// time, PIECES pieces of each a lane.
template <int TEAM, int PIECES, int ROWS, int KIND>
__global__ void __launch_bounds__(256) norm_warp_kernel(const NormArgs args) {
    const NormArgs a = made_for<KIND>(args);
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x % TEAM, pieces = a.dim / 8;
    const int first = (blockIdx.x * (256 / TEAM) + threadIdx.x / TEAM) * ROWS;
    NormPiece p[ROWS][PIECES];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        if (first + r >= a.rows) break;
        const NormRow at = norm_row(a, first + r);
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
            if (lane + i * TEAM < pieces) load_piece(a, at, 8 * (lane + i * TEAM), p[r][i]);
    }
    float w[PIECES][8];
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
        if (lane + i * TEAM < pieces) load_weight(a, 8 * (lane + i * TEAM), w[i]);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const bool live = first + r < a.rows;   // (a team past the end still takes part in its warp's sums)
        float h[PIECES][8], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
            if (live && lane + i * TEAM < pieces) open_piece(a, p[r][i], h[i], sum);
#pragma unroll
        for (int o = TEAM / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float inv = rsqrtf(fmaf(sum, a.whole, a.eps));
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
            if (live && lane + i * TEAM < pieces)
                close_piece(a, p[r][i], (long long)(first + r) * a.dim + 8 * (lane + i * TEAM), inv, w[i], h[i]);
    }
}

// Longer rows: CTAs that stay, with their rows' values some rows ahead on the way to a
// ring in shared memory, a bulk copy an input and row.  (With the next row's values in
// registers instead, 4096 rows of 5120 took 67 us; a CTA a row 43.)
constexpr int kStreamBytes = 200 * 1024;   // of an SM's shared memory

// After a wait that gave up, where nothing more is fetched: waits for the copies still on their way
// to the `left` stages from `stage` on, so that none lands in shared memory that is another CTA's by then.
__device__ __noinline__ void ring_drain(const uint64_t* full, int stages, int stage, uint32_t phase, int left, uint64_t limit_ns) {
    for (; left > 0; --left) {
        (void)sm100::mbar_wait_drain(sm100::smem_u32(&full[stage]), phase, limit_ns);
        if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
        }
    }
}
constexpr uint64_t kStreamDrainNs = 20000000;

struct NormRing {
    int stages, row_bytes, r_at, g_at;   // a stage: x, then the residual, then the gate
};

__device__ __forceinline__ Raw8 shared_raw8(const unsigned char* row, int d, int is_f32) {
    Raw8 r;
    if (is_f32) {
        const uint4* p = reinterpret_cast<const uint4*>(row + 4 * d);
        r.a = p[0];
        r.b = p[1];
    } else {
        r.a = *reinterpret_cast<const uint4*>(row + 2 * d);
        r.b = make_uint4(0, 0, 0, 0);
    }
    return r;
}

template <int THREADS, int PIECES, int CTAS, int KIND>
__global__ void __launch_bounds__(THREADS, CTAS) norm_stream_kernel(const NormArgs args, const NormRing ring) {
    const NormArgs a = made_for<KIND>(args);
    extern __shared__ __align__(128) unsigned char rows[];
    __shared__ __align__(8) uint64_t full[16];
    __shared__ float part[2][THREADS / 32];
    constexpr int n = THREADS;
    const int pieces = a.dim / 8;
    if (threadIdx.x == 0) {
        for (int i = 0; i < ring.stages; ++i) sm100::mbar_init(sm100::smem_u32(&full[i]), 1);
        sm100::fence_barrier_init();
    }
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();
    auto fetch = [&](int row, int stage) {   // one thread
        const NormRow at = norm_row(a, row);
        const uint32_t to = sm100::smem_u32(rows + stage * ring.row_bytes), bar = sm100::smem_u32(&full[stage]);
        const uint32_t xb = a.dim * (a.x_f32 ? 4 : 2), rb = a.residual ? a.dim * (a.r_f32 ? 4 : 2) : 0, gb = a.gate ? a.dim * (a.g_f32 ? 4 : 2) : 0;
        sm100::mbar_arrive_expect_tx(bar, xb + rb + gb);
        sm100::bulk_load(to, static_cast<const unsigned char*>(a.x) + at.x * (a.x_f32 ? 4 : 2), xb, bar);
        if (rb) sm100::bulk_load(to + ring.r_at, static_cast<const unsigned char*>(a.residual) + at.r * (a.r_f32 ? 4 : 2), rb, bar);
        if (gb) sm100::bulk_load(to + ring.g_at, static_cast<const unsigned char*>(a.gate) + at.g * (a.g_f32 ? 4 : 2), gb, bar);
    };
    const int step = gridDim.x, count = (a.rows - 1 - (int)blockIdx.x) / step + 1;   // rows of this CTA
    if (threadIdx.x == 0)
        for (int i = 0; i < ring.stages && i < count; ++i) fetch(blockIdx.x + i * step, i);
    float w[PIECES][8];
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
        if (threadIdx.x + i * n < pieces) load_weight(a, 8 * (threadIdx.x + i * n), w[i]);
    int stage = 0;
    uint32_t phase = 0;
    for (int k = 0; k < count; ++k) {
        const int row = blockIdx.x + k * step;
        const bool landed = wait_tries(sm100::smem_u32(&full[stage]), phase, kWaitTries);
        const unsigned char* src = rows + stage * ring.row_bytes;
        NormPiece p[PIECES];
        float h[PIECES][8], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int d = 8 * (threadIdx.x + i * n);
            if (d < a.dim) {
                p[i].x = shared_raw8(src, d, a.x_f32);
                if (a.residual) p[i].r = shared_raw8(src + ring.r_at, d, a.r_f32);
                if (a.gate) p[i].g = shared_raw8(src + ring.g_at, d, a.g_f32);
                open_piece(a, p[i], h[i], sum);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (threadIdx.x % 32 == 0) part[k & 1][threadIdx.x / 32] = sum;
        // (two sets of parts: a warp may be a row ahead, never two)
        if (!__syncthreads_and(landed)) {   // one thread's wait gave up: the CTA ends here
            if (threadIdx.x == 0) {
                report_device_error(&g_norm_error, TERN_DEVERR_NORM_WAIT);
                ring_drain(full, ring.stages, stage, phase, min(ring.stages, count - k), kStreamDrainNs);
            }
            return;
        }
        if (threadIdx.x == 0 && k + ring.stages < count) fetch(row + ring.stages * step, stage);
        sum = threadIdx.x % 32 < n / 32 ? part[k & 1][threadIdx.x % 32] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float inv = rsqrtf(fmaf(sum, a.whole, a.eps));
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int d = 8 * (threadIdx.x + i * n);
            if (d < a.dim) close_piece(a, p[i], (long long)row * a.dim + d, inv, w[i], h[i]);
        }
        if (++stage == ring.stages) {
            stage = 0;
            phase ^= 1u;
        }
    }
}

// Calls of a few rows, where the ring would only be in the way, and rows past 10240 values:
// a CTA a row, the first 5120 values in registers, those past them read again.
constexpr int kRowThreads = 640;
__global__ void __launch_bounds__(kRowThreads) norm_row_kernel(const NormArgs a) {
    __shared__ float part[kRowThreads / 32];
    pdl_launch_dependents();
    pdl_wait();
    const NormRow at = norm_row(a, blockIdx.x);
    const int first = 8 * threadIdx.x;
    const long long out = (long long)blockIdx.x * a.dim;
    float sum = 0.0f, h[8], w[8];
    NormPiece p;
    if (first < a.dim) {
        load_piece(a, at, first, p);
        load_weight(a, first, w);
        open_piece(a, p, h, sum);
    }
    for (int d = first + 8 * kRowThreads; d < a.dim; d += 8 * kRowThreads) {
        NormPiece q;
        float g[8];
        load_piece(a, at, d, q);
        open_piece(a, q, g, sum);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
    __syncthreads();
    sum = threadIdx.x % 32 < blockDim.x / 32 ? part[threadIdx.x % 32] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = rsqrtf(fmaf(sum, a.whole, a.eps));
    if (first < a.dim) close_piece(a, p, out + first, inv, w, h);
    for (int d = first + 8 * kRowThreads; d < a.dim; d += 8 * kRowThreads) {
        NormPiece q;
        float g[8], unused = 0.0f;
        load_piece(a, at, d, q);
        load_weight(a, d, w);
        open_piece(a, q, g, unused);
        close_piece(a, q, out + d, inv, w, g);
    }
}

// The ring's wait, of a CTA of two warps: of four rows through two stages the third never comes
// (one copy of 16 bytes lands, 16 bytes more are waited for).
__global__ void __launch_bounds__(64) norm_wait_selftest_kernel(uint32_t tries, uint64_t limit_ns, const int* from) {
    __shared__ __align__(16) unsigned char rows[2][16];
    __shared__ __align__(8) uint64_t full[2];
    constexpr int kRows = 4;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) sm100::mbar_init(sm100::smem_u32(&full[i]), 1);
        sm100::fence_barrier_init();
    }
    __syncthreads();
    auto fetch = [&](int k) {
        const uint32_t bar = sm100::smem_u32(&full[k & 1]);
        sm100::mbar_arrive_expect_tx(bar, k == 2 ? 32 : 16);
        sm100::bulk_load(sm100::smem_u32(rows[k & 1]), from, 16, bar);
    };
    if (threadIdx.x == 0) {
        fetch(0);
        fetch(1);
    }
    for (int k = 0; k < kRows; ++k) {
        const bool landed = wait_tries(sm100::smem_u32(&full[k & 1]), k / 2, tries);
        if (!__syncthreads_and(landed)) {
            if (threadIdx.x == 0) {
                report_device_error(&g_norm_error, TERN_DEVERR_NORM_WAIT);
                ring_drain(full, 2, k & 1, k / 2, min(2, kRows - k), limit_ns);
            }
            return;
        }
        if (threadIdx.x == 0 && k + 2 < kRows) fetch(k + 2);
    }
}

template <int TEAM, int PIECES, int ROWS>
cudaError_t launch_warp(const NormArgs& a, cudaStream_t stream) {
    const int per = 256 / TEAM * ROWS;
    const NormKind kind = norm_kind(a);
    auto kernel = kind == kHeads         ? norm_warp_kernel<TEAM, PIECES, ROWS, kHeads>
                  : kind == kHeadsGate16 ? norm_warp_kernel<TEAM, PIECES, ROWS, kHeadsGate16>
                  : kind == kHeadsGate32 ? norm_warp_kernel<TEAM, PIECES, ROWS, kHeadsGate32>
                                         : norm_warp_kernel<TEAM, PIECES, ROWS, kAny>;
    return launch_pdl(kernel, dim3((a.rows + per - 1) / per), dim3(256), 0, stream, true, a);
}
template <int THREADS, int PIECES, int CTAS>
cudaError_t launch_stream(const NormArgs& a, int sms, cudaStream_t stream) {
    NormRing r;
    auto bytes = [&](const void* p, int f32) { return p ? (a.dim * (f32 ? 4 : 2) + 127) / 128 * 128 : 0; };
    r.r_at = bytes(a.x, a.x_f32);
    r.g_at = r.r_at + bytes(a.residual, a.r_f32);
    r.row_bytes = r.g_at + bytes(a.gate, a.g_f32);
    r.stages = std::min(kStreamBytes / CTAS / r.row_bytes, 16);
    const NormKind kind = norm_kind(a);
    auto kernel = kind == kBefore16   ? norm_stream_kernel<THREADS, PIECES, CTAS, kBefore16>
                  : kind == kBefore32 ? norm_stream_kernel<THREADS, PIECES, CTAS, kBefore32>
                  : kind == kAfter32  ? norm_stream_kernel<THREADS, PIECES, CTAS, kAfter32>
                                      : norm_stream_kernel<THREADS, PIECES, CTAS, kAny>;
    static bool attr_set[64][kAfter32 + 1] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev][kind]) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamBytes / CTAS);
        if (e != cudaSuccess) return e;
        attr_set[dev][kind] = true;
    }
    return launch_pdl(kernel, dim3(std::min(a.rows, CTAS * sms)), dim3(THREADS), (size_t)r.stages * r.row_bytes, stream, true, a, r);
}

__device__ __align__(16) int g_norm_selftest[4];

}  // namespace

cudaError_t launch_norm_wait_selftest(uint64_t limit_ns, cudaStream_t stream) {
    void* from = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&from, g_norm_selftest);
    if (e != cudaSuccess) return e;
    const uint64_t tries = limit_ns / kWaitNap;
    norm_wait_selftest_kernel<<<1, 64, 0, stream>>>(tries > 0 ? (uint32_t)tries : 1u, limit_ns, static_cast<const int*>(from));
    return cudaGetLastError();
}

cudaError_t read_norm_device_error(int* code) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_norm_error, sizeof(int));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_norm_error, &zero, sizeof(int));
}

}  // namespace tern

using namespace tern;

extern "C" tern_status tern_rms_norm(const void* x, int x_is_f32, long long x_token, long long x_head,
                                     const void* residual, int residual_is_f32, long long residual_token,
                                     long long residual_head, const void* gate, int gate_is_f32, long long gate_token,
                                     long long gate_head, int gate_act, const float* weight, float weight_offset,
                                     float scale, float eps, int after, int T, int heads, int dim, void* out,
                                     int out_is_f32, void* residual_out, tern_stream_t stream) {
    set_launch_count(0);
    if (T < 0 || heads < 1 || heads > 65535 || (long long)T * heads > (1LL << 30) || dim < 8 || dim % 8 != 0 || dim > kMaxDim)
        return TERN_ERR_SHAPE;
    const long long strides[6] = {x_token, x_head, residual_token, residual_head, gate_token, gate_head};
    for (long long s : strides)
        if (s < 0 || s % 8 != 0 || s >= (1LL << 37)) return TERN_ERR_SHAPE;
    if ((gate_act != TERN_GATE_SILU && gate_act != TERN_GATE_SIGMOID) || !(eps >= 0.0f) || (after && residual_out) ||
        (residual_out && !residual))
        return TERN_ERR_SHAPE;
    if (!weight || (T > 0 && (!x || !out))) return TERN_ERR_NULL;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(gate) || !aligned16(weight) || !aligned16(out) ||
        !aligned16(residual_out))
        return TERN_ERR_ALIGN;
    int sms = 0;
    const tern_status st = check_device(&sms);
    if (st != TERN_OK) return st;
    if (T == 0) return TERN_OK;
    int k = 0, b = 0;
    while (1 << k < dim) ++k;
    while (1 << b < heads) ++b;
    // (exact for rows below 2^31: 2^b < 2 heads)
    const unsigned div = (unsigned)(((1ull << (31 + b)) + heads - 1) / heads);
    const NormArgs a{x, residual, gate, weight, out, residual_out, x_token, x_head, residual_token, residual_head,
                     gate_token, gate_head, x_is_f32, residual_is_f32, gate_is_f32, out_is_f32, heads, dim, T * heads,
                     after, gate_act == TERN_GATE_SIGMOID, div, b > 0 ? (unsigned)b - 1 : 0u, scale, eps, weight_offset,
                     ldexpf(1.0f, -k), (float)(1 << k) / (float)dim};
    auto* s = (cudaStream_t)stream;
    const cudaError_t e = dim <= 64     ? launch_warp<8, 1, 2>(a, s)
                          : dim <= 128  ? launch_warp<16, 1, 2>(a, s)
                          : dim <= 256  ? launch_warp<32, 1, 2>(a, s)
                          : dim <= 512  ? launch_warp<32, 2, 1>(a, s)
                          : dim > 10240 || a.rows <= 2 * sms ? launch_pdl(norm_row_kernel, dim3(a.rows), dim3(std::min((dim / 8 + 31) / 32 * 32, kRowThreads)), 0, s, true, a)
                          : dim <= 2560 ? launch_stream<320, 1, 2>(a, sms, s)
                          : dim <= 5120 ? launch_stream<320, 2, 2>(a, sms, s)
                                        : launch_stream<640, 2, 1>(a, sms, s);
    if (e != cudaSuccess) return TERN_ERR_CUDA;
    set_launch_count(1);
    return TERN_OK;
}
