// tern_norm.cu -- the norms before and after a block, fused with the residual
// stream and the block's gate.
//
//   before:  h = residual + s x,   y = h / sqrt(mean h^2 + eps) (w + c) [act(gate)]
//   after:   y = residual + s (x / sqrt(mean x^2 + eps) (w + c) [act(gate)])
//
// A row's values stay in the registers of a team of threads between the sum of
// squares and the output: every input is read once, every output written once,
// and the weight stays in registers over all rows of a team.  Bound by those
// bytes; a call of a few rows by its latency.
#include <math.h>

#include "tern_state.cuh"

namespace tern {
namespace {

constexpr int kMaxDim = 32768;

struct NormArgs {
    const void *x, *residual, *gate;
    const float* weight;
    void *out, *residual_out;
    long long x_token, x_head, r_token, r_head, g_token, g_head;   // strides in elements
    int x_f32, r_f32, g_f32, out_f32;
    int heads, dim, rows, after, sigmoid_gate;
    float scale, eps, offset, part, whole;   // part: 2^-k >= 1 / (2 dim); whole: 2^k / dim
};

__device__ __forceinline__ float act(float z, int only_sigmoid) {
    const float s = sigmoid(z);
    return only_sigmoid ? s : z * s;
}

struct NormRow {
    long long x, r, g;
};
__device__ __forceinline__ NormRow norm_row(const NormArgs& a, int row) {
    const int t = a.heads == 1 ? row : (int)((unsigned)row / (unsigned)a.heads), h = row - t * a.heads;
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
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(h[e] * a.part, h[e], sum);
}
__device__ __forceinline__ void close_piece(const NormArgs& a, const NormPiece& p, long long out, float inv,
                                            const float (&w)[8], float (&h)[8]) {
    if (a.residual_out) store_raw8(a.residual_out, out, a.r_f32, h);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = h[e] * inv * w[e];
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

// Rows of up to 1024 values: a team of TEAM lanes of a warp holds ROWS rows at a
// time, PIECES pieces of each a lane.
template <int TEAM, int PIECES, int ROWS>
__global__ void __launch_bounds__(256) norm_warp_kernel(const NormArgs a) {
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

// Longer rows: a CTA a row, the next row's values on their way while this one's
// sum is formed.
template <int PIECES>
__global__ void __launch_bounds__(1024) norm_cta_kernel(const NormArgs a) {
    __shared__ float part[2][32];
    pdl_launch_dependents();
    pdl_wait();
    const int n = blockDim.x, pieces = a.dim / 8, warps = n / 32;
    float w[PIECES][8];
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
        if (threadIdx.x + i * n < pieces) load_weight(a, 8 * (threadIdx.x + i * n), w[i]);
    NormPiece next[PIECES];
    int row = blockIdx.x;
    auto load = [&](int r) {
        const NormRow at = norm_row(a, r);
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
            if (threadIdx.x + i * n < pieces) load_piece(a, at, 8 * (threadIdx.x + i * n), next[i]);
    };
    if (row < a.rows) load(row);
    for (int turn = 0; row < a.rows; turn ^= 1) {
        NormPiece p[PIECES];
        float h[PIECES][8], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            p[i] = next[i];
            if (threadIdx.x + i * n < pieces) open_piece(a, p[i], h[i], sum);
        }
        const int after = row > a.rows - 1 - (int)gridDim.x ? a.rows : row + gridDim.x;
        if (after < a.rows) load(after);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (threadIdx.x % 32 == 0) part[turn][threadIdx.x / 32] = sum;
        __syncthreads();   // (two sets of parts: a warp may be a row ahead, never two)
        sum = threadIdx.x % 32 < warps ? part[turn][threadIdx.x % 32] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float inv = rsqrtf(fmaf(sum, a.whole, a.eps));
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
            if (threadIdx.x + i * n < pieces)
                close_piece(a, p[i], (long long)row * a.dim + 8 * (threadIdx.x + i * n), inv, w[i], h[i]);
        row = after;
    }
}

template <int TEAM, int PIECES, int ROWS>
cudaError_t launch_warp(const NormArgs& a, cudaStream_t stream) {
    const int per = 256 / TEAM * ROWS;
    return launch_pdl(norm_warp_kernel<TEAM, PIECES, ROWS>, dim3((a.rows + per - 1) / per), dim3(256), 0, stream, true,
                      a);
}
template <int PIECES>
cudaError_t launch_cta(const NormArgs& a, int sms, cudaStream_t stream) {
    const int threads = (a.dim / 8 + 32 * PIECES - 1) / (32 * PIECES) * 32;
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, norm_cta_kernel<PIECES>, threads, 0) != cudaSuccess)
        return cudaErrorUnknown;
    const int most = sms * (per_sm > 0 ? per_sm : 1);
    return launch_pdl(norm_cta_kernel<PIECES>, dim3(a.rows < most ? a.rows : most), dim3(threads), 0, stream, true, a);
}

}  // namespace
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
    int k = 0;
    while (1 << k < dim) ++k;
    const NormArgs a{x, residual, gate, weight, out, residual_out, x_token, x_head, residual_token, residual_head,
                     gate_token, gate_head, x_is_f32, residual_is_f32, gate_is_f32, out_is_f32, heads, dim, T * heads,
                     after, gate_act == TERN_GATE_SIGMOID, scale, eps, weight_offset,
                     ldexpf(1.0f, -k), (float)(1 << k) / (float)dim};
    auto* s = (cudaStream_t)stream;
    const cudaError_t e = dim <= 64     ? launch_warp<8, 1, 2>(a, s)
                          : dim <= 128  ? launch_warp<16, 1, 2>(a, s)
                          : dim <= 256  ? launch_warp<32, 1, 2>(a, s)
                          : dim <= 512  ? launch_warp<32, 2, 1>(a, s)
                          : dim <= 8192 ? launch_cta<1>(a, sms, s)
                          : dim <= 16384 ? launch_cta<2>(a, sms, s)
                                         : launch_cta<4>(a, sms, s);
    if (e != cudaSuccess) return TERN_ERR_CUDA;
    set_launch_count(1);
    return TERN_OK;
}
