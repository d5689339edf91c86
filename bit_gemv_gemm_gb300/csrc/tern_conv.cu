// tern_conv.cu -- the short causal convolution along the tokens, channel by
// channel, with its state.
//
//   y[t] = act(bias + sum_{w < W} weight[w] x[t - (W - 1) + w]),
//   the inputs before a sequence's first token from its state, which is its last
//   W - 1 inputs.
//
// A thread owns 4 channels and walks a stretch of one sequence's tokens with the
// last W - 1 inputs in registers, so each input is read once (but for W - 1 at
// the start of a stretch).  Bound by the bytes read and written.
#include "tern_state.cuh"

namespace tern {
namespace {

__device__ int g_conv_error;

constexpr int kConvThreads = 128, kConvBatch = 8, kConvStretch = 32;

struct ConvArgs {
    StateSeqView s;
    const void* x;
    long long x_token;
    const float *weight, *bias;
    float* state;
    __nv_bfloat16* out;
    int channels, in_f32, silu;
};

__device__ __forceinline__ uint4 load4(const ConvArgs& a, long long at) {
    if (a.in_f32) return *reinterpret_cast<const uint4*>(static_cast<const float*>(a.x) + at);
    const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.x) + at);
    return make_uint4(v.x, v.y, 0, 0);
}
__device__ __forceinline__ float4 widen4(const ConvArgs& a, uint4 r) {
    if (a.in_f32)
        return make_float4(__uint_as_float(r.x), __uint_as_float(r.y), __uint_as_float(r.z), __uint_as_float(r.w));
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u), __uint_as_float(r.y << 16),
                       __uint_as_float(r.y & 0xFFFF0000u));
}

template <int W>
__global__ void __launch_bounds__(kConvThreads) short_conv_kernel(const ConvArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int c = 4 * (blockIdx.x * kConvThreads + threadIdx.x);
    const StateSeq q = load_state_seq(a.s, blockIdx.y, &g_conv_error);
    const long long stretch = (long long)blockIdx.z * kConvStretch;
    // (the first stretch's CTA is there for a sequence without tokens too: its state moves)
    if (c >= a.channels || (stretch >= q.n && blockIdx.z > 0)) return;
    const int first = (int)stretch, last = min(first + kConvStretch, q.n);
    const long long base = (long long)q.t0 * a.x_token + c;

    uint4 in[kConvBatch];
    auto load = [&](int t) {
#pragma unroll
        for (int i = 0; i < kConvBatch; ++i)
            if (t + i < last) in[i] = load4(a, base + (t + i) * a.x_token);
    };
    load(first);
    // the inputs before the stretch: back[0] the oldest
    float4 back[W - 1];
    float4* const old = reinterpret_cast<float4*>(a.state + (long long)q.src * (W - 1) * a.channels + c);
#pragma unroll
    for (int w = 0; w < W - 1; ++w) {
        const int t = first - (W - 1) + w;
        back[w] = t >= 0 ? widen4(a, load4(a, base + t * a.x_token))
                  : q.src >= 0 ? old[(long long)w * (a.channels / 4)]
                               : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    float4 weight[W], bias = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (a.bias) bias = make_float4(a.bias[c], a.bias[c + 1], a.bias[c + 2], a.bias[c + 3]);
    {
        // [C][W]: the 4 channels' weights lie in a row
        const float* p = a.weight + (long long)c * W;
#pragma unroll
        for (int w = 0; w < W; ++w) weight[w] = make_float4(p[w], p[W + w], p[2 * W + w], p[3 * W + w]);
    }
    // the new state, by the thread that has read the old one: its first tokens may be what is left of that
    if (blockIdx.z == 0 && q.dst >= 0 && (q.n > 0 || q.dst != q.src)) {
        float4* const to = reinterpret_cast<float4*>(a.state + (long long)q.dst * (W - 1) * a.channels + c);
        float4 keep[W - 1];
#pragma unroll
        for (int w = 0; w < W - 1; ++w) {
            const int t = q.n - (W - 1) + w;
            keep[w] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (t >= 0) {
                keep[w] = widen4(a, load4(a, base + t * a.x_token));
            } else {
#pragma unroll
                for (int o = 0; o < W - 1; ++o)
                    if (o == q.n + w) keep[w] = back[o];
            }
        }
#pragma unroll
        for (int w = 0; w < W - 1; ++w) to[(long long)w * (a.channels / 4)] = keep[w];
    }
    for (int t = first; t < last; t += kConvBatch) {
        float4 x[kConvBatch];
#pragma unroll
        for (int i = 0; i < kConvBatch; ++i) x[i] = widen4(a, in[i]);
        load(t + kConvBatch);
#pragma unroll
        for (int i = 0; i < kConvBatch; ++i) {
            if (t + i >= last) break;
            float4 y = bias;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const int j = i - (W - 1) + w;
                const float4 v = j >= 0 ? x[j < 0 ? 0 : j] : back[j < 0 ? j + W - 1 : 0];
                y.x = fmaf(weight[w].x, v.x, y.x);
                y.y = fmaf(weight[w].y, v.y, y.y);
                y.z = fmaf(weight[w].z, v.z, y.z);
                y.w = fmaf(weight[w].w, v.w, y.w);
            }
            if (a.silu) {
                y.x *= sigmoid(y.x);
                y.y *= sigmoid(y.y);
                y.z *= sigmoid(y.z);
                y.w *= sigmoid(y.w);
            }
            *reinterpret_cast<uint2*>(a.out + (long long)(q.t0 + t + i) * a.channels + c) =
                make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
        }
#pragma unroll
        for (int w = 0; w < W - 1; ++w) back[w] = x[kConvBatch - (W - 1) + w];
    }
}

}  // namespace

cudaError_t read_conv_device_error(int* code) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_conv_error, sizeof(int));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_conv_error, &zero, sizeof(int));
}

}  // namespace tern

using namespace tern;

extern "C" tern_status tern_short_conv(const void* x, int x_is_f32, long long x_token, const float* weight, int width,
                                       const float* bias, int silu, float* state, int pool, const int* slots,
                                       const int* dst_slots, const int* past, const int* q_start, int B, int T,
                                       int max_new, int channels, void* out, tern_stream_t stream) {
    set_launch_count(0);
    ConvArgs a;
    tern_status st = make_state_seq_view(q_start, slots, dst_slots, past, B, T, max_new, pool, &a.s);
    if (st != TERN_OK) return st;
    if (width < 2 || width > 4 || channels < 8 || channels % 8 != 0 || channels > (1 << 20) ||
        a.s.max_new > (1 << 20) || (x_token < channels && T > 1) || x_token < 0 || x_token % 8 != 0 || x_token >= (1LL << 37))
        return TERN_ERR_SHAPE;
    if (!weight || !state || (T > 0 && (!x || !out))) return TERN_ERR_NULL;
    if (!aligned16(x) || !aligned16(weight) || !aligned_to(bias, 4) || !aligned16(state) || !aligned16(out))
        return TERN_ERR_ALIGN;
    st = check_device(nullptr);
    if (st != TERN_OK) return st;
    a.x = x;
    a.x_token = x_token;
    a.weight = weight;
    a.bias = bias;
    a.state = state;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.channels = channels;
    a.in_f32 = x_is_f32;
    a.silu = silu;
    auto kernel = width == 2 ? short_conv_kernel<2> : width == 3 ? short_conv_kernel<3> : short_conv_kernel<4>;
    const int most = a.s.max_new > 1 ? a.s.max_new : 1;
    const dim3 grid((channels / 4 + kConvThreads - 1) / kConvThreads, B, (most + kConvStretch - 1) / kConvStretch);
    if (launch_pdl(kernel, grid, dim3(kConvThreads), 0, (cudaStream_t)stream, true, a) != cudaSuccess)
        return TERN_ERR_CUDA;
    set_launch_count(1);
    return TERN_OK;
}
