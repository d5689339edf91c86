// tern_conv.cu -- the short causal convolution along the tokens, channel by
// channel, with its state.
//
//   y[t] = act(bias + sum_{w < W} weight[w] x[t - (W - 1) + w]),
//   the inputs before a sequence's first token from its state, which is its last
//   W - 1 inputs.
//
// A thread owns 4 channels and walks a stretch of one sequence's tokens with the
// last W - 1 inputs in registers, so each input is read once (but for W - 1 at
// the start of a stretch), a batch of tokens ahead.  Bound by the bytes read and written:
// four prompts, 11467 tokens of 8192 channels in bf16, 65 us, 85 % of the copy bandwidth;
// sixteen single tokens 3.5 us, a launch and three dependent loads.
#include "tern_state.cuh"

namespace tern {
namespace {

__device__ int g_conv_error;

constexpr int kConvThreads = 128, kConvStretch = 128;
constexpr int kPairs = 2;   // of channels a thread (4: 89 us for four prompts)
constexpr int kBatch = 16;   // tokens in flight
// In calls of few tokens a batch is all of them, in less code: 16 sequences of one token 3.5 us,
// 5.1 with 16 in flight; four prompts of up to 4096 65.4 us, 73 with 8 (and 72 with 20, of more
// registers).
constexpr int kFewTokens = 8;

struct ConvArgs {
    StateSeqView s;
    const void* x;
    long long x_token;
    const float *weight, *bias;
    float* state;
    __nv_bfloat16* out;
    int channels, silu;
};

// A thread's channels of one token as they lie in memory, and as pairs.
template <bool F32>
struct Raw {
    uint32_t u[kPairs * (F32 ? 2 : 1)];
};
template <bool F32>
__device__ __forceinline__ void load_raw(const void* base, long long at, Raw<F32>& r) {
    constexpr int kWords = kPairs * (F32 ? 2 : 1);
    const void* p = F32 ? static_cast<const void*>(static_cast<const float*>(base) + at)
                        : static_cast<const void*>(static_cast<const __nv_bfloat16*>(base) + at);
    if constexpr (kWords == 2) {
        const uint2 v = *static_cast<const uint2*>(p);
        r.u[0] = v.x;
        r.u[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
            const uint4 v = static_cast<const uint4*>(p)[i];
            r.u[4 * i] = v.x;
            r.u[4 * i + 1] = v.y;
            r.u[4 * i + 2] = v.z;
            r.u[4 * i + 3] = v.w;
        }
    }
}
template <bool F32>
__device__ __forceinline__ void widen(const Raw<F32>& r, uint64_t (&x)[kPairs]) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
        x[i] = F32 ? pack2(__uint_as_float(r.u[2 * i]), __uint_as_float(r.u[2 * i + (F32 ? 1 : 0)]))
                   : pack2(__uint_as_float(r.u[i] << 16), __uint_as_float(r.u[i] & 0xFFFF0000u));
}

// BATCH: tokens in flight
template <int W, bool F32, int BATCH>
__global__ void __launch_bounds__(kConvThreads) short_conv_kernel(const ConvArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int c = 2 * kPairs * (blockIdx.x * kConvThreads + threadIdx.x);
    const StateSeq q = load_state_seq(a.s, blockIdx.y, &g_conv_error);
    const long long stretch = (long long)blockIdx.z * kConvStretch;
    // (the first stretch's CTA is there for a sequence without tokens too: its state moves)
    if (c >= a.channels || (stretch >= q.n && blockIdx.z > 0)) return;
    const int first = (int)stretch, last = min(first + kConvStretch, q.n);
    const long long base = (long long)q.t0 * a.x_token + c;

    Raw<F32> in[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
        if (first + i < last) load_raw<F32>(a.x, base + (first + i) * a.x_token, in[i]);
    auto input = [&](int t, uint64_t (&x)[kPairs]) {
        Raw<F32> r;
        load_raw<F32>(a.x, base + t * a.x_token, r);
        widen<F32>(r, x);
    };
    auto state_of = [&](int slot, int w) {
        return reinterpret_cast<uint64_t*>(a.state + ((long long)slot * (W - 1) + w) * a.channels + c);
    };
    // the inputs before the stretch: back[0] the oldest
    uint64_t back[W - 1][kPairs];
#pragma unroll
    for (int w = 0; w < W - 1; ++w) {
        const int t = first - (W - 1) + w;
        if (t >= 0) {
            input(t, back[w]);
        } else {
#pragma unroll
            for (int i = 0; i < kPairs; i += 2) {
                const ulonglong2 v = q.src >= 0 ? *reinterpret_cast<const ulonglong2*>(state_of(q.src, w) + i) : make_ulonglong2(0, 0);
                back[w][i] = v.x;
                back[w][i + 1] = v.y;
            }
        }
    }
    uint64_t weight[W][kPairs], bias[kPairs];
    {
        float p[2 * kPairs * W], b[2 * kPairs] = {};   // [channel][W]
#pragma unroll
        for (int i = 0; i < kPairs * W / 2; ++i) {
            const float4 v = reinterpret_cast<const float4*>(a.weight + (long long)c * W)[i];
            p[4 * i] = v.x, p[4 * i + 1] = v.y, p[4 * i + 2] = v.z, p[4 * i + 3] = v.w;
        }
        if (a.bias) {
#pragma unroll
            for (int i = 0; i < 2 * kPairs; ++i) b[i] = a.bias[c + i];
        }
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            bias[i] = pack2(b[2 * i], b[2 * i + 1]);
#pragma unroll
            for (int w = 0; w < W; ++w) weight[w][i] = pack2(p[2 * i * W + w], p[(2 * i + 1) * W + w]);
        }
    }
    // the new state, by the thread that has read the old one: its first tokens may be what is left of that
    if (blockIdx.z == 0 && q.dst >= 0 && (q.n > 0 || q.dst != q.src)) {
        uint64_t keep[W - 1][kPairs];
#pragma unroll
        for (int w = 0; w < W - 1; ++w) {
            const int t = q.n - (W - 1) + w;
            if (t >= 0) {
                input(t, keep[w]);
            } else {
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                    keep[w][i] = 0;
#pragma unroll
                    for (int o = 0; o < W - 1; ++o) keep[w][i] = o == q.n + w ? back[o][i] : keep[w][i];
                }
            }
        }
#pragma unroll
        for (int w = 0; w < W - 1; ++w)
#pragma unroll
            for (int i = 0; i < kPairs; i += 2)
                *reinterpret_cast<ulonglong2*>(state_of(q.dst, w) + i) = make_ulonglong2(keep[w][i], keep[w][i + 1]);
    }
    __nv_bfloat16* out = a.out + (long long)(q.t0 + first) * a.channels + c;
    for (int t = first; t < last; t += BATCH) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            if (t + i >= last) return;
            uint64_t x[kPairs];
            uint32_t y[kPairs];
            widen<F32>(in[i], x);
            if (t + i + BATCH < last) load_raw<F32>(a.x, base + (t + i + BATCH) * a.x_token, in[i]);
#pragma unroll
            for (int p = 0; p < kPairs; ++p) {
                uint64_t s = bias[p];
#pragma unroll
                for (int w = 0; w < W - 1; ++w) s = fma2(weight[w][p], back[w][p], s);
                float u, v;
                unpack2(fma2(weight[W - 1][p], x[p], s), u, v);
#pragma unroll
                for (int w = 0; w < W - 2; ++w) back[w][p] = back[w + 1][p];
                back[W - 2][p] = x[p];
                if (a.silu) {
                    u *= sigmoid(u);
                    v *= sigmoid(v);
                }
                y[p] = pack_bf16(u, v);
            }
            *reinterpret_cast<uint2*>(out) = make_uint2(y[0], y[1]);
            out += a.channels;
        }
    }
}

template <int W, bool F32>
auto pick(bool few) {
    return few ? short_conv_kernel<W, F32, kFewTokens> : short_conv_kernel<W, F32, kBatch>;
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
    a.silu = silu;
    const bool few = a.s.max_new <= kFewTokens;
    auto kernel = width == 2   ? (x_is_f32 ? pick<2, true>(few) : pick<2, false>(few))
                  : width == 3 ? (x_is_f32 ? pick<3, true>(few) : pick<3, false>(few))
                               : (x_is_f32 ? pick<4, true>(few) : pick<4, false>(few));
    const int most = a.s.max_new > 1 ? a.s.max_new : 1;
    const dim3 grid((channels / (2 * kPairs) + kConvThreads - 1) / kConvThreads, B, (most + kConvStretch - 1) / kConvStretch);
    if (launch_pdl(kernel, grid, dim3(kConvThreads), 0, (cudaStream_t)stream, true, a) != cudaSuccess)
        return TERN_ERR_CUDA;
    set_launch_count(1);
    return TERN_OK;
}
