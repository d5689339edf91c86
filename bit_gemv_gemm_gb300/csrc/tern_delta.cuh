// tern_delta.cuh -- the gated delta rule's arguments, shared by its kernels.  Internal.
#pragma once

#include "tern_state.cuh"

namespace tern {

struct DeltaArgs {
    StateSeqView s;
    const __nv_bfloat16 *q, *k, *v;
    long long q_token, k_token, v_token;    // strides in elements
    const float *g, *beta;
    long long g_token, beta_token;
    const float *a_log, *dt_bias;           // null: g and beta are as given
    float* state;                           // [pool][v_heads][dv][dk]
    __nv_bfloat16* out;                     // [T][v_heads][dv]
    int k_heads, v_heads, dk, dv, group, norm;
    float scale;
};

constexpr float kDeltaNormEps = 1e-6f;

// The gates of one token and value head as they lie in memory...
__device__ __forceinline__ float2 delta_raw_gates(const DeltaArgs& a, long long token, int h) {
    return make_float2(a.g[token * a.g_token + h], a.beta[token * a.beta_token + h]);
}
// ... and the log of the decay and the step that they stand for.  A log below -200 (a
// decay of 0 in 32 bits all the same) becomes -200, so that differences of sums of it
// stay numbers.
struct DeltaHead {
    bool raw;
    float rate, bias;
};
__device__ __forceinline__ DeltaHead delta_head(const DeltaArgs& a, int h) {
    return a.a_log ? DeltaHead{true, expf(a.a_log[h]), a.dt_bias[h]} : DeltaHead{false, 0.0f, 0.0f};
}
__device__ __forceinline__ float2 delta_gates(const DeltaHead& head, float2 raw) {
    float g = raw.x, b = raw.y;
    if (head.raw) {
        const float x = g + head.bias;
        g = -head.rate * (fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x))));
        b = 1.0f / (1.0f + expf(-b));
    }
    return make_float2(g < -200.0f ? -200.0f : g, b);
}

cudaError_t launch_delta_step(const DeltaArgs& a, cudaStream_t stream);
cudaError_t launch_delta_chunk(const DeltaArgs& a, cudaStream_t stream);

}  // namespace tern
