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

// The gates of one token and value head: the log of the decay, and the step.  A
// log below -200 (a decay of 0 in 32 bits all the same) becomes -200, so that
// differences of sums of it stay numbers.
__device__ __forceinline__ float2 delta_gates(const DeltaArgs& a, long long token, int h) {
    float g = a.g[token * a.g_token + h], b = a.beta[token * a.beta_token + h];
    if (a.a_log) {
        const float x = g + a.dt_bias[h];
        g = -expf(a.a_log[h]) * (fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x))));
        b = 1.0f / (1.0f + expf(-b));
    }
    return make_float2(g < -200.0f ? -200.0f : g, b);
}

cudaError_t launch_delta_step(const DeltaArgs& a, cudaStream_t stream);
cudaError_t launch_delta_chunk(const DeltaArgs& a, cudaStream_t stream);

}  // namespace tern
