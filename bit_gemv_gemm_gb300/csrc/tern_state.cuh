// tern_state.cuh -- sequences of new tokens with a state slot each, as the
// kernels of a linear-attention layer see them: argument checks shared by the
// entry points, and the per-sequence view with its device-side bounds checks.
// Internal.
#pragma once

#include "tern_cache.cuh"
#include "tern_mma.cuh"

namespace tern {

// The tokens of B sequences in a row; each reads its state from slots[b] and
// leaves the new one in dst_slots[b].
struct StateSeqView {
    const int* q_start;     // [B + 1] first new token of each sequence; null: T / B each
    const int* slots;       // [B]; negative: starts from zeros
    const int* dst_slots;   // [B]; negative: not stored
    const int* past;        // [B]; 0: starts from zeros, whatever the slot holds; null: none is 0
    int B, T, max_new, pool;
};

// One sequence: its new tokens t0 .. t0 + n - 1, the slot it reads (-1: zeros) and
// the one it writes (-1: none).  Values that do not fit the call's arrays are
// reported; a bad range is cut to what fits, a bad slot is neither read nor written.
struct StateSeq {
    int t0, n, src, dst;
};
__device__ __forceinline__ StateSeq load_state_seq(const StateSeqView& s, int b, int* err) {
    StateSeq r;
    if (s.q_start) {
        const int a = s.q_start[b], e = s.q_start[b + 1];
        r.t0 = min(max(a, 0), s.T);
        r.n = min(max(e, r.t0), s.T) - r.t0;
        if (a != r.t0 || e != r.t0 + r.n || r.n > s.max_new) report_device_error(err, TERN_DEVERR_CACHE_SEQUENCE);
        r.n = min(r.n, s.max_new);
    } else {
        r.n = s.T / s.B;
        r.t0 = b * r.n;
    }
    r.src = s.slots[b];
    r.dst = s.dst_slots[b];
    if (r.src >= s.pool || r.dst >= s.pool) {
        report_device_error(err, TERN_DEVERR_STATE_SLOT);
        r.src = r.src >= s.pool ? -1 : r.src;
        r.dst = r.dst >= s.pool ? -1 : r.dst;
    }
    if (r.src < 0 || (s.past && s.past[b] == 0)) r.src = -1;
    return r;
}

inline tern_status make_state_seq_view(const int* q_start, const int* slots, const int* dst_slots, const int* past,
                                       int B, int T, int max_new, int pool, StateSeqView* s) {
    if (B < 1 || B > 65535 || T < 0 || max_new < 0 || pool < 1) return TERN_ERR_SHAPE;
    if (!q_start && T % B != 0) return TERN_ERR_SHAPE;
    if (!slots) return TERN_ERR_NULL;
    if (!aligned_to(q_start, 4) || !aligned_to(slots, 4) || !aligned_to(dst_slots, 4) || !aligned_to(past, 4))
        return TERN_ERR_ALIGN;
    *s = StateSeqView{q_start, slots, dst_slots ? dst_slots : slots, past, B, T,
                      q_start ? (max_new < T ? max_new : T) : T / B, pool};
    return TERN_OK;
}

// ---- 8 values as they lie in memory (fp32: both registers; bf16: the first) ----
struct Raw8 {
    uint4 a, b;
};
__device__ __forceinline__ Raw8 load_raw8(const void* base, long long at, int is_f32) {
    Raw8 r;
    if (is_f32) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + at);
        r.a = p[0];
        r.b = p[1];
    } else {
        r.a = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
        r.b = make_uint4(0, 0, 0, 0);
    }
    return r;
}
__device__ __forceinline__ void widen8(const Raw8& r, int is_f32, float (&x)[8]) {
    const uint32_t u[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
    if (is_f32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    }
}
__device__ __forceinline__ void store_raw8(void* base, long long at, int is_f32, const float (&x)[8]) {
    if (is_f32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
        p[0] = make_float4(x[0], x[1], x[2], x[3]);
        p[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + at) =
            make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    }
}
// 1 / (1 + e^-x) by the approximate exponential and reciprocal: some units in the last
// place, far below a bf16's step.  (The exact quotient took a third of a convolution's time.)
__device__ __forceinline__ float sigmoid(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.0f + exp2_fast(-1.44269504088896341f * x)));
    return y;
}

constexpr uint32_t kWaitTries = 1u << 19, kWaitNap = 2000;   // of a wait, and ns of each: a second, far beyond any real one
// A thread's wait for an mbarrier, which gives up after a number of tries.  (Short: some forty
// of them stand in loops of gated_delta whose code has to stay in the instruction cache, and
// asking the time takes longer than most of them.  Every lane asks; one for all made the others
// wait longer.)
__device__ __forceinline__ bool wait_tries(uint32_t bar, uint32_t parity, uint32_t tries) {
    uint32_t ok = 0;
#pragma unroll 1
    for (uint32_t n = tries; !ok && n > 0; --n)
        asm volatile(
            "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\nselp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(kWaitNap)
            : "memory");
    return ok != 0;
}

}  // namespace tern
