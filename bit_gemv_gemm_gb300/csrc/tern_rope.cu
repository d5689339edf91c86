// tern_rope.cu -- rotary positions of a step's queries and keys, and the
// append of its keys and values to the paged cache, in one pass.
//
//   y[2i], y[2i+1]  (or y[i], y[i + r/2])  =  the pair turned by pos * inv_freq[i],
//   cos and sin multiplied by attn_factor; values past the first r pass through.
//
// One CTA a token.  The r/2 sines and cosines are computed once per token and
// shared by its heads through shared memory, while the token's values are
// already on their way to registers; every value is read and written once, in
// 16-byte pieces.  Bound by those bytes.  A unit of work is 8 pairs of one head
// (or 16 values that only pass through), as two pieces far enough apart that a
// warp's accesses stay contiguous, which needs r and the head to be multiples of
// 16; other sizes take a plainer kernel, 8 values at a time with each value's
// partner read again.
#include <math.h>

#include "tern_cache.cuh"

namespace tern {
namespace {

__device__ int g_rope_error;

// Small CTAs, many an SM: each is a chain of waits (position, values, stores).
// 8192 tokens of 24 heads of 256: 34.5 us (5.8 TB/s); 36.3 with 192 threads a
// CTA, 42.9 with 384, 45.7 with three units a thread in flight and six CTAs.
constexpr int kRopeThreads = 128, kRopeCtas = 12;

struct RopeArgs {
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    const int* positions;
    const long long* slots;
    const float* inv_freq;
    float factor;
    int rot, T, q_heads;
    __nv_bfloat16 *q_out, *k_cache, *v_cache;
    CacheView c;
};

template <bool F32>
__device__ __forceinline__ void load8(const void* base, long long at, float (&x)[8]) {
    if constexpr (F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
        const float4 a = p[0], b = p[1];
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

// The angle of one position and frequency, reduced to half turns in 64 bits:
// pos * inv_freq grows past 1e5 radians in a long context, where 32 bits would
// leave an error near 1e-2.
__device__ __forceinline__ float2 turn(int pos, float inv_freq, float factor) {
    const double half_turns = (double)inv_freq * 0.31830988618379067154 * (double)pos;
    const double r = half_turns - 2.0 * rint(0.5 * half_turns);
    float s, c;
    sincospif((float)r, &s, &c);
    return make_float2(c * factor, s * factor);
}

// Where a token's keys and values go; -1: nowhere.
__device__ __forceinline__ long long cache_at(const RopeArgs& a, long long slot) {
    if (slot < 0) return -1;
    if (slot >= (long long)a.c.pages * a.c.page_size) {
        if (threadIdx.x == 0) report_device_error(&g_rope_error, TERN_DEVERR_CACHE_SLOT);
        return -1;
    }
    const long long page = slot <= 0x7fffffff ? (long long)((unsigned)slot / (unsigned)a.c.page_size) : slot / a.c.page_size;
    return page * a.c.page_stride + (slot - page * a.c.page_size) * a.c.slot_stride;
}

template <bool F32, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_append_kernel(const RopeArgs a) {
    extern __shared__ float2 turns[];   // [rot / 2] cos, sin
    pdl_launch_dependents();
    pdl_wait();
    const int D = a.c.head_dim, half = a.rot / 2, per = D / 16;
    const int t = blockIdx.x, pos = a.positions[t];
    const long long at = cache_at(a, a.slots[t]);
    const int units = (at < 0 ? a.q_heads : a.q_heads + 2 * a.c.kv_heads) * per;
    bool ready = false;
    for (int i = threadIdx.x; i < units || !ready; i += kRopeThreads) {
        // loads first
        float x[2][8];
        __nv_bfloat16* to = nullptr;
        int off = 0, pair = -1;   // from a unit's first piece to its second; its first pair, -1: no turn
        if (i < units) {
            const int h = (unsigned)i / (unsigned)per, u = i - h * per;
            const bool is_q = h < a.q_heads, is_v = h >= a.q_heads + a.c.kv_heads;
            const int hk = is_v ? h - a.q_heads - a.c.kv_heads : h - a.q_heads;
            const bool turned = !is_v && u < a.rot / 16;
            // the two pieces lie half the turning (or passing) part apart, so that neighbours touch neighbours
            const int d = turned || is_v ? 8 * u : a.rot + 8 * (u - a.rot / 16);
            off = is_v ? D / 2 : turned ? half : (D - a.rot) / 2;
            pair = !turned ? -1 : INTERLEAVED ? 4 * u : 8 * u;
            const void* src = is_q ? a.q : is_v ? a.v : a.k;
            const long long row = is_q ? t * a.q_stride + (long long)h * D
                                       : (is_v ? t * a.v_stride : t * a.k_stride) + (long long)hk * D;
            load8<F32>(src, row + d, x[0]);
            load8<F32>(src, row + d + off, x[1]);
            to = (is_q ? a.q_out + ((long long)t * a.q_heads + h) * D
                       : (is_v ? a.v_cache : a.k_cache) + at + hk * a.c.head_stride) + d;
        }
        if (!ready) {
            for (int k = threadIdx.x; k < half; k += kRopeThreads) turns[k] = turn(pos, a.inv_freq[k], a.factor);
            __syncthreads();
            ready = true;
        }
        if (i >= units) break;
        if (pair >= 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // pair e: interleaved, neighbours of one piece; else the same place of both
                float& p = INTERLEAVED ? x[e >> 2][2 * (e & 3)] : x[0][e];
                float& q = INTERLEAVED ? x[e >> 2][2 * (e & 3) + 1] : x[1][e];
                const float2 cs = turns[INTERLEAVED ? pair + (e & 3) + (e >> 2) * (half / 2) : pair + e];
                const float y = p * cs.x - q * cs.y;
                q = q * cs.x + p * cs.y;
                p = y;
            }
        }
        store8(to, x[0]);
        store8(to + off, x[1]);
    }
}

// Any even rot and any head of a multiple of 8.
template <bool F32, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_append_any_kernel(const RopeArgs a) {
    extern __shared__ float2 turns[];   // [rot / 2] cos, sin
    pdl_launch_dependents();
    pdl_wait();
    const int t = blockIdx.x, D = a.c.head_dim, half = a.rot / 2;
    const int pos = a.positions[t];
    for (int i = threadIdx.x; i < half; i += kRopeThreads) turns[i] = turn(pos, a.inv_freq[i], a.factor);
    const long long at = cache_at(a, a.slots[t]);
    __syncthreads();
    const int heads = at < 0 ? a.q_heads : a.q_heads + 2 * a.c.kv_heads;
    const int per = D / 8;
    for (int i = threadIdx.x; i < heads * per; i += kRopeThreads) {
        const int h = i / per, d = (i - h * per) * 8;
        const bool is_q = h < a.q_heads, is_v = h >= a.q_heads + a.c.kv_heads;
        const int hk = is_v ? h - a.q_heads - a.c.kv_heads : h - a.q_heads;
        const void* src = is_q ? a.q : is_v ? a.v : a.k;
        const long long row = is_q ? t * a.q_stride + (long long)h * D
                                   : (is_v ? t * a.v_stride : t * a.k_stride) + (long long)hk * D;
        float x[8], y[8];
        load8<F32>(src, row + d, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[e];
        if (!is_v && d < a.rot) {
            if constexpr (INTERLEAVED) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (d + 2 * e >= a.rot) break;
                    const float2 cs = turns[d / 2 + e];
                    y[2 * e] = x[2 * e] * cs.x - x[2 * e + 1] * cs.y;
                    y[2 * e + 1] = x[2 * e + 1] * cs.x + x[2 * e] * cs.y;
                }
            } else {
                for (int e = 0; e < 8; ++e) {
                    const int dd = d + e;
                    if (dd >= a.rot) break;
                    const bool low = dd < half;
                    const float2 cs = turns[low ? dd : dd - half];
                    const long long o = row + (low ? dd + half : dd - half);
                    const float other = F32 ? static_cast<const float*>(src)[o]
                                            : __bfloat162float(static_cast<const __nv_bfloat16*>(src)[o]);
                    y[e] = low ? x[e] * cs.x - other * cs.y : x[e] * cs.x + other * cs.y;
                }
            }
        }
        __nv_bfloat16* dst = is_q ? a.q_out + ((long long)t * a.q_heads + h) * D + d
                                  : (is_v ? a.v_cache : a.k_cache) + at + hk * a.c.head_stride + d;
        store8(dst, y);
    }
}

}  // namespace

cudaError_t read_rope_device_error(int* code) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_rope_error, sizeof(int));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_rope_error, &zero, sizeof(int));
}

}  // namespace tern

using namespace tern;

extern "C" tern_status tern_rope_frequencies_host(int rot_dim, double base, int scaling, double factor,
                                                  int original_len, double turns_fast, double turns_slow,
                                                  float* inv_freq, float* attn_factor) {
    if (rot_dim < 2 || rot_dim % 2 != 0 || !(base > 1.0) || scaling < TERN_ROPE_PLAIN || scaling > TERN_ROPE_PARTS ||
        (scaling != TERN_ROPE_PLAIN && !(factor >= 1.0)))
        return TERN_ERR_SHAPE;
    if (scaling == TERN_ROPE_PARTS && (original_len < 1 || !(turns_fast > turns_slow) || !(turns_slow > 0.0)))
        return TERN_ERR_SHAPE;
    if (!inv_freq || !attn_factor) return TERN_ERR_NULL;
    const int half = rot_dim / 2;
    if (scaling == TERN_ROPE_BASE && rot_dim > 2) base *= pow(factor, (double)rot_dim / (rot_dim - 2));
    double lo = 0, hi = 0;
    if (scaling == TERN_ROPE_PARTS) {
        // the pair index whose wave makes `turns` turns in the original length
        auto at = [&](double turns) {
            return rot_dim * log(original_len / (turns * 6.283185307179586477)) / (2.0 * log(base));
        };
        lo = fmax(0.0, floor(at(turns_fast)));
        hi = fmin(rot_dim - 1.0, ceil(at(turns_slow)));   // (may lie past the last pair: the ramp then ends there, unfinished)
    }
    for (int i = 0; i < half; ++i) {
        double f = pow(base, -2.0 * i / rot_dim);
        if (scaling == TERN_ROPE_LINEAR) f /= factor;
        if (scaling == TERN_ROPE_PARTS) {
            const double ramp = fmin(1.0, fmax(0.0, (i - lo) / fmax(hi - lo, 1e-3)));
            f = f / factor * ramp + f * (1.0 - ramp);
        }
        inv_freq[i] = (float)f;
    }
    *attn_factor = scaling == TERN_ROPE_PARTS ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
    return TERN_OK;
}

extern "C" tern_status tern_rope_append(const void* q, const void* k, const void* v, int in_is_f32,
                                        long long q_stride, long long k_stride, long long v_stride,
                                        const int* positions, const long long* slots, const float* inv_freq,
                                        float attn_factor, int rot_dim, int interleaved, int T, int q_heads,
                                        void* q_out, void* k_cache, void* v_cache, const tern_cache_layout* layout,
                                        tern_stream_t stream) {
    set_launch_count(0);
    RopeArgs a;
    tern_status st = make_cache_view(layout, &a.c);
    if (st != TERN_OK) return st;
    if (T < 0 || q_heads < 0 || q_heads > 65535 || rot_dim < 0 || rot_dim % 2 != 0 || rot_dim > a.c.head_dim)
        return TERN_ERR_SHAPE;
    // 16-byte pieces of each token's heads
    if (q_stride < 0 || k_stride < 0 || v_stride < 0 || q_stride % 8 || k_stride % 8 || v_stride % 8)
        return TERN_ERR_SHAPE;
    if ((T > 0 && ((q_heads > 0 && (!q || !q_out)) || !k || !v || !positions || !slots || (rot_dim > 0 && !inv_freq))) ||
        !k_cache || !v_cache)
        return TERN_ERR_NULL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_cache) ||
        !aligned16(v_cache) || !aligned_to(positions, 4) || !aligned_to(slots, 8) || !aligned_to(inv_freq, 4))
        return TERN_ERR_ALIGN;
    st = check_device(nullptr);
    if (st != TERN_OK) return st;
    if (T == 0) return TERN_OK;
    a.q = q; a.k = k; a.v = v;
    a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.positions = positions;
    a.slots = slots;
    a.inv_freq = inv_freq;
    a.factor = attn_factor;
    a.rot = rot_dim;
    a.T = T;
    a.q_heads = q_heads;
    a.q_out = static_cast<__nv_bfloat16*>(q_out);
    a.k_cache = static_cast<__nv_bfloat16*>(k_cache);
    a.v_cache = static_cast<__nv_bfloat16*>(v_cache);
    auto kernel = in_is_f32 ? (interleaved ? rope_append_kernel<true, true> : rope_append_kernel<true, false>)
                            : (interleaved ? rope_append_kernel<false, true> : rope_append_kernel<false, false>);
    if (rot_dim % 16 != 0 || a.c.head_dim % 16 != 0)
        kernel = in_is_f32 ? (interleaved ? rope_append_any_kernel<true, true> : rope_append_any_kernel<true, false>)
                           : (interleaved ? rope_append_any_kernel<false, true> : rope_append_any_kernel<false, false>);
    if (launch_pdl(kernel, dim3(T), dim3(kRopeThreads), (size_t)(rot_dim / 2) * sizeof(float2),
                   (cudaStream_t)stream, true, a) != cudaSuccess)
        return TERN_ERR_CUDA;
    set_launch_count(1);
    return TERN_OK;
}
