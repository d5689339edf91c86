// tern_delta.cuh -- the gated delta rule's arguments, shared by its kernels.  Internal.
#pragma once

#include "tern_state.cuh"

namespace tern {

// A sequence's chunks in `count` pieces of equal length, each run at once with the others
// from S = 0 (the first from the sequence's own): what it makes of S = 0 and, rows of the
// unit matrix in place of S's and no v, what it does to any S.  By linearity
//   S after it = S M + B,  out = S out_move + out,
// which the join kernels make of the arrays here.
struct DeltaPieces {
    int count;
    float* state;            // [B][v_heads][count][dv][dk] fp32: B of each piece (the first: S after it)
    unsigned char* move;     // [B][v_heads][count - 1]: parts of M of each but the first, dk rows
    unsigned char* parts;    // [B][v_heads][128 rows][count - 1]: parts of S after each but the last, 128 rows
    float* out;              // [chunks behind first pieces][v_heads][128 rows][64 tokens][rows] fp32
    unsigned char* out_move; // [chunks][v_heads]: parts of it, 64 rows
};
// Two parts of a matrix of dk columns, each in tiles of 64 columns with 128-byte swizzled rows.
__host__ __device__ constexpr uint32_t delta_parts_bytes(int rows, int dk) { return 4u * (uint32_t)rows * (uint32_t)dk; }
constexpr int kDeltaChunk = 64, kDeltaRows = 128, kDeltaPieceChunks = 8;   // (the fewest chunks that go in pieces)

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
    int by_length;                          // more CTAs than SMs: the longest of each 32 neighbours first
    float scale;
    DeltaPieces p;
};

constexpr float kDeltaNormEps = 1e-6f;

// The chunks of a piece of a sequence of n tokens; short ones are one piece.
__device__ __forceinline__ int delta_piece_chunks(const DeltaPieces& p, int n) {
    const int chunks = (n + kDeltaChunk - 1) / kDeltaChunk;
    return chunks < kDeltaPieceChunks ? chunks : (chunks + p.count - 1) / p.count;
}
// Where in out and out_move sequence b's chunks behind its first piece begin.  Of its n tokens
// they are fewer than n (count - 1) / (64 count) + 1: sequences in a row stay apart, the last
// ends at (T - T / count) / 64 + 2 B at most.
__host__ __device__ inline long long delta_piece_chunk(int count, int t0, int b) {
    return (t0 - t0 / count) / kDeltaChunk + 2LL * b;
}
// a - a bf16 pair
__device__ __forceinline__ uint64_t less_bf16(uint64_t a, uint32_t b) {
    return fma2(pack2(__uint_as_float(b << 16), __uint_as_float(b & 0xFFFF0000u)), pack2(-1.0f, -1.0f), a);
}
// Two neighbours as a bf16 pair and what it leaves of them as another.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = pack_bf16(a, b);
    float x, y;
    unpack2(less_bf16(pack2(a, b), hi), x, y);
    lo = pack_bf16(x, y);
}

// Where the parts of S after a piece lie, of rows 128 `tile` on of `tiles` such.
__device__ __forceinline__ unsigned char* delta_parts(const DeltaPieces& p, int b, int v_heads, int h, int dk, int tiles, int tile, int piece) {
    return p.parts + ((((long long)b * v_heads + h) * tiles + tile) * (p.count - 1) + piece) * (long long)delta_parts_bytes(kDeltaRows, dk);
}
// Stores 8 neighbours of a row from column `col` on as parts.
__device__ __forceinline__ void put_parts8(unsigned char* parts, int rows, int dk, int row, int col, const float* v) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) split2(v[2 * e], v[2 * e + 1], hi[e], lo[e]);
    unsigned char* at = parts + col / 64 * (rows * 128) + row * 128 + ((col % 64 / 8 ^ (row & 7)) << 4);
    *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(at + rows * dk * 2) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}

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

// What a token is to the rows of S: its key and query, divided by their lengths and times the
// scale where they are to be, and its decay, step and k.q.  A warp each.
template <int DK>
__device__ __forceinline__ void delta_stage(const DeltaArgs& a, long long t, int h, int lane, float* k_to, float* q_to, float4* gate_to) {
    constexpr int MY = DK / 32;
    const __nv_bfloat16* kp = a.k + t * a.k_token + h / a.group * DK + MY * lane;
    const __nv_bfloat16* qp = a.q + t * a.q_token + h / a.group * DK + MY * lane;
    float k[MY], q[MY], kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
    for (int e = 0; e < MY; e += 2) {
        const float2 k2 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(kp + e));
        const float2 q2 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(qp + e));
        k[e] = k2.x;
        k[e + 1] = k2.y;
        q[e] = q2.x;
        q[e + 1] = q2.y;
    }
#pragma unroll
    for (int e = 0; e < MY; ++e) {
        kk = fmaf(k[e], k[e], kk);
        qq = fmaf(q[e], q[e], qq);
        kq = fmaf(k[e], q[e], kq);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        kk += __shfl_xor_sync(0xffffffffu, kk, o);
        qq += __shfl_xor_sync(0xffffffffu, qq, o);
        kq += __shfl_xor_sync(0xffffffffu, kq, o);
    }
    const float ik = a.norm ? 1.0f / sqrtf(kk + kDeltaNormEps) : 1.0f;
    const float iq = (a.norm ? 1.0f / sqrtf(qq + kDeltaNormEps) : 1.0f) * a.scale;
#pragma unroll
    for (int e = 0; e < MY; ++e) {
        k_to[MY * lane + e] = k[e] * ik;
        q_to[MY * lane + e] = q[e] * iq;
    }
    if (lane == 0) {
        const float2 gb = delta_gates(delta_head(a, h), delta_raw_gates(a, t, h));
        *gate_to = make_float4(expf(gb.x), gb.y, kq * ik * iq, 0.0f);
    }
}

// A warp's wait.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, uint32_t tries = kWaitTries) {
    return __all_sync(0xffffffffu, wait_tries(bar, parity, tries));
}
// One lane of a warp whose lanes all come here: what it alone then does is known to be
// done by one, and its operands stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(e));
    return e != 0;
}

cudaError_t launch_delta_step(const DeltaArgs& a, cudaStream_t stream);
cudaError_t launch_delta_chunk(const DeltaArgs& a, cudaStream_t stream);
cudaError_t launch_delta_join(const DeltaArgs& a, int sms, cudaStream_t stream);

}  // namespace tern
