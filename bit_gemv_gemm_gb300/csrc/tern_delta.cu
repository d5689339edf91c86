// tern_delta.cu -- the gated delta rule, token by token.
//
//   a = exp(g),  u = beta (v - a S k),  S <- a S + u k^T,  o = scale S q
//
// per value head, S [dv][dk] in 32 bits.  A CTA owns some rows of one head's S,
// which depend on one another's only through q and k: they stay in registers
// from the first token to the last, so a call of a few tokens reads and writes
// every state once and is bound by that: one token of 64 sequences of 48 heads of 128 x 128
// 61.4 us, 97 % of the copy bandwidth.  Each token more costs a CTA some 0.8 us of products
// and of sums over the 8 lanes that share a row: five of 8 sequences of 32 heads 9.9 us, of
// which 6.2 are the states'.  (Products by pairs, fewer sums and 16 rows a warp in place of
// 8 each change that by 5 % at most, and lose as much where few CTAs run.)
#include "tern_delta.cuh"

#include <algorithm>

namespace tern {
namespace {

__device__ int g_delta_error;

constexpr int kStepThreads = 128, kStepBatch = 8;
// The most tokens of a sequence that go one by one.  24 (32) tokens so and by chunks, 32 heads of
// 128 x 128: one sequence 13.1 against 16.7 us (16.8, 16.9), eight 32.7 against 35.7 (42.6,
// 36.1), sixty-four 223 against 246 (293, 249).
constexpr int kStepTokens = 24;

// 8 lanes share a row: lane l has the values 32 i + 4 l + {0..3}, so that a row's
// loads are 128 bytes in a piece.  A warp holds 4 x ROWS rows.
template <int DK>
__global__ void __launch_bounds__(kStepThreads) delta_step_kernel(const DeltaArgs a) {
    constexpr int V4 = DK / 32, ROWS = 256 / DK, PER_WARP = 4 * ROWS, PER_CTA = 4 * PER_WARP;
    __shared__ __align__(16) float ks[kStepBatch][DK], qs[kStepBatch][DK];
    __shared__ float4 gates[kStepBatch];          // decay, beta, k.q, unused
    __shared__ float vs[kStepBatch][PER_CTA];
    __shared__ __nv_bfloat16 os[kStepBatch][PER_CTA];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, sub = lane % 8;
    const int h = blockIdx.y, row0 = blockIdx.x * PER_CTA;
    const StateSeq s = load_state_seq(a.s, blockIdx.z, &g_delta_error);
    const int live = min(PER_CTA, a.dv - row0);

    float4 S[ROWS][V4];
    const int mine = warp * PER_WARP + lane / 8;   // and every fourth row after it
    const long long head = (long long)a.dv * DK;
    {
        const float* from = a.state + ((long long)s.src * a.v_heads + h) * head + (long long)row0 * DK;
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int i = 0; i < V4; ++i)
                S[r][i] = s.src >= 0 && mine + 4 * r < live
                              ? *reinterpret_cast<const float4*>(from + (mine + 4 * r) * DK + 32 * i + 4 * sub)
                              : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    for (int t0 = 0; t0 < s.n; t0 += kStepBatch) {
        const int n = min(kStepBatch, s.n - t0);
        // a warp a token: its query and key (divided by their lengths), its gates and values
        for (int i = warp; i < n; i += 4) {
            const long long t = s.t0 + t0 + i;
            for (int r = lane; r < live; r += 32)
                vs[i][r] = __bfloat162float(a.v[t * a.v_token + (long long)h * a.dv + row0 + r]);
            delta_stage<DK>(a, t, h, lane, ks[i], qs[i], &gates[i]);
        }
        __syncthreads();
        for (int i = 0; i < n; ++i) {
            float4 k[V4], q[V4];
#pragma unroll
            for (int c = 0; c < V4; ++c) {
                k[c] = *reinterpret_cast<const float4*>(&ks[i][32 * c + 4 * sub]);
                q[c] = *reinterpret_cast<const float4*>(&qs[i][32 * c + 4 * sub]);
            }
            const float4 gate = gates[i];
            float sk[ROWS], sq[ROWS];
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                sk[r] = sq[r] = 0.0f;
#pragma unroll
                for (int c = 0; c < V4; ++c) {
                    sk[r] = fmaf(S[r][c].x, k[c].x, fmaf(S[r][c].y, k[c].y, fmaf(S[r][c].z, k[c].z, fmaf(S[r][c].w, k[c].w, sk[r]))));
                    sq[r] = fmaf(S[r][c].x, q[c].x, fmaf(S[r][c].y, q[c].y, fmaf(S[r][c].z, q[c].z, fmaf(S[r][c].w, q[c].w, sq[r]))));
                }
            }
#pragma unroll
            for (int o = 4; o > 0; o >>= 1)
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    sk[r] += __shfl_xor_sync(0xffffffffu, sk[r], o);
                    sq[r] += __shfl_xor_sync(0xffffffffu, sq[r], o);
                }
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const float u = gate.y * (vs[i][mine + 4 * r] - gate.x * sk[r]);
#pragma unroll
                for (int c = 0; c < V4; ++c) {
                    S[r][c].x = fmaf(u, k[c].x, gate.x * S[r][c].x);
                    S[r][c].y = fmaf(u, k[c].y, gate.x * S[r][c].y);
                    S[r][c].z = fmaf(u, k[c].z, gate.x * S[r][c].z);
                    S[r][c].w = fmaf(u, k[c].w, gate.x * S[r][c].w);
                }
                if (sub == 0) os[i][mine + 4 * r] = __float2bfloat16(fmaf(u, gate.z, gate.x * sq[r]));
            }
        }
        __syncthreads();
        for (int j = threadIdx.x; j < n * PER_CTA; j += kStepThreads) {
            const int i = j / PER_CTA, r = j % PER_CTA;
            if (r < live) a.out[((long long)(s.t0 + t0 + i) * a.v_heads + h) * a.dv + row0 + r] = os[i][r];
        }
        // (the next batch's staging touches neither os nor anything read above)
    }
    if (s.dst < 0 || (s.n == 0 && s.dst == s.src)) return;
    float* to = a.state + ((long long)s.dst * a.v_heads + h) * head + (long long)row0 * DK;
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int i = 0; i < V4; ++i)
            if (mine + 4 * r < live) *reinterpret_cast<float4*>(to + (mine + 4 * r) * DK + 32 * i + 4 * sub) = S[r][i];
}

}  // namespace

cudaError_t launch_delta_step(const DeltaArgs& a, cudaStream_t stream) {
    const int per = a.dk == 128 ? 32 : 64;
    return launch_pdl(a.dk == 128 ? delta_step_kernel<128> : delta_step_kernel<64>,
                      dim3((a.dv + per - 1) / per, a.v_heads, a.s.B), dim3(kStepThreads), 0, stream, true, a);
}

cudaError_t read_delta_device_error(int* code) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_delta_error, sizeof(int));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_delta_error, &zero, sizeof(int));
}

}  // namespace tern

using namespace tern;

namespace {
// How many pieces the sequences go in: no more than let every CTA of them have an SM of its own
// (a piece behind the first takes two, one for what it does to any state), and no more than
// the root of the longest one's chunks, past which the steps from piece to piece take longer
// than they save (8192 tokens of 2 heads: 11 pieces 113 us, 16 119; 4096: 8 pieces 82 us, 16 101).
// From kDeltaPieceChunks on; one sequence in pieces and whole, 128 x 128: 512 tokens of 16 heads 36.7
// against 42.8 us, 2048 77 and 138, of 32 heads 39.3 and 42.7, 99 and 138, of 48 heads 40.3
// and 43.0, 107 and 139; with 7 chunks the join takes what the pieces save.  The outputs of all
// pieces but the first go through the workspace: calls that would need more than a gigabyte
// of it go whole.
constexpr size_t kMostWorkspace = (size_t)1 << 30;
int delta_pieces(int B, int max_new, int v_heads, int dv, int sms) {
    const int chunks = (max_new + kDeltaChunk - 1) / kDeltaChunk;
    if (chunks < kDeltaPieceChunks) return 1;
    const long long moves = (long long)B * v_heads, ctas = moves * ((dv + kDeltaRows - 1) / kDeltaRows);
    const long long most = (sms + moves) / (ctas + moves);
    int count = 1;
    while (count < most && (long long)(count + 1) * (count + 1) <= chunks) ++count;
    return count;
}
struct PieceSizes {
    size_t state, move, parts, out, out_move;   // bytes
    size_t all() const { return state + move + parts + out + out_move; }
};
PieceSizes piece_sizes(int count, int B, int T, int v_heads, int dk, int dv) {
    const size_t heads = (size_t)B * v_heads, chunks = (size_t)delta_piece_chunk(count, T, B) * v_heads;
    return {heads * count * dv * dk * 4, heads * (count - 1) * delta_parts_bytes(dk, dk),
            heads * ((dv + kDeltaRows - 1) / kDeltaRows) * (count - 1) * delta_parts_bytes(kDeltaRows, dk), chunks * dv * kDeltaChunk * 4,
            chunks * delta_parts_bytes(kDeltaChunk, dk)};
}
}  // namespace

extern "C" size_t tern_gated_delta_workspace_bytes(int B, int T, int max_new, int v_heads, int dk, int dv) {
    int sms = 0;
    if (B < 1 || B > 65535 || T < 1 || max_new < 0 || v_heads < 1 || v_heads > 65535 || (dk != 64 && dk != 128) || dv < 16 ||
        dv % 16 != 0 || dv > 256 || check_device(&sms) != TERN_OK)
        return 0;
    const int count = delta_pieces(B, std::min(max_new, T), v_heads, dv, sms);
    const size_t bytes = count > 1 ? piece_sizes(count, B, T, v_heads, dk, dv).all() : 0;
    return bytes <= kMostWorkspace ? bytes : 0;
}

extern "C" tern_status tern_gated_delta(const void* q, const void* k, const void* v, long long q_token,
                                        long long k_token, long long v_token, const float* g, long long g_token,
                                        const float* beta, long long beta_token, const float* a_log,
                                        const float* dt_bias, float scale, int qk_norm, float* state, int pool,
                                        const int* slots, const int* dst_slots, const int* past, const int* q_start,
                                        int B, int T, int max_new, int k_heads, int v_heads, int dk, int dv, void* out,
                                        void* workspace, size_t workspace_bytes, tern_stream_t stream) {
    set_launch_count(0);
    DeltaArgs a;
    tern_status st = make_state_seq_view(q_start, slots, dst_slots, past, B, T, max_new, pool, &a.s);
    if (st != TERN_OK) return st;
    if ((dk != 64 && dk != 128) || dv < 16 || dv % 16 != 0 || dv > 256 || k_heads < 1 || v_heads < 1 || v_heads > 65535 ||
        v_heads % k_heads != 0 || !(fabsf(scale) < INFINITY))
        return TERN_ERR_SHAPE;
    const long long strides[5] = {q_token, k_token, v_token, g_token, beta_token};
    const long long least[5] = {(long long)k_heads * dk, (long long)k_heads * dk, (long long)v_heads * dv, v_heads, v_heads};
    for (int i = 0; i < 5; ++i)
        if (strides[i] < 0 || (T > 1 && strides[i] < least[i]) || strides[i] >= (1LL << 37) || (i < 3 && strides[i] % 8 != 0))
            return TERN_ERR_SHAPE;
    if (!state || (!a_log) != (!dt_bias) || (T > 0 && (!q || !k || !v || !g || !beta || !out))) return TERN_ERR_NULL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(state) || !aligned16(out) || !aligned_to(g, 4) ||
        !aligned_to(beta, 4) || !aligned_to(a_log, 4) || !aligned_to(dt_bias, 4) || !aligned_to(workspace, 256))
        return TERN_ERR_ALIGN;
    int sms = 0;
    st = check_device(&sms);
    if (st != TERN_OK) return st;
    a.p = DeltaPieces{1, nullptr, nullptr, nullptr, nullptr, nullptr};
    const size_t need = workspace ? tern_gated_delta_workspace_bytes(B, T, a.s.max_new, v_heads, dk, dv) : 0;
    if (workspace_bytes < need) return TERN_ERR_WORKSPACE;
    if (need > 0) {
        a.p.count = delta_pieces(B, a.s.max_new, v_heads, dv, sms);
        const PieceSizes sizes = piece_sizes(a.p.count, B, T, v_heads, dk, dv);
        unsigned char* at = static_cast<unsigned char*>(workspace);
        a.p.state = reinterpret_cast<float*>(at);
        a.p.move = at += sizes.state;
        a.p.parts = at += sizes.move;
        a.p.out = reinterpret_cast<float*>(at += sizes.parts);
        a.p.out_move = at + sizes.out;
    }
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.q_token = q_token;
    a.k_token = k_token;
    a.v_token = v_token;
    a.g = g;
    a.beta = beta;
    a.g_token = g_token;
    a.beta_token = beta_token;
    a.a_log = a_log;
    a.dt_bias = dt_bias;
    a.state = state;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.k_heads = k_heads;
    a.v_heads = v_heads;
    a.dk = dk;
    a.dv = dv;
    a.group = v_heads / k_heads;
    a.norm = qk_norm;
    a.scale = scale;
    a.by_length = q_start && (long long)((dv + kDeltaRows - 1) / kDeltaRows) * v_heads * B > sms;
    cudaError_t e = a.s.max_new > kStepTokens ? launch_delta_chunk(a, (cudaStream_t)stream)
                                              : launch_delta_step(a, (cudaStream_t)stream);
    if (e == cudaSuccess && a.p.count > 1) e = launch_delta_join(a, sms, (cudaStream_t)stream);
    if (e != cudaSuccess) return TERN_ERR_CUDA;
    set_launch_count(a.p.count == 1 ? 1 : a.p.count == 2 ? 2 : 3);
    return TERN_OK;
}
