// tern_attn.cu -- attention of new tokens over the paged cache, and the
// attention weight that each cached key received.
//
//   s_ij = scale q_i . k_j for the keys that query i sees,
//   o_i = sum_j exp(s_ij - lse_i) v_j,   lse_i = log sum_j exp(s_ij),
//   mass_j <- decay mass_j + sum_i exp(s_ij - lse_i)  (the queries of all the
//   heads that share key j's head).
#include <algorithm>

#include "tern_attn.cuh"

namespace tern {
namespace {

__device__ int g_attn_error;

struct MassArgs {
    const __nv_bfloat16* q;
    long long q_stride;
    const __nv_bfloat16* k_cache;
    CacheView c;
    SeqView s;
    int q_heads;
    float scale;
    int window;
    const float* lse;
    float decay;
    const float* mass;
    float* out;
};

// One warp a (sequence, key head, key): it runs over the queries that see it.
template <int D>
__global__ void __launch_bounds__(256) mass_kernel(const MassArgs a) {
    constexpr int E = D / 32;
    pdl_launch_dependents();
    pdl_wait();
    const int b = blockIdx.z, hk = blockIdx.y, lane = threadIdx.x & 31, group = a.q_heads / a.c.kv_heads;
    const Seq q = load_seq(a.s, a.c.page_size, b, &g_attn_error);
    for (int j = blockIdx.x * 8 + (threadIdx.x >> 5); j < q.len; j += gridDim.x * 8) {
        const int page = checked_page(a.s.table[(long long)b * a.s.width + j / a.c.page_size], a.c.pages, &g_attn_error);
        const int slot = j % a.c.page_size;
        const long long at = page * a.c.page_stride + hk * a.c.head_stride + slot * a.c.slot_stride + lane * E;
        float k[E], sum = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) k[e] = __bfloat162float(a.k_cache[at + e]);
        // key j is seen by positions j .. j + window - 1
        const int i0 = max(j - (q.len - q.n), 0);
        const int i1 = a.window > 0 ? (int)min((long long)q.n, (long long)j - (q.len - q.n) + a.window) : q.n;
        for (int i = i0; i < i1; ++i)
            for (int g = 0; g < group; ++g) {
                const int h = hk * group + g;
                const __nv_bfloat16* qp = a.q + (long long)(q.q0 + i) * a.q_stride + (long long)h * D + lane * E;
                float s = 0.0f;
#pragma unroll
                for (int e = 0; e < E; ++e) s = fmaf(__bfloat162float(qp[e]), k[e], s);
#pragma unroll
                for (int r = 16; r; r >>= 1) s += __shfl_xor_sync(0xffffffffu, s, r);
                const float lse = a.lse[(long long)(q.q0 + i) * a.q_heads + h];
                if (lse > -INFINITY) sum += expf(s * a.scale - lse);
            }
        if (lane == 0) {
            const long long m = ((long long)page * a.c.kv_heads + hk) * a.c.page_size + slot;
            a.out[m] = a.decay * a.mass[m] + sum;
        }
    }
}

tern_status check_heads(const CacheView& c, int q_heads, long long q_stride) {
    if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return TERN_ERR_SHAPE;
    if (q_heads < 1 || q_heads % c.kv_heads != 0 || q_heads / c.kv_heads > 64) return TERN_ERR_SHAPE;
    if (q_stride < (long long)q_heads * c.head_dim || q_stride % 8 != 0) return TERN_ERR_SHAPE;
    return TERN_OK;
}

}  // namespace

cudaError_t read_attn_device_error(int* code) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_attn_error, sizeof(int));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_attn_error, &zero, sizeof(int));
}

}  // namespace tern

using namespace tern;

extern "C" size_t tern_paged_attention_workspace_bytes(int B, int T, int max_new, int q_heads, int kv_heads,
                                                       int head_dim) {
    if (B < 1 || T < 0 || max_new < 0 || kv_heads < 1 || q_heads < 1 || q_heads % kv_heads != 0 ||
        (head_dim != 64 && head_dim != 128 && head_dim != 256))
        return 0;
    return kAttnCounterBytes + std::max(attn_rows_workspace(), attn_tiles_workspace());
}

extern "C" tern_status tern_paged_attention(const void* q, long long q_stride, const void* k_cache,
                                            const void* v_cache, const tern_cache_layout* layout, const int* table,
                                            int table_width, const int* lens, const int* q_start, int B, int T,
                                            int max_new, int q_heads, float scale, int window, void* out, float* lse,
                                            void* workspace, size_t workspace_bytes, tern_stream_t stream) {
    set_launch_count(0);
    AttnArgs a;
    tern_status st = make_cache_view(layout, &a.c);
    if (st == TERN_OK) st = make_seq_view(table, table_width, lens, q_start, B, T, max_new, &a.s);
    if (st == TERN_OK) st = check_heads(a.c, q_heads, q_stride);
    if (st != TERN_OK) return st;
    if (window < 0 || !(fabsf(scale) < INFINITY)) return TERN_ERR_SHAPE;
    if (!k_cache || !v_cache || (T > 0 && (!q || !out))) return TERN_ERR_NULL;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned_to(lse, 4))
        return TERN_ERR_ALIGN;
    if (!workspace || workspace_bytes < tern_paged_attention_workspace_bytes(B, T, max_new, q_heads, a.c.kv_heads,
                                                                             a.c.head_dim))
        return TERN_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return TERN_ERR_ALIGN;
    int sms = 0;
    st = check_device(&sms);
    if (st != TERN_OK) return st;
    if (sms > kMaxSms) sms = kMaxSms;
    if (a.s.max_new == 0 || T == 0) return TERN_OK;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.q_stride = q_stride;
    a.q_heads = q_heads;
    a.group = q_heads / a.c.kv_heads;
    // (0 becomes a number that scores cannot notice: -inf times it is still -inf)
    a.scale_log2 = scale == 0.0f ? 1e-30f : scale * 1.44269504088896341f;
    a.window = window;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.counters = static_cast<unsigned*>(workspace);
    a.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + kAttnCounterBytes);
    const long long rows = (long long)a.s.max_new * a.group;
    // few rows: bound by reading the cache, which the rows kernel does once for
    // 32 rows (16 at D = 256); more rows: the tensor cores
    const bool few = rows <= (a.c.head_dim == 256 ? 16 : 32);
    const cudaError_t e = few ? launch_attn_rows(a, k_cache, v_cache, sms, (cudaStream_t)stream)
                              : launch_attn_tiles(a, k_cache, v_cache, sms, (cudaStream_t)stream);
    if (e != cudaSuccess) return TERN_ERR_CUDA;
    set_launch_count(1);
    return TERN_OK;
}

extern "C" tern_status tern_attention_mass(const void* q, long long q_stride, const void* k_cache,
                                           const tern_cache_layout* layout, const int* table, int table_width,
                                           const int* lens, const int* q_start, int B, int T, int max_new, int q_heads,
                                           float scale, int window, const float* lse, float decay, const float* mass,
                                           float* mass_out, tern_stream_t stream) {
    set_launch_count(0);
    MassArgs a;
    tern_status st = make_cache_view(layout, &a.c);
    if (st == TERN_OK) st = make_seq_view(table, table_width, lens, q_start, B, T, max_new, &a.s);
    if (st == TERN_OK) st = check_heads(a.c, q_heads, q_stride);
    if (st != TERN_OK) return st;
    if (window < 0 || !(fabsf(scale) < INFINITY) || !(fabsf(decay) < INFINITY)) return TERN_ERR_SHAPE;
    if (!k_cache || !mass || !mass_out || (T > 0 && (!q || !lse))) return TERN_ERR_NULL;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned_to(lse, 4) || !aligned_to(mass, 4) ||
        !aligned_to(mass_out, 4))
        return TERN_ERR_ALIGN;
    int sms = 0;
    st = check_device(&sms);
    if (st != TERN_OK) return st;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.q_stride = q_stride;
    a.k_cache = static_cast<const __nv_bfloat16*>(k_cache);
    a.q_heads = q_heads;
    a.scale = scale;
    a.window = window;
    a.lse = lse;
    a.decay = decay;
    a.mass = mass;
    a.out = mass_out;
    const long long keys = (long long)table_width * a.c.page_size;
    const int grid = (int)((keys + 7) / 8 < 4096 ? (keys + 7) / 8 : 4096);
    auto kernel = a.c.head_dim == 64 ? mass_kernel<64> : a.c.head_dim == 128 ? mass_kernel<128> : mass_kernel<256>;
    if (launch_pdl(kernel, dim3(grid, a.c.kv_heads, B), dim3(256), 0, (cudaStream_t)stream, true, a) != cudaSuccess)
        return TERN_ERR_CUDA;
    set_launch_count(1);
    return TERN_OK;
}
