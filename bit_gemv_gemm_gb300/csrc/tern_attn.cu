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

// The rows kernel of the mass holds this many query rows of a sequence and head.
constexpr int kMassRows = 64;

// The scale of scores in powers of two.  One too small to matter becomes 1e-30,
// so that masked scores (-inf) stay -inf under it.
float to_log2(float scale) {
    const float s = scale * 1.44269504088896341f;
    return fabsf(s) < 1e-30f ? copysignf(1e-30f, s) : s;
}

// A window of all the keys that a sequence may have hides none.  (Without it the
// kernels' 32-bit first - window + 1 has no room to wrap.)
template <typename Args>
int useful_window(const Args& a, int window) {
    return window < (long long)a.s.width * a.c.page_size ? window : 0;
}

// few rows: bound by reading the cache and by latency, which suits mma.sync
// and warps that work alone; more rows, from 17 on: tcgen05 (20 rows a head over
// 32k keys, 4 sequences: 92 us, against 115 from the rows kernel with 32 rows an item);
// past one row tile the kernel with three S buffers, which at heads of 256 has room
// for two only and gains nothing (512 tokens over 32k keys: 245 us against 241)
enum class AttnKernel { rows, tiles, chunk };
AttnKernel attn_kernel(int max_new, int group, int head_dim) {
    if ((long long)max_new * group <= 16) return AttnKernel::rows;
    return max_new <= 128 / group || head_dim == 256 ? AttnKernel::tiles : AttnKernel::chunk;
}

tern_status check_heads(const CacheView& c, int q_heads, long long q_stride) {
    if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return TERN_ERR_SHAPE;
    if (q_heads < 1 || q_heads % c.kv_heads != 0 || q_heads / c.kv_heads > 64) return TERN_ERR_SHAPE;
    if (q_stride < (long long)q_heads * c.head_dim || q_stride % 8 != 0 || q_stride >= (1LL << 37))
        return TERN_ERR_SHAPE;
    return TERN_OK;
}

}  // namespace

}  // namespace tern

using namespace tern;

extern "C" size_t tern_paged_attention_workspace_bytes(int B, int T, int max_new, int q_heads, int kv_heads,
                                                       int head_dim) {
    if (B < 1 || T < 0 || max_new < 0 || kv_heads < 1 || q_heads < 1 || q_heads % kv_heads != 0 ||
        (head_dim != 64 && head_dim != 128 && head_dim != 256))
        return 0;
    // the longest sequence's tokens: the average at least (a call without q_start has all equal)
    const int most = std::max(std::min(max_new, T), T / B);
    const AttnKernel kernel = attn_kernel(most, q_heads / kv_heads, head_dim);
    return kAttnCounterBytes + (kernel == AttnKernel::rows    ? attn_rows_workspace(head_dim)
                                : kernel == AttnKernel::tiles ? attn_tiles_workspace(head_dim)
                                                              : attn_chunk_workspace(head_dim));
}

extern "C" tern_status tern_paged_attention(const void* q, long long q_stride, const void* k_cache,
                                            const void* v_cache, const tern_cache_layout* layout, const int* table,
                                            int table_width, const int* lens, const int* q_start, int B, int T,
                                            int max_new, int q_heads, float scale, int window, void* out, float* lse,
                                            void* workspace, size_t workspace_bytes, tern_stream_t stream) {
    set_launch_count(0);
    AttnArgs a;
    tern_status st = make_cache_view(layout, &a.c);
    if (st == TERN_OK) st = make_seq_view(table, table_width, a.c.page_size, lens, q_start, B, T, max_new, &a.s);
    if (st == TERN_OK) st = check_heads(a.c, q_heads, q_stride);
    if (st != TERN_OK) return st;
    if (window < 0 || !(fabsf(to_log2(scale)) < INFINITY)) return TERN_ERR_SHAPE;
    if (!k_cache || !v_cache || (T > 0 && (!q || !out))) return TERN_ERR_NULL;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned_to(lse, 4))
        return TERN_ERR_ALIGN;
    if (!workspace || workspace_bytes < tern_paged_attention_workspace_bytes(B, T, a.s.max_new, q_heads, a.c.kv_heads,
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
    a.scale_log2 = to_log2(scale);
    a.window = useful_window(a, window);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.counters = static_cast<unsigned*>(workspace);
    a.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + kAttnCounterBytes);
    const AttnKernel kernel = attn_kernel(a.s.max_new, a.group, a.c.head_dim);
    auto launch = kernel == AttnKernel::rows ? launch_attn_rows : kernel == AttnKernel::tiles ? launch_attn_tiles : launch_attn_chunk;
    const cudaError_t e = launch(a, k_cache, v_cache, sms, (cudaStream_t)stream);
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
    if (st == TERN_OK) st = make_seq_view(table, table_width, a.c.page_size, lens, q_start, B, T, max_new, &a.s);
    if (st == TERN_OK) st = check_heads(a.c, q_heads, q_stride);
    if (st != TERN_OK) return st;
    if (window < 0 || !(fabsf(to_log2(scale)) < INFINITY) || !(fabsf(decay) < INFINITY)) return TERN_ERR_SHAPE;
    if (!k_cache || !mass || !mass_out || (T > 0 && (!q || !lse))) return TERN_ERR_NULL;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned_to(lse, 4) || !aligned_to(mass, 4) ||
        !aligned_to(mass_out, 4))
        return TERN_ERR_ALIGN;
    int sms = 0;
    st = check_device(&sms);
    if (st != TERN_OK) return st;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.q_stride = q_stride;
    if (sms > kMaxSms) sms = kMaxSms;
    a.q_heads = q_heads;
    a.group = q_heads / a.c.kv_heads;
    a.tiles = 0;
    a.scale_log2 = to_log2(scale);
    a.window = useful_window(a, window);
    a.lse = lse;
    a.decay = decay;
    a.mass = mass;
    a.out = mass_out;
    const bool few = (long long)a.s.max_new * a.group <= kMassRows;
    const cudaError_t e = few ? launch_mass_rows(a, k_cache, sms, (cudaStream_t)stream)
                              : launch_mass_tiles(a, k_cache, sms, (cudaStream_t)stream);
    if (e != cudaSuccess) return TERN_ERR_CUDA;
    set_launch_count(1);
    return TERN_OK;
}
