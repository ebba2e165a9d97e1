// token_abi.cu -- the extern "C" entry points of the token operators
// (declared in include/bevpool.h): argument checks on the host, dispatch,
// status codes.
#include <cmath>

#include "paged_attention.cuh"

using namespace bevpool;

namespace {

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bevpool_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return BEVPOOL_OK;
    cudaGetLastError();   // clear the runtime's last-error slot
    return BEVPOOL_ERR_CUDA;
}

constexpr int64_t kMaxStride = static_cast<int64_t>(1) << 40;

bool stride_ok(int64_t s) { return s >= 0 && s < kMaxStride && s % 8 == 0; }

bool rows_ok(const void *p, int64_t ts, int64_t hs) { return p && aligned(p, 16) && stride_ok(ts) && stride_ok(hs); }

bool dtype_ok(bevpool_dtype d) { return d == BEVPOOL_F16 || d == BEVPOOL_BF16; }

// Sizes of head rows; head_dim out of the supported set is reported apart.
bevpool_status heads_ok(int32_t T, int32_t Hq, int32_t Hk, int32_t D) {
    if (T < 0 || Hq < 1 || Hk < 1 || Hq > 65535 || Hk > 65535 || D < 1) return BEVPOOL_ERR_INVALID_ARG;
    if (D % 8 != 0 || D < 32 || D > kMaxHeadDim) return BEVPOOL_ERR_UNSUPPORTED;
    return BEVPOOL_OK;
}

// The position arguments, into *r.
bool rotary_ok(const int32_t *positions, int32_t n_axes, const int32_t *sections, int32_t rotary_dim, const float *inv_freq,
               int32_t interleaved, int32_t D, RotaryArgs *r) {
    if (!positions || !aligned(positions, 4) || !inv_freq || !aligned(inv_freq, 4) || !sections) return false;
    if (n_axes < 1 || n_axes > kMaxAxes) return false;
    if (rotary_dim < 16 || rotary_dim > D || rotary_dim % 16 != 0) return false;
    r->positions = positions;
    r->inv_freq = inv_freq;
    r->n_axes = n_axes;
    r->rotary_dim = rotary_dim;
    r->interleaved = interleaved != 0;
    int32_t end = 0;
    for (int a = 0; a < kMaxAxes; ++a) {
        if (a < n_axes) {
            if (sections[a] < 0 || sections[a] > rotary_dim / 2 - end) return false;
            end += sections[a];
        }
        r->axis_end[a] = end;
    }
    return end == rotary_dim / 2;
}

bool eps_ok(float eps) { return std::isfinite(eps) && eps >= 0.0f; }

bool weight_ok(const float *w) { return aligned(w, 4); }

bool scale_ok(float s) { return std::isfinite(s) && s > 0.0f && std::isfinite(1.0f / s); }

// 1 / s as hi + lo, s > 0.  hi is rounded towards zero and lo is never zero (2^-60 of
// hi where hi is exact), so that an infinite value times either has its sign.
AppendArgs::Inverse inverse(float s) {
    const double inv = 1.0 / static_cast<double>(s);
    float hi = static_cast<float>(inv);
    if (hi > inv) hi = std::nextafter(hi, 0.0f);
    const float lo = static_cast<float>(std::fmax(inv - hi, hi * 0x1p-60));
    return {hi, std::fmax(lo, 0x1p-149f)};
}

// The cache arguments, into *g.  eb: bytes of an element.
bevpool_status cache_ok(const void *k_cache, const void *v_cache, int64_t page_stride, int64_t slot_stride,
                        int64_t head_stride, int32_t n_pages, int32_t page_size, const int32_t *block_table,
                        int32_t table_pages, const int32_t *kv_len, const int32_t *cu_q, int32_t n_seqs, int32_t Hk,
                        int32_t D, int eb, PagedArgs *g) {
    if (page_size < 1 || n_pages < 1 || table_pages < 1 || n_seqs < 0) return BEVPOOL_ERR_INVALID_ARG;
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) != 0) return BEVPOOL_ERR_UNSUPPORTED;
    const int64_t unit = 16 / eb;
    for (const int64_t s : {page_stride, slot_stride, head_stride})
        if (s < 0 || s >= kMaxStride / 2 || s % unit != 0) return BEVPOOL_ERR_INVALID_ARG;
    // rows must not overlap; the stride of an axis of one entry is never used
    if (slot_stride < D || (n_pages > 1 && page_stride < D) || (Hk > 1 && head_stride < D)) return BEVPOOL_ERR_INVALID_ARG;
    if (!k_cache || !v_cache || !aligned(k_cache, 16) || !aligned(v_cache, 16)) return BEVPOOL_ERR_INVALID_ARG;
    const int32_t *idx[] = {block_table, kv_len, cu_q};
    for (const int32_t *p : idx)
        if (!p || !aligned(p, 4)) return BEVPOOL_ERR_INVALID_ARG;
    if ((static_cast<int64_t>(table_pages) + 1) * page_size > INT32_MAX) return BEVPOOL_ERR_INVALID_ARG;
    g->page_stride = page_stride;
    g->slot_stride = slot_stride;
    g->head_stride = head_stride;
    g->n_pages = n_pages;
    g->page_size = page_size;
    g->page_shift = 0;
    while ((1 << g->page_shift) < page_size) ++g->page_shift;
    g->table_pages = table_pages;
    g->n_seqs = n_seqs;
    g->block_table = block_table;
    g->kv_len = kv_len;
    g->cu_q = cu_q;
    return BEVPOOL_OK;
}

}  // namespace

extern "C" {

bevpool_status bevpool_qk_norm_rope(
    bevpool_dtype dtype, const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k,
    int64_t k_token_stride, int64_t k_head_stride, int32_t n_tokens, int32_t n_q_heads, int32_t n_k_heads,
    int32_t head_dim, const float *q_weight, const float *k_weight, float eps, const int32_t *positions,
    int32_t n_axes, const int32_t *sections, int32_t rotary_dim, const float *inv_freq, int32_t interleaved,
    void *q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, void *k_out, int64_t k_out_token_stride,
    int64_t k_out_head_stride, void *stream) {
    if (!dtype_ok(dtype)) return BEVPOOL_ERR_UNSUPPORTED;
    const bevpool_status st = heads_ok(n_tokens, n_q_heads, n_k_heads, head_dim);
    if (st != BEVPOOL_OK) return st;
    if (n_tokens == 0) return BEVPOOL_OK;
    NormRopeArgs a = {};
    if (!rows_ok(q, q_token_stride, q_head_stride) || !rows_ok(k, k_token_stride, k_head_stride) ||
        !rows_ok(q_out, q_out_token_stride, q_out_head_stride) || !rows_ok(k_out, k_out_token_stride, k_out_head_stride) ||
        !weight_ok(q_weight) || !weight_ok(k_weight) || !eps_ok(eps) ||
        !rotary_ok(positions, n_axes, sections, rotary_dim, inv_freq, interleaved, head_dim, &a.rot))
        return BEVPOOL_ERR_INVALID_ARG;
    a.dtype = dtype;
    a.q = {q, q_token_stride, q_head_stride};
    a.k = {k, k_token_stride, k_head_stride};
    a.q_out = {q_out, q_out_token_stride, q_out_head_stride};
    a.k_out = {k_out, k_out_token_stride, k_out_head_stride};
    a.T = n_tokens;
    a.Hq = n_q_heads;
    a.Hk = n_k_heads;
    a.D = head_dim;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.eps = eps;
    a.stream = static_cast<cudaStream_t>(stream);
    return cuda_status(launch_norm_rope(a));
}

size_t bevpool_qk_norm_rope_backward_workspace_size(int32_t n_tokens, int32_t n_q_heads, int32_t n_k_heads,
                                                    int32_t head_dim) {
    if (heads_ok(n_tokens, n_q_heads, n_k_heads, head_dim) != BEVPOOL_OK) return 0;
    return static_cast<size_t>(norm_rope_back_ctas(n_tokens, n_q_heads, n_k_heads, head_dim)) * 2 * head_dim *
           sizeof(float);
}

bevpool_status bevpool_qk_norm_rope_backward(
    bevpool_dtype dtype, const void *dq_out, int64_t dq_out_token_stride, int64_t dq_out_head_stride,
    const void *dk_out, int64_t dk_out_token_stride, int64_t dk_out_head_stride, const void *q,
    int64_t q_token_stride, int64_t q_head_stride, const void *k, int64_t k_token_stride, int64_t k_head_stride,
    int32_t n_tokens, int32_t n_q_heads, int32_t n_k_heads, int32_t head_dim, const float *q_weight,
    const float *k_weight, float eps, const int32_t *positions, int32_t n_axes, const int32_t *sections,
    int32_t rotary_dim, const float *inv_freq, int32_t interleaved, void *dq, int64_t dq_token_stride,
    int64_t dq_head_stride, void *dk, int64_t dk_token_stride, int64_t dk_head_stride, float *dq_weight,
    float *dk_weight, void *workspace, size_t workspace_bytes, void *stream) {
    if (!dtype_ok(dtype)) return BEVPOOL_ERR_UNSUPPORTED;
    const bevpool_status st = heads_ok(n_tokens, n_q_heads, n_k_heads, head_dim);
    if (st != BEVPOOL_OK) return st;
    NormRopeBackArgs a = {};
    if (n_tokens == 0) {
        if (!weight_ok(dq_weight) || !weight_ok(dk_weight) || !q_weight != !dq_weight || !k_weight != !dk_weight)
            return BEVPOOL_ERR_INVALID_ARG;
        a.f.D = head_dim;
        a.f.Hq = n_q_heads;
        a.f.Hk = n_k_heads;
        a.f.stream = static_cast<cudaStream_t>(stream);
        a.dq_weight = dq_weight;
        a.dk_weight = dk_weight;
        return cuda_status(launch_norm_rope_back(a));
    }
    if (!rows_ok(q, q_token_stride, q_head_stride) || !rows_ok(k, k_token_stride, k_head_stride) ||
        !rows_ok(dq_out, dq_out_token_stride, dq_out_head_stride) ||
        !rows_ok(dk_out, dk_out_token_stride, dk_out_head_stride) || !rows_ok(dq, dq_token_stride, dq_head_stride) ||
        !rows_ok(dk, dk_token_stride, dk_head_stride) || !weight_ok(q_weight) || !weight_ok(k_weight) ||
        !weight_ok(dq_weight) || !weight_ok(dk_weight) || !eps_ok(eps) ||
        !rotary_ok(positions, n_axes, sections, rotary_dim, inv_freq, interleaved, head_dim, &a.f.rot))
        return BEVPOOL_ERR_INVALID_ARG;
    if (!q_weight != !dq_weight || !k_weight != !dk_weight) return BEVPOOL_ERR_INVALID_ARG;
    const size_t need = bevpool_qk_norm_rope_backward_workspace_size(n_tokens, n_q_heads, n_k_heads, head_dim);
    if ((q_weight || k_weight) && need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need))
        return BEVPOOL_ERR_WORKSPACE;
    a.f.dtype = dtype;
    a.f.q = {q, q_token_stride, q_head_stride};
    a.f.k = {k, k_token_stride, k_head_stride};
    a.f.q_out = {dq, dq_token_stride, dq_head_stride};
    a.f.k_out = {dk, dk_token_stride, dk_head_stride};
    a.f.T = n_tokens;
    a.f.Hq = n_q_heads;
    a.f.Hk = n_k_heads;
    a.f.D = head_dim;
    a.f.q_weight = q_weight;
    a.f.k_weight = k_weight;
    a.f.eps = eps;
    a.f.stream = static_cast<cudaStream_t>(stream);
    a.dq_out = {dq_out, dq_out_token_stride, dq_out_head_stride};
    a.dk_out = {dk_out, dk_out_token_stride, dk_out_head_stride};
    a.dq_weight = dq_weight;
    a.dk_weight = dk_weight;
    a.partial = static_cast<float *>(workspace);
    return cuda_status(launch_norm_rope_back(a));
}

bevpool_status bevpool_kv_append(
    bevpool_dtype dtype, bevpool_dtype cache_dtype, const void *k, int64_t k_token_stride, int64_t k_head_stride,
    const void *v, int64_t v_token_stride, int64_t v_head_stride, const void *q, int64_t q_token_stride,
    int64_t q_head_stride, int32_t n_tokens, int32_t n_q_heads, int32_t n_k_heads, int32_t head_dim,
    const float *q_weight, const float *k_weight, float eps, const int32_t *positions, int32_t n_axes,
    const int32_t *sections, int32_t rotary_dim, const float *inv_freq, int32_t interleaved, void *q_out,
    int64_t q_out_token_stride, int64_t q_out_head_stride, void *k_cache, void *v_cache, int64_t page_stride,
    int64_t slot_stride, int64_t head_stride, int32_t n_pages, int32_t page_size, const int32_t *block_table,
    int32_t table_pages, const int32_t *kv_len, const int32_t *cu_q, int32_t n_seqs, float k_scale, float v_scale,
    void *stream) {
    if (!dtype_ok(dtype) || (cache_dtype != dtype && cache_dtype != BEVPOOL_E4M3)) return BEVPOOL_ERR_UNSUPPORTED;
    const bool e4m3 = cache_dtype == BEVPOOL_E4M3;
    bevpool_status st = heads_ok(n_tokens, q ? n_q_heads : 1, n_k_heads, head_dim);
    if (st != BEVPOOL_OK) return st;
    if (n_tokens == 0) return BEVPOOL_OK;
    AppendArgs g = {};
    st = cache_ok(k_cache, v_cache, page_stride, slot_stride, head_stride, n_pages, page_size, block_table, table_pages,
                  kv_len, cu_q, n_seqs, n_k_heads, head_dim, e4m3 ? 1 : 2, &g.pg);
    if (st != BEVPOOL_OK) return st;
    if (!rows_ok(k, k_token_stride, k_head_stride) || !rows_ok(v, v_token_stride, v_head_stride) ||
        !weight_ok(q_weight) || !weight_ok(k_weight) || !eps_ok(eps) ||
        !rotary_ok(positions, n_axes, sections, rotary_dim, inv_freq, interleaved, head_dim, &g.f.rot))
        return BEVPOOL_ERR_INVALID_ARG;
    if (q && (!rows_ok(q, q_token_stride, q_head_stride) || !rows_ok(q_out, q_out_token_stride, q_out_head_stride)))
        return BEVPOOL_ERR_INVALID_ARG;
    if (e4m3 && (!scale_ok(k_scale) || !scale_ok(v_scale))) return BEVPOOL_ERR_INVALID_ARG;
    g.f.dtype = dtype;
    g.f.q = {q, q_token_stride, q_head_stride};
    g.f.k = {k, k_token_stride, k_head_stride};
    g.f.q_out = {q_out, q_out_token_stride, q_out_head_stride};
    g.f.T = n_tokens;
    g.f.Hq = q ? n_q_heads : 0;
    g.f.Hk = n_k_heads;
    g.f.D = head_dim;
    g.f.q_weight = q_weight;
    g.f.k_weight = k_weight;
    g.f.eps = eps;
    g.f.stream = static_cast<cudaStream_t>(stream);
    g.v = {v, v_token_stride, v_head_stride};
    g.cache_e4m3 = e4m3;
    g.k_cache = k_cache;
    g.v_cache = v_cache;
    if (e4m3) {
        g.k_inv = inverse(k_scale);
        g.v_inv = inverse(v_scale);
    }
    return cuda_status(launch_kv_append(g));
}

namespace {

bevpool_status attention_sizes_ok(int32_t n_seqs, int32_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t max_q_len,
                                  int32_t max_kv_len) {
    const bevpool_status st = heads_ok(T, Hq, Hk, D);
    if (st != BEVPOOL_OK) return st;
    if (D != 64 && D != 128) return BEVPOOL_ERR_UNSUPPORTED;
    if (Hq % Hk != 0 || n_seqs < 0 || n_seqs > 65535 || max_q_len < 0 || max_kv_len < 0) return BEVPOOL_ERR_INVALID_ARG;
    if (static_cast<int64_t>(T) * Hq > INT32_MAX || static_cast<int64_t>(max_q_len) * (Hq / Hk) > INT32_MAX - 1024 ||
        max_kv_len > INT32_MAX - 1024)
        return BEVPOOL_ERR_INVALID_ARG;
    return BEVPOOL_OK;
}

}  // namespace

size_t bevpool_paged_attention_workspace_size(int32_t n_seqs, int32_t n_tokens, int32_t n_q_heads, int32_t n_k_heads,
                                              int32_t head_dim, int32_t max_q_len, int32_t max_kv_len, int32_t window) {
    if (attention_sizes_ok(n_seqs, n_tokens, n_q_heads, n_k_heads, head_dim, max_q_len, max_kv_len) != BEVPOOL_OK ||
        window < 0)
        return 0;
    if (n_seqs == 0 || n_tokens == 0 || max_q_len == 0) return 0;
    return attention_workspace_bytes({n_seqs, n_tokens, n_q_heads, n_k_heads, head_dim, max_q_len, max_kv_len, window, 0});
}

bevpool_status bevpool_paged_attention(
    bevpool_dtype dtype, bevpool_dtype cache_dtype, const void *q, int64_t q_token_stride, int64_t q_head_stride,
    const void *k_cache, const void *v_cache, int64_t page_stride, int64_t slot_stride, int64_t head_stride,
    int32_t n_pages, int32_t page_size, const int32_t *block_table, int32_t table_pages, const int32_t *kv_len,
    const int32_t *cu_q, int32_t n_seqs, int32_t n_tokens, int32_t n_q_heads, int32_t n_k_heads, int32_t head_dim,
    int32_t max_q_len, int32_t max_kv_len, float scale, int32_t causal, int32_t window, float k_scale,
    float v_scale, void *out, int64_t out_token_stride, int64_t out_head_stride, float *lse, void *workspace,
    size_t workspace_bytes, void *stream) {
    if (!dtype_ok(dtype) || (cache_dtype != dtype && cache_dtype != BEVPOOL_E4M3)) return BEVPOOL_ERR_UNSUPPORTED;
    const bool e4m3 = cache_dtype == BEVPOOL_E4M3;
    bevpool_status st = attention_sizes_ok(n_seqs, n_tokens, n_q_heads, n_k_heads, head_dim, max_q_len, max_kv_len);
    if (st != BEVPOOL_OK) return st;
    if (n_tokens == 0 || n_seqs == 0 || max_q_len == 0) return BEVPOOL_OK;
    AttnArgs a = {};
    st = cache_ok(k_cache, v_cache, page_stride, slot_stride, head_stride, n_pages, page_size, block_table, table_pages,
                  kv_len, cu_q, n_seqs, n_k_heads, head_dim, e4m3 ? 1 : 2, &a.pg);
    if (st != BEVPOOL_OK) return st;
    if (!rows_ok(q, q_token_stride, q_head_stride) || !rows_ok(out, out_token_stride, out_head_stride) || !aligned(lse, 4))
        return BEVPOOL_ERR_INVALID_ARG;
    if (!e4m3) k_scale = v_scale = 1.0f;
    if (!(scale > 0.0f) || !scale_ok(k_scale) || !scale_ok(v_scale) || !std::isfinite(scale * k_scale * 1.4427f))
        return BEVPOOL_ERR_INVALID_ARG;
    if (window < 0 || (window > 0 && !causal)) return BEVPOOL_ERR_INVALID_ARG;
    const size_t need =
        attention_workspace_bytes({n_seqs, n_tokens, n_q_heads, n_k_heads, head_dim, max_q_len, max_kv_len, window, 0});
    if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return BEVPOOL_ERR_WORKSPACE;
    a.dtype = dtype;
    a.cache_e4m3 = e4m3;
    a.q = {q, q_token_stride, q_head_stride};
    a.out = {out, out_token_stride, out_head_stride};
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.T = n_tokens;
    a.Hq = n_q_heads;
    a.Hk = n_k_heads;
    a.G = n_q_heads / n_k_heads;
    a.D = head_dim;
    a.max_q_len = max_q_len;
    a.max_kv_len = max_kv_len;
    a.scale_log2 = static_cast<float>(static_cast<double>(scale) * k_scale * 1.4426950408889634);
    a.v_scale = v_scale;
    a.causal = causal != 0;
    a.window = window;
    a.lse = lse;
    a.stream = static_cast<cudaStream_t>(stream);
    return cuda_status(launch_paged_attention(a, workspace));
}

bevpool_status bevpool_attention_timeouts(int64_t *h_count) {
    if (!h_count) return BEVPOOL_ERR_INVALID_ARG;
    return cuda_status(attention_timeouts(h_count));
}

}  // extern "C"
