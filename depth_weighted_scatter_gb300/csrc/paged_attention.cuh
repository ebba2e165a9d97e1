// paged_attention.cuh -- arguments and shared device code of the attention
// over a paged cache.
#pragma once

#include "rotary.cuh"

namespace bevpool {

struct AttnArgs {
    int dtype, cache_e4m3;
    HeadRows q;
    HeadRowsOut out;
    const void *k_cache, *v_cache;
    PagedArgs pg;
    int32_t T, Hq, Hk, G, D;          // G = Hq / Hk
    int32_t max_q_len, max_kv_len;
    float scale_log2;                 // scale * k_scale * log2(e)
    float v_scale;
    int32_t causal, window;
    float *lse;
    void *workspace;
    cudaStream_t stream;
};
size_t attention_workspace_bytes(int32_t n_seqs, int32_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t max_q_len,
                                 int32_t max_kv_len);
cudaError_t launch_paged_attention(const AttnArgs &a);

// ---------------------------------------------------------------- device

// One request's bounds, from device arrays that may hold anything.
struct Request {
    int32_t q0, q_len, q_rows;        // first token, new tokens, those that are computed
    int32_t kv_len;                   // keys that may be seen
    int32_t pos0;                     // place of the first new token
};

__device__ __forceinline__ Request request_of(const AttnArgs &a, int b) {
    Request r;
    const int32_t c0 = a.pg.cu_q[b], c1 = a.pg.cu_q[b + 1];
    r.q0 = min(max(c0, 0), a.T);
    r.q_len = max(min(c1, a.T) - r.q0, 0);
    r.q_rows = min(r.q_len, a.max_q_len);
    const int32_t n = max(a.pg.kv_len[b], 0);
    const int64_t table = static_cast<int64_t>(a.pg.table_pages) << a.pg.page_shift;
    r.kv_len = static_cast<int32_t>(min(static_cast<int64_t>(min(n, a.max_kv_len)), table));
    r.pos0 = n - r.q_len;
    return r;
}

// Keys that token i of a request sees: [*lo, *hi).
__device__ __forceinline__ void seen_keys(const AttnArgs &a, const Request &r, int32_t i, int32_t *lo, int32_t *hi) {
    const int32_t pos = r.pos0 + i;
    *hi = a.causal ? min(max(pos + 1, 0), r.kv_len) : r.kv_len;
    *lo = a.window > 0 ? static_cast<int32_t>(max(static_cast<int64_t>(pos) - a.window + 1, static_cast<int64_t>(0))) : 0;
}

// E elements of a cache row as FP32.
template <typename T, bool E4M3, int E>
__device__ __forceinline__ void load_cache(const void *p, int64_t at, float *x) {
    if constexpr (E4M3) {
        const uint8_t *s = static_cast<const uint8_t *>(p) + at;
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(*reinterpret_cast<const uint16_t *>(s + i), __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            x[i] = f.x;
            x[i + 1] = f.y;
        }
    } else {
        const T *s = static_cast<const T *>(p) + at;
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = static_cast<float>(s[i]);
    }
}

// One query row over the keys [lo, hi) by one warp, element by element: lane l
// holds elements l*E .. l*E+E-1.  The running maximum *m (base 2), sum *l and
// acc follow the softmax; keys not seen are never touched.
template <typename T, bool E4M3, int D>
__device__ void attend_row(const AttnArgs &a, int b, int hk, const float *q, int32_t lo, int32_t hi, float *m, float *l,
                           float *acc) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int32_t *table = a.pg.block_table + static_cast<int64_t>(b) * a.pg.table_pages;
    for (int32_t j = lo; j < hi;) {
        const int32_t page = table[j >> a.pg.page_shift];
        const int32_t end = min(hi, ((j >> a.pg.page_shift) + 1) << a.pg.page_shift);
        if (page < 0 || page >= a.pg.n_pages) {
            j = end;
            continue;
        }
        int64_t at = page * a.pg.page_stride + (j & (a.pg.page_size - 1)) * a.pg.slot_stride + hk * a.pg.head_stride +
                     lane * E;
        for (; j < end; ++j, at += a.pg.slot_stride) {
            float k[E], v[E];
            load_cache<T, E4M3, E>(a.k_cache, at, k);
            load_cache<T, E4M3, E>(a.v_cache, at, v);
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < E; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            s *= a.scale_log2;
            const float mn = fmaxf(*m, s);
            const float base = mn == -INFINITY ? 0.0f : mn;
            const float r = exp2f(*m - base), p = exp2f(s - base);
            *m = mn;
            *l = fmaf(*l, r, p);
#pragma unroll
            for (int i = 0; i < E; ++i) acc[i] = fmaf(acc[i], r, p * v[i]);
        }
    }
}

}  // namespace bevpool
