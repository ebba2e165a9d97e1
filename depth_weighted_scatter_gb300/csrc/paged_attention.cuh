// paged_attention.cuh -- arguments and shared device code of the attention
// over a paged cache.
#pragma once

#include "rotary.cuh"

namespace bevpool {

// What a cache holds: the heads' type; E4M3 codes of one scale; of a scale a page
// and key head.
enum { kCacheSame, kCacheE4M3, kCacheScaled };

struct AttnArgs {
    int dtype, cache;
    HeadRows q;
    HeadRowsOut out;
    const void *k_cache, *v_cache;
    const float *k_scales, *v_scales; // kCacheScaled: [n_pages][Hk]
    PagedArgs pg;
    int32_t T, Hq, Hk, G, D;          // G = Hq / Hk
    int32_t max_q_len, max_kv_len;
    float scale_log2;                 // scale * k_scale * log2(e)
    float v_scale;
    int32_t causal, window;
    float *lse;
    float *part_o;                    // partial results: [parts][D]; what a part is says the plan
    float *part_ml;                   // [parts][2]: maximum (base 2), sum
    int2 *cut;                        // shared tiles, [n_seqs][Hk][tiles]: first and last CTA that have a part; -1: one alone
    cudaStream_t stream;
};

struct AttnSizes {
    int32_t n_seqs, T, Hq, Hk, D, max_q_len, max_kv_len, window, causal, scaled;
};

// How one call is laid out, from its sizes alone.
struct AttnPlan {
    int32_t few;              // 1: at most 16 query rows a request and key head
    int32_t codes;            // 1: at most 8, over codes with page scales
    int32_t align;            // the first chunk starts at a multiple of this many keys, and has a multiple of it
    int32_t rows;             // query rows a request and key head, at most
    int32_t chunk;            // keys of one CTA
    int32_t n_chunks;         // CTAs along the keys; above 1 their results are joined by a second kernel: parts are
                              // [n_seqs][Hk][n_chunks][rows]
    int32_t tiles;            // many rows: pairs of row tiles a request and key head
    int32_t share;            // many rows: CTAs that share all pairs' blocks of keys evenly, or 0.  Parts are then
                              // [share][2][kPairRows]: of the pair that began before the CTA's share, of the one that goes on
    int64_t parts;            // rows of partial results
};
constexpr int32_t kPairRows = 256;     // rows of a pair of row tiles
constexpr int32_t kCodesCtas = 3;      // CTAs of attend_codes.cu that an SM holds
AttnPlan attention_plan(const AttnSizes &z);
cudaError_t launch_attend_few(const AttnArgs &a, const AttnPlan &pl);      // attend_few.cu
cudaError_t launch_attend_few_scaled(const AttnArgs &a, const AttnPlan &pl);       // attend_few_scaled.cu: kCacheScaled
cudaError_t launch_attend_codes(const AttnArgs &a, const AttnPlan &pl);    // attend_codes.cu: kCacheScaled, at most 8 rows
cudaError_t launch_attend_tile(const AttnArgs &a, const AttnPlan &pl);     // attend_tile.cu
cudaError_t launch_attend_tile_scaled_1(const AttnArgs &a, const AttnPlan &pl);    // attend_tile_scaled_*.cu: by the groups of a
cudaError_t launch_attend_tile_scaled_2(const AttnArgs &a, const AttnPlan &pl);    // block of keys that have scales of their own
cudaError_t launch_attend_tile_scaled_8(const AttnArgs &a, const AttnPlan &pl);
// Waits of each file's kernels that ran out, added to *count.
cudaError_t attend_codes_timeouts(int64_t *count);
cudaError_t attend_tile_timeouts(int64_t *count);
cudaError_t attend_tile_scaled_1_timeouts(int64_t *count);
cudaError_t attend_tile_scaled_2_timeouts(int64_t *count);
cudaError_t attend_tile_scaled_8_timeouts(int64_t *count);
cudaError_t attention_timeouts(int64_t *count);
cudaError_t launch_attend_join(const AttnArgs &a, const AttnPlan &pl);     // attend_join.cu: where there are parts

size_t attention_workspace_bytes(AttnSizes z);     // causal or not
cudaError_t launch_paged_attention(const AttnArgs &a, void *workspace);

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

// Where the keys of a request's chunks start, and how many chunks it has (one
// at least: it writes the rows that see nothing).
__device__ __forceinline__ int32_t chunks_of(const AttnArgs &a, const Request &r, const AttnPlan &pl, int32_t *base) {
    int32_t lo, hi, x;
    seen_keys(a, r, 0, &lo, &x);
    seen_keys(a, r, max(r.q_rows - 1, 0), &x, &hi);
    *base = min(lo, hi) / pl.align * pl.align;
    const int64_t n = (static_cast<int64_t>(hi) - *base + pl.chunk - 1) / pl.chunk;
    return static_cast<int32_t>(min(max(n, static_cast<int64_t>(1)), static_cast<int64_t>(pl.n_chunks)));
}

// 2^x, 2^-inf = 0; results below 2^-126 are zero.
__device__ __forceinline__ float pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Scales of a page and head as the products use them.  A key's score in base 2 is
// q.code * score, its weight in the product with the values' codes 2^(that + lift),
// and the sum takes the weights times `sum`, so that one exponential a key serves
// both although the values' scales differ.  Scales stay within [2^-48, 2^48], so the
// lift moves two keys at most 2^96 apart: what counts in the sum is no smaller than
// 2^-126 of the largest weight.
struct PageFactors {
    float score, lift, sum;
};

__device__ __forceinline__ PageFactors page_factors(float score, float ks, float vs) {
    PageFactors f;
    const float v = fminf(fmaxf(vs, 0x1p-48f), 0x1p48f);   // NaN: the least
    // never 0, as 0 * -inf is NaN; tiles of bf16 rows see to their factor besides (least_exponent)
    f.score = fmaxf(score * fminf(fmaxf(ks, 0x1p-48f), 0x1p48f), 0x1p-126f);
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(f.lift) : "f"(v));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(f.sum) : "f"(v));
    return f;
}

// Two E4M3 codes (low 16 bits) as two 16-bit values.
template <typename T>
__device__ __forceinline__ uint32_t widen2(uint32_t codes) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3);
    if constexpr (std::is_same<T, __half>::value) {
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        return pack2<T>(f.x, f.y);
    }
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
template <typename T, int C, int D>
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
        PageFactors f = {a.scale_log2, 0.0f, 1.0f};
        if constexpr (C == kCacheScaled) {
            const int64_t i = static_cast<int64_t>(page) * a.Hk + hk;
            f = page_factors(a.scale_log2, a.k_scales[i], a.v_scales[i]);
        }
        int64_t at = page * a.pg.page_stride + (j & (a.pg.page_size - 1)) * a.pg.slot_stride + hk * a.pg.head_stride +
                     lane * E;
        for (; j < end; ++j, at += a.pg.slot_stride) {
            float k[E], v[E];
            load_cache<T, C != kCacheSame, E>(a.k_cache, at, k);
            load_cache<T, C != kCacheSame, E>(a.v_cache, at, v);
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < E; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            s = C == kCacheScaled ? fmaf(s, f.score, f.lift) : s * a.scale_log2;
            const float mn = fmaxf(*m, s);
            const float base = mn == -INFINITY ? 0.0f : mn;
            const float r = exp2f(*m - base), p = exp2f(s - base);
            *m = mn;
            *l = fmaf(*l, r, C == kCacheScaled ? p * f.sum : p);
#pragma unroll
            for (int i = 0; i < E; ++i) acc[i] = fmaf(acc[i], r, p * v[i]);
        }
    }
}

// The keys [c0, c1) of one row again, by attend_row: *m, *l, acc (lane l:
// elements l*E ..).
template <typename T, int C, int D>
__device__ __noinline__ void redo_row(const AttnArgs &a, const Request &r, int b, int hk, int i, int h, int32_t c0,
                                      int32_t c1, float *m, float *l, float *acc) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const T *qp = static_cast<const T *>(a.q.p) + static_cast<int64_t>(r.q0 + i) * a.q.token_stride + h * a.q.head_stride +
                  lane * E;
    float q[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = static_cast<float>(qp[e]);
        acc[e] = 0.0f;
    }
    *m = -INFINITY;
    *l = 0.0f;
    int32_t lo, hi;
    seen_keys(a, r, i, &lo, &hi);
    attend_row<T, C, D>(a, b, hk, q, max(lo, c0), min(hi, c1), m, l, acc);
}

__device__ __forceinline__ int64_t part_row(const AttnArgs &a, const AttnPlan &pl, int b, int hk, int chunk, int row) {
    return ((static_cast<int64_t>(b) * a.Hk + hk) * pl.n_chunks + chunk) * pl.rows + row;
}

// The end of a row, held by a warp (lane l: elements l*E ..): to out and lse, or
// to the partial results' row `at`, if that is not below 0.
template <typename T, int E>
__device__ __forceinline__ void store_row(const AttnArgs &a, const Request &r, int i, int h, int64_t at, float m, float l,
                                          const float *acc) {
    const int lane = threadIdx.x & 31;
    if (at >= 0) {
        float *o = a.part_o + at * (32 * E) + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = acc[e];
        if (lane == 0) *reinterpret_cast<float2 *>(a.part_ml + at * 2) = make_float2(m, l);
        return;
    }
    const int64_t t = r.q0 + i;
    const bool some = !(l == 0.0f);
    const float inv = some ? a.v_scale / l : 0.0f;
    T *op = static_cast<T *>(a.out.p) + t * a.out.token_stride + h * a.out.head_stride + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t *>(op + e) = pack2<T>(acc[e] * inv, acc[e + 1] * inv);
    if (a.lse && lane == 0) a.lse[t * a.Hq + h] = some ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace bevpool
