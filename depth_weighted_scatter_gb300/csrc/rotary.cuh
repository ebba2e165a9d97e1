// rotary.cuh -- the head rows of the token operators: lane layout, rotary
// angles, norm and rotation of a row, and their device helpers.
//
// A head row of D elements is held by LPR lanes of a warp (LPR = the power of
// two from D / 8 up), 8 elements (16 bytes) a lane, so a warp holds
// 32 / LPR rows at once and every row is read and written once with 16-byte
// accesses.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "bevpool_internal.cuh"

namespace bevpool {

constexpr int kMaxAxes = 4;
constexpr int kMaxHeadDim = 256;

struct HeadRows {            // [token][head][D] rows, strides in elements
    const void *p;
    int64_t token_stride, head_stride;
};
struct HeadRowsOut {
    void *p;
    int64_t token_stride, head_stride;
};

struct RotaryArgs {
    const int32_t *positions;     // [T][n_axes]
    const float *inv_freq;        // [R / 2]
    int32_t n_axes;
    int32_t axis_end[kMaxAxes];   // first pair past axis a
    int32_t rotary_dim;
    int32_t interleaved;
};

struct PagedArgs {                // cache geometry, shared by append and attention
    int64_t page_stride, slot_stride, head_stride;
    int32_t n_pages, page_size, page_shift, table_pages, n_seqs;
    const int32_t *block_table, *kv_len, *cu_q;
};

// Norms and rotation of q and k (head_norm_rope.cu).
struct NormRopeArgs {
    int dtype;
    HeadRows q, k;
    HeadRowsOut q_out, k_out;
    int32_t T, Hq, Hk, D;
    const float *q_weight, *k_weight;
    float eps;
    RotaryArgs rot;
    cudaStream_t stream;
};
cudaError_t launch_norm_rope(const NormRopeArgs &a);

struct NormRopeBackArgs {
    NormRopeArgs f;               // q, k, weights, positions; q_out / k_out are dq / dk
    HeadRows dq_out, dk_out;
    float *dq_weight, *dk_weight;
    float *partial;               // workspace: [CTAs][2][D]
};
int norm_rope_back_ctas(int32_t T, int32_t Hq, int32_t Hk, int32_t D);
cudaError_t launch_norm_rope_back(const NormRopeBackArgs &a);

// Append to the paged cache (kv_append.cu).
struct AppendArgs {
    NormRopeArgs f;               // k_out unused; q.p null: no queries
    HeadRows v;
    int cache_e4m3;
    void *k_cache, *v_cache;
    PagedArgs pg;
    float k_scale, v_scale;
};
cudaError_t launch_kv_append(const AppendArgs &a);

// ---------------------------------------------------------------- device

// Eight 16-bit elements <-> FP32.
template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &w, float *x) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 f;
        if constexpr (std::is_same<T, __half>::value)
            f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
        else
            f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float *x) {
    return make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
}

// Eight FP32 values as E4M3 codes, nearest even, saturating.
__device__ __forceinline__ uint2 pack8_e4m3(const float *x) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i], x[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// Frequencies as fractions of a turn per position, 0.64 fixed point, into
// shared memory (one entry a pair).  With them the angle of any int32
// position is one wrapping 64-bit product: whole turns drop out exactly, and
// what is left is off by at most 2^-53 * |position| * inv_freq / (2 pi) turns.
__device__ __forceinline__ void load_turns(const RotaryArgs &r, unsigned long long *turns) {
    for (int p = threadIdx.x; p < r.rotary_dim / 2; p += blockDim.x) {
        double t = static_cast<double>(r.inv_freq[p]) * 0.15915494309189535;      // 1 / (2 pi)
        t -= floor(t);
        turns[p] = static_cast<unsigned long long>(t * 18446744073709551616.0);   // 2^64, saturating
    }
}

// cos and sin of position * inv_freq.
__device__ __forceinline__ void turn_cos_sin(unsigned long long turns, int32_t pos, float *c, float *s) {
    const uint32_t top = static_cast<uint32_t>((turns * static_cast<unsigned long long>(static_cast<long long>(pos))) >> 32);
    sincospif(static_cast<float>(static_cast<int32_t>(top)) * 4.656612873077393e-10f, s, c);   // half turns, 2^-31
}

__device__ __forceinline__ int pair_axis(const RotaryArgs &r, int p) {
    int a = 0;
#pragma unroll
    for (int i = 0; i < kMaxAxes - 1; ++i) a += (i < r.n_axes - 1 && p >= r.axis_end[i]) ? 1 : 0;
    return a;
}

// What lane c of a row needs of its 8 elements: cos, and sin with the sign its
// own element takes in  y = own * cos + partner * sin  (the forward turn);
// cos 1, sin 0 past rotary_dim.
template <bool IL>
__device__ __forceinline__ void lane_cos_sin(const RotaryArgs &r, const unsigned long long *turns, int64_t t, int c,
                                             float *cs, float *sn) {
    const int half = r.rotary_dim / 2;
    if (c * 8 >= r.rotary_dim) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            cs[i] = 1.0f;
            sn[i] = 0.0f;
        }
        return;
    }
    const int32_t *pos = r.positions + t * r.n_axes;
    if constexpr (IL) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = c * 4 + i;
            float cc, ss;
            turn_cos_sin(turns[p], pos[pair_axis(r, p)], &cc, &ss);
            cs[2 * i] = cs[2 * i + 1] = cc;
            sn[2 * i] = -ss;
            sn[2 * i + 1] = ss;
        }
    } else {
        const bool second = c * 8 >= half;
        const int p0 = c * 8 - (second ? half : 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float cc, ss;
            turn_cos_sin(turns[p0 + i], pos[pair_axis(r, p0 + i)], &cc, &ss);
            cs[i] = cc;
            sn[i] = second ? ss : -ss;
        }
    }
}

// The lane that holds the partner elements of lane c's (interleaved pairs are
// inside a lane).
template <bool IL>
__device__ __forceinline__ int partner_lane(const RotaryArgs &r, int c, int lane) {
    if (IL || c * 8 >= r.rotary_dim) return lane;
    return c * 8 < r.rotary_dim / 2 ? lane + r.rotary_dim / 16 : lane - r.rotary_dim / 16;
}

// Partner elements of a row's raw 16-bit words (a lane past rotary_dim gets
// its own, unused).
template <bool IL>
__device__ __forceinline__ uint4 partner_words(const uint4 &w, int src) {
    if constexpr (IL) {
        auto swap = [](uint32_t x) { return __byte_perm(x, x, 0x1032); };
        return make_uint4(swap(w.x), swap(w.y), swap(w.z), swap(w.w));
    } else {
        return make_uint4(__shfl_sync(0xffffffffu, w.x, src), __shfl_sync(0xffffffffu, w.y, src),
                          __shfl_sync(0xffffffffu, w.z, src), __shfl_sync(0xffffffffu, w.w, src));
    }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// 1 / sqrt(mean(x^2) + eps) of a row.
template <int LPR>
__device__ __forceinline__ float row_rstd(const float *x, float inv_d, float eps) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
    return rsqrtf(fmaf(row_sum<LPR>(s), inv_d, eps));
}

// Coefficients of a token for one of q, k: y_i = rstd * (a_i x_i + b_i x'_i),
// x' the partner elements.  weight null: ones.
__device__ __forceinline__ void row_coefs(const float *cs, const float *sn, const float *w, int c, int cp, bool il,
                                          float *a, float *b) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a[i] = cs[i] * (w ? w[c * 8 + i] : 1.0f);
        b[i] = sn[i] * (w ? w[cp * 8 + (il ? i ^ 1 : i)] : 1.0f);
    }
}

// One row: norm (if on) and turn, FP32 out.
template <typename T, int LPR, bool IL>
__device__ __forceinline__ void turn_row(const uint4 &w, int src, bool turned, const float *a, const float *b, bool norm,
                                         float inv_d, float eps, float *y) {
    float x[8], xp[8];
    const uint4 wp = partner_words<IL>(w, src);
    unpack8<T>(w, x);
    unpack8<T>(wp, xp);
    const float r = norm ? row_rstd<LPR>(x, inv_d, eps) : 1.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = r * (turned ? fmaf(b[i], xp[i], a[i] * x[i]) : a[i] * x[i]);
}

}  // namespace bevpool
