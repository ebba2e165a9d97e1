// rotary.cuh -- the head rows of the token operators: lane layout, rotary
// angles, norm and rotation of a row, and their device helpers.
//
// A head row of D elements is held by LPR lanes of a warp (LPR = the power of
// two from D / 8 up), 8 elements a lane in two runs of four, so a warp holds
// 32 / LPR rows at once (a step).  A lane's two runs hold four whole pairs:
// elements 4c.. and rotary_dim/2 + 4c.. of lane c where pairs are split, 8c..
// where they are interleaved, so that the rotation needs no exchange between
// lanes; lanes past rotary_dim / 8 hold the unturned elements 8c...  Two FP32
// values go through one packed instruction.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "bevpool_internal.cuh"
#include "packed.cuh"

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
    struct Inverse {              // 1 / scale, in two parts of one sign
        float hi, lo;
    } k_inv, v_inv;
};
cudaError_t launch_kv_append(const AppendArgs &a);

// Append to a cache with scales of its own (kv_append_scaled.cu).
struct ScaledAppendArgs {
    AppendArgs g;                 // an E4M3 cache; k_inv, v_inv unused
    float *k_scales, *v_scales;   // [n_pages][Hk]
};
cudaError_t launch_append_scaled(const ScaledAppendArgs &a);

// ---------------------------------------------------------------- device

// Two 16-bit elements as two FP32 values in one register pair, and back.
template <typename T>
__device__ __forceinline__ uint64_t widen(uint32_t u) {
    if constexpr (std::is_same<T, __half>::value) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u));
        return pair(f.x, f.y);
    } else {
        return pair(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
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
__device__ __forceinline__ uint32_t pack(uint64_t v) {
    float a, b;
    unpair(v, &a, &b);
    return pack2<T>(a, b);
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float *x) {
    return make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
}

// Four FP32 values as E4M3 codes, nearest even, saturating.
__device__ __forceinline__ uint32_t pack4_e4m3(uint64_t u, uint64_t v) {
    float a, b, c, d;
    unpair(u, &a, &b);
    unpair(v, &c, &d);
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// A frequency as a fraction of a turn per position, 0.64 fixed point.  With it
// the angle of any int32 position is one wrapping 64-bit product: whole turns
// drop out exactly, and what is left is off by at most 2^-53 * |position| *
// inv_freq / (2 pi) turns.
__device__ __forceinline__ unsigned long long turn_of(float inv_freq) {
    double t = static_cast<double>(inv_freq) * 0.15915494309189535;          // 1 / (2 pi)
    t -= floor(t);
    return static_cast<unsigned long long>(t * 18446744073709551616.0);     // 2^64, saturating
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

// A lane's place in a row: its two runs of four elements start at e0 and e1.
struct LaneRow {
    int c, e0, e1;
    bool live, turned;
};

template <bool IL>
__device__ __forceinline__ LaneRow lane_row(const RotaryArgs &r, int D, int c) {
    LaneRow p;
    p.c = c;
    p.live = c * 8 < D;
    p.turned = c * 8 < r.rotary_dim;
    p.e0 = !IL && p.turned ? c * 4 : c * 8;
    p.e1 = !IL && p.turned ? r.rotary_dim / 2 + c * 4 : c * 8 + 4;
    return p;
}

// The 16-bit elements of a lane: words 0, 1 hold its first run, 2, 3 its second.
struct LaneWords {
    uint32_t w[4];
};

template <bool IL, typename T>
__device__ __forceinline__ void store_words(T *row, const LaneRow &p, const LaneWords &x) {
    if constexpr (IL) {
        *reinterpret_cast<uint4 *>(row + p.e0) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
    } else {
        *reinterpret_cast<uint2 *>(row + p.e0) = make_uint2(x.w[0], x.w[1]);
        *reinterpret_cast<uint2 *>(row + p.e1) = make_uint2(x.w[2], x.w[3]);
    }
}

template <bool IL, typename T>
__device__ __forceinline__ void store_lane(T *row, const LaneRow &p, const uint64_t *y) {
    LaneWords x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x.w[i] = pack<T>(y[i]);
    store_words<IL, T>(row, p, x);
}

template <bool IL>
__device__ __forceinline__ void store_lane_e4m3(uint8_t *row, const LaneRow &p, const uint64_t *y) {
    const uint32_t a = pack4_e4m3(y[0], y[1]), b = pack4_e4m3(y[2], y[3]);
    if constexpr (IL) {
        *reinterpret_cast<uint2 *>(row + p.e0) = make_uint2(a, b);
    } else {
        *reinterpret_cast<uint32_t *>(row + p.e0) = a;
        *reinterpret_cast<uint32_t *>(row + p.e1) = b;
    }
}

// The angles of a warp's token.  The 32 / LPR rows of a step share them, so a
// lane works out N of its row's four pairs and gets the others from the lanes
// at its place in the other rows.
template <int LPR>
struct LaneTurns {
    static constexpr int N = LPR / 8 > 0 ? LPR / 8 : 1;
    static constexpr int ROWS = 4 / N;                     // rows that share the work
    unsigned long long turns[N];
    int axis[N], pos[N];

    __device__ __forceinline__ LaneTurns(const RotaryArgs &r, const LaneRow &p, int rg) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int pr = p.c * 4 + (rg % ROWS) * N + i;
            turns[i] = p.turned ? turn_of(r.inv_freq[pr]) : 0;
            axis[i] = p.turned ? pair_axis(r, pr) : 0;
        }
    }
    // A token's positions, read a token ahead.
    __device__ __forceinline__ void read(const RotaryArgs &r, int64_t t) {
#pragma unroll
        for (int i = 0; i < N; ++i) pos[i] = r.positions[t * r.n_axes + axis[i]];
    }
    // cos and sin of the row's four pairs at these positions (1, 0 for an
    // unturned lane).
    __device__ __forceinline__ void cos_sin(const LaneRow &p, float *cs, float *sn) const {
        float c[N], s[N];
#pragma unroll
        for (int i = 0; i < N; ++i) turn_cos_sin(turns[i], pos[i], &c[i], &s[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (N == 4) {
                cs[i] = c[i];
                sn[i] = s[i];
            } else {
                cs[i] = __shfl_sync(0xffffffffu, c[i % N], p.c + (i / N) * LPR);
                sn[i] = __shfl_sync(0xffffffffu, s[i % N], p.c + (i / N) * LPR);
            }
        }
    }
};

// The weights of q and k in shared memory (ones where there is no weight).
struct RowWeights {
    float w[2][kMaxHeadDim];

    __device__ __forceinline__ void load(const float *q, const float *k, int D) {
        for (int i = threadIdx.x; i < kMaxHeadDim; i += blockDim.x) {
            w[0][i] = q && i < D ? q[i] : 1.0f;
            w[1][i] = k && i < D ? k[i] : 1.0f;
        }
    }
};

// A lane's two runs of a row of weights.
__device__ __forceinline__ void lane_weights(const float *w, const LaneRow &p, float *u, float *v) {
    const float4 a = *reinterpret_cast<const float4 *>(w + p.e0), b = *reinterpret_cast<const float4 *>(w + p.e1);
    u[0] = a.x, u[1] = a.y, u[2] = a.z, u[3] = a.w;
    v[0] = b.x, v[1] = b.y, v[2] = b.z, v[3] = b.w;
}

// A lane's factors: word pair i becomes  own * a[i] + other * b[i], where the
// other elements are word pair i ^ 2 (split pairs) or the two of the word
// swapped (interleaved).  u, v: the weights of its two runs.
template <bool IL>
__device__ __forceinline__ void lane_factors(const float *cs, const float *sn, const float *u, const float *v, uint64_t *a,
                                             uint64_t *b) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int x = 2 * i, y = x + 1;
        if constexpr (IL) {
            a[i] = pair(cs[i] * u[x], cs[i] * u[y]), b[i] = pair(-sn[i] * u[y], sn[i] * u[x]);
            a[i + 2] = pair(cs[i + 2] * v[x], cs[i + 2] * v[y]), b[i + 2] = pair(-sn[i + 2] * v[y], sn[i + 2] * v[x]);
        } else {
            a[i] = pair(cs[x] * u[x], cs[y] * u[y]), b[i] = pair(-sn[x] * v[x], -sn[y] * v[y]);
            a[i + 2] = pair(cs[x] * v[x], cs[y] * v[y]), b[i + 2] = pair(sn[x] * u[x], sn[y] * u[y]);
        }
    }
}

// own * a + other * b of a lane's elements.  FULL: the whole head is turned;
// else the other elements of an unturned lane are no partners (0 times an
// infinity must not reach it).
template <bool IL, bool FULL>
__device__ __forceinline__ void turn_lane(const uint64_t *x, const uint64_t *a, const uint64_t *b, bool turned, uint64_t *y) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint64_t other = x[i ^ 2];
        if constexpr (IL) {
            float p, q;
            unpair(x[i], &p, &q);
            other = pair(q, p);
        }
        const uint64_t own = mul2(x[i], a[i]);
        y[i] = FULL || turned ? fma2(other, b[i], own) : own;
    }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over a lane's elements of x * y.
__device__ __forceinline__ float lane_dot(const uint64_t *x, const uint64_t *y) {
    const uint64_t s = fma2(x[0], y[0], mul2(x[1], y[1])), t = fma2(x[2], y[2], mul2(x[3], y[3]));
    float a, b;
    unpair(add2(s, t), &a, &b);
    return a + b;
}

// One row: norm (if on) and turn, FP32 out.
template <typename T, int LPR, bool IL, bool FULL>
__device__ __forceinline__ void turn_row(const LaneWords &w, const LaneRow &p, const uint64_t *a, const uint64_t *b, bool norm,
                                         float inv_d, float eps, uint64_t *y) {
    uint64_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = widen<T>(w.w[i]);
    turn_lane<IL, FULL>(x, a, b, p.turned, y);
    if (norm) {                                            // the same for the whole grid
        const float r = rsqrtf(fmaf(row_sum<LPR>(lane_dot(x, x)), inv_d, eps));
        const uint64_t r2 = pair(r, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], r2);
    }
}

// What the warps of a launch take: token u / split, and part u % split of its
// steps.  32 bits hold it: split is 1 unless there are few tokens.
struct Units {
    uint32_t n, stride, first, split;

    __device__ __forceinline__ Units(int32_t T, int32_t s)
        : n(static_cast<uint32_t>(T) * s), stride(gridDim.x * kWarps), first(blockIdx.x * kWarps + (threadIdx.x >> 5)), split(s) {}
    __device__ __forceinline__ int32_t token(uint32_t u) const { return static_cast<int32_t>(split == 1 ? u : u / split); }
    __device__ __forceinline__ void steps(uint32_t u, int steps, int *s0, int *s1) const {
        *s0 = 0;
        *s1 = steps;
        if (split > 1) {
            const uint32_t part = u % split;
            *s0 = static_cast<int>(part * steps / split);
            *s1 = static_cast<int>((part + 1) * steps / split);
        }
    }
};

// Steps of a token's H rows: 32 / LPR rows each.
template <int LPR>
__host__ __device__ __forceinline__ int steps_of(int H) {
    return (H + 32 / LPR - 1) / (32 / LPR);
}

// The rows of a warp's units, one tensor's steps after the other's, read ahead
// into a ring in shared memory by asynchronous copies: STREAMS of 512 bytes a
// step, DEPTH steps in flight whatever tensor or token they belong to.
template <int LPR, int PARTS, int STREAMS, int DEPTH>
class RowStream {
public:
    static constexpr int RPS = 32 / LPR;
    static constexpr int BYTES = STREAMS * DEPTH * 512;    // of a warp

    struct Part {                          // one tensor (its STREAMS arrays)
        const char *p[STREAMS];
        int64_t token_bytes[STREAMS], head_bytes[STREAMS];
        int H, end;                        // its rows, and the first step past it

        __device__ __forceinline__ void set(int i, const HeadRows &r) {
            p[i] = static_cast<const char *>(r.p);
            token_bytes[i] = r.token_stride * 2;
            head_bytes[i] = r.head_stride * 2;
        }
    };

    __device__ __forceinline__ RowStream(const Units &units, const Part *parts, uint32_t ring, const LaneRow &row, int rg, int D)
        : units_(units), parts_(parts), exact_(D == LPR * 8), live_(row.live), c_(row.c), rg_(rg),
          dst_(ring + (threadIdx.x & 31) * 16), a0_(ring + rg * (LPR * 16) + row.e0 * 2),
          a1_(ring + rg * (LPR * 16) + row.e1 * 2), u_(units.first) {
        if (u_ < units_.n) {
            units_.steps(u_, parts_[PARTS - 1].end, &s_, &s1_);
            seek();
        }
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) fetch(i * (STREAMS * 512));
    }

    // The next step's rows; its place in the ring is filled again.
    __device__ __forceinline__ void next(LaneWords *x) {
        asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
        __syncwarp();
        const uint32_t a0 = a0_ + at_, a1 = a1_ + at_;
#pragma unroll
        for (int i = 0; i < STREAMS; ++i) {
            asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(x[i].w[0]), "=r"(x[i].w[1]) : "r"(a0 + i * 512) : "memory");
            asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(x[i].w[2]), "=r"(x[i].w[3]) : "r"(a1 + i * 512) : "memory");
        }
        __syncwarp();
        fetch(at_);
        at_ = at_ == (DEPTH - 1) * STREAMS * 512 ? 0 : at_ + STREAMS * 512;
    }

private:
    __device__ __forceinline__ void seek() {               // to step s_ of unit u_
        int part = 0;
#pragma unroll
        for (int i = 0; i < PARTS - 1; ++i) part += s_ >= parts_[i].end ? 1 : 0;
        const Part &q = parts_[part];
        const int64_t t = units_.token(u_);
        const int row = (s_ - (part ? parts_[part - 1].end : 0)) * RPS + rg_;
        left_ = min(q.end, s1_) - s_;
        s_ += left_;
        whole_ = exact_ && q.H % RPS == 0;
        rows_ = live_ ? (q.H - row + RPS - 1) / RPS : 0;   // steps in which this lane has a row
#pragma unroll
        for (int i = 0; i < STREAMS; ++i) {
            step_[i] = RPS * q.head_bytes[i];
            p_[i] = q.p[i] + t * q.token_bytes[i] + row * q.head_bytes[i] + c_ * 16;
        }
    }
    __device__ __forceinline__ void fetch(uint32_t at) {
        if (left_ > 0) {                                   // the same for the whole warp, as all branches here
            if (whole_) {
#pragma unroll
                for (int i = 0; i < STREAMS; ++i)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst_ + at + i * 512), "l"(p_[i]) : "memory");
            } else {
                const bool on = rows_ > 0;                 // else zeros
                --rows_;
#pragma unroll
                for (int i = 0; i < STREAMS; ++i)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst_ + at + i * 512),
                                 "l"(on ? p_[i] : parts_[0].p[0]), "r"(on ? 16 : 0)
                                 : "memory");
            }
            if (--left_ > 0) {
#pragma unroll
                for (int i = 0; i < STREAMS; ++i) p_[i] += step_[i];
            } else {
                if (s_ == s1_ && units_.n - u_ > units_.stride) {
                    u_ += units_.stride;
                    units_.steps(u_, parts_[PARTS - 1].end, &s_, &s1_);
                }
                if (s_ < s1_) seek();
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }

    const Units &units_;
    const Part *parts_;
    bool exact_, live_, whole_ = true;
    int c_, rg_;
    uint32_t dst_, a0_, a1_, u_, at_ = 0;
    int s_ = 0, s1_ = 0, left_ = 0, rows_ = 0;             // the step past this run of one tensor, and past the unit
    const char *p_[STREAMS];
    int64_t step_[STREAMS];
};

}  // namespace bevpool
