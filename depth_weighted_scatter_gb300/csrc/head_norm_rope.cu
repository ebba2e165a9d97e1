// head_norm_rope.cu -- norms of queries and keys for each head and their
// rotary positions in one pass, forward and backward.
//
// forward, row x with weight w:   y = turn(x * rstd * w),  rstd = 1/sqrt(mean(x^2)+eps)
// backward, dy the row's gradient: g = turn^-1(dy),  xh = x * rstd,
//     dx = rstd * (g w - xh * mean(g w xh)),   dw = sum over tokens and heads of g xh
//
// Both are bound by memory: the forward reads and writes each row once, the
// backward reads two rows and writes one.  A warp takes one token (or a slice
// of its rows, when there are few tokens): cos, sin and the weights are
// folded into two coefficients an element, once for all rows of the token, so
// a row costs its loads, one reduction and two multiply-adds an element.
#include "rotary.cuh"

namespace bevpool {

namespace {

// Rows of one kind (q or k) that a warp takes in one step.
template <int LPR>
constexpr int kRowsPerStep = 32 / LPR;

// Steps of a token: ceil(H / rows per step) for q, then for k.
template <int LPR>
__host__ __device__ __forceinline__ int steps_of(int H) {
    return (H + kRowsPerStep<LPR> - 1) / kRowsPerStep<LPR>;
}

template <typename T, int LPR, bool IL>
__device__ __forceinline__ void forward_rows(const HeadRows &in, const HeadRowsOut &out, int64_t t, int H, int s0, int s1,
                                             int c, int rg, bool live, int src, bool turned, const float *cs,
                                             const float *sn, const float *w, int cp, int D, float eps) {
    constexpr int U = 4;                                   // rows in flight a lane
    float a[8], b[8];
    if (live) row_coefs(cs, sn, w, c, cp, IL, a, b);
    const T *ip = static_cast<const T *>(in.p) + t * in.token_stride + c * 8;
    T *op = static_cast<T *>(out.p) + t * out.token_stride + c * 8;
    const float inv_d = 1.0f / static_cast<float>(D);
    for (int s = s0; s < s1; s += U) {
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = (s + u) * kRowsPerStep<LPR> + rg;
            const bool on = live && s + u < s1 && h < H;
            x[u] = on ? *reinterpret_cast<const uint4 *>(ip + h * in.head_stride) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u >= s1) break;                        // the same for the whole warp
            const int h = (s + u) * kRowsPerStep<LPR> + rg;
            float y[8];
            turn_row<T, LPR, IL>(x[u], src, turned, a, b, w != nullptr, inv_d, eps, y);
            if (live && h < H) *reinterpret_cast<uint4 *>(op + h * out.head_stride) = pack8<T>(y);
        }
    }
}

template <typename T, int LPR, bool IL>
__global__ void __launch_bounds__(kThreads)
k_norm_rope(NormRopeArgs a, int split) {
    __shared__ unsigned long long turns[kMaxHeadDim / 2];
    load_turns(a.rot, turns);
    __syncthreads();
    const int lane = threadIdx.x & 31, c = lane % LPR, rg = lane / LPR;
    const bool live = c * 8 < a.D;
    const int src = partner_lane<IL>(a.rot, c, lane), cp = c + src - lane;
    const bool turned = c * 8 < a.rot.rotary_dim;
    const int nq = steps_of<LPR>(a.Hq), n = nq + steps_of<LPR>(a.Hk);
    const int64_t units = static_cast<int64_t>(a.T) * split;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units;
         u += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t t = u / split;
        const int part = static_cast<int>(u - t * split);
        const int s0 = part * n / split, s1 = (part + 1) * n / split;
        float cs[8], sn[8];
        lane_cos_sin<IL>(a.rot, turns, t, c, cs, sn);
        if (s0 < nq)
            forward_rows<T, LPR, IL>(a.q, a.q_out, t, a.Hq, s0, min(s1, nq), c, rg, live, src, turned, cs, sn, a.q_weight,
                                     cp, a.D, a.eps);
        if (s1 > nq)
            forward_rows<T, LPR, IL>(a.k, a.k_out, t, a.Hk, max(s0 - nq, 0), s1 - nq, c, rg, live, src, turned, cs, sn,
                                     a.k_weight, cp, a.D, a.eps);
    }
}

template <typename T, int LPR, bool IL>
__device__ __forceinline__ void backward_rows(const HeadRows &grad, const HeadRows &in, const HeadRowsOut &out, int64_t t,
                                              int H, int s0, int s1, int c, int rg, bool live, int src, bool turned,
                                              const float *cs, const float *sn, const float *w, int D, float eps,
                                              float *dw) {
    constexpr int U = 2;                                   // rows in flight a lane, two loads each
    const T *gp = static_cast<const T *>(grad.p) + t * grad.token_stride + c * 8;
    const T *ip = static_cast<const T *>(in.p) + t * in.token_stride + c * 8;
    T *op = static_cast<T *>(out.p) + t * out.token_stride + c * 8;
    const float inv_d = 1.0f / static_cast<float>(D);
    float wt[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) wt[i] = live && w ? w[c * 8 + i] : 1.0f;
    for (int s = s0; s < s1; s += U) {
        uint4 gw[U], xw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = (s + u) * kRowsPerStep<LPR> + rg;
            const bool on = live && s + u < s1 && h < H;
            gw[u] = on ? *reinterpret_cast<const uint4 *>(gp + h * grad.head_stride) : make_uint4(0, 0, 0, 0);
            xw[u] = on && w ? *reinterpret_cast<const uint4 *>(ip + h * in.head_stride) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u >= s1) break;                        // the same for the whole warp
            const int h = (s + u) * kRowsPerStep<LPR> + rg;
            float g[8], gx[8], x[8];
            const uint4 pw = partner_words<IL>(gw[u], src);
            unpack8<T>(gw[u], g);
            unpack8<T>(pw, gx);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = turned ? fmaf(-sn[i], gx[i], cs[i] * g[i]) : g[i];
            if (w) {                                       // the same for the whole grid
                unpack8<T>(xw[u], x);
                const float r = row_rstd<LPR>(x, inv_d, eps);
                float dot = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[i] *= r;                             // xh
                    dw[i] = fmaf(g[i], x[i], dw[i]);
                    g[i] *= wt[i];
                    dot = fmaf(g[i], x[i], dot);
                }
                dot = row_sum<LPR>(dot) * inv_d;
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = r * fmaf(-x[i], dot, g[i]);
            }
            if (live && h < H) *reinterpret_cast<uint4 *>(op + h * out.head_stride) = pack8<T>(g);
        }
    }
}

// The weights' gradients are summed over a lane's rows in registers, over a
// warp by shuffles, over a CTA in shared memory, and over CTAs by k_sum_dw,
// always in the same order.
template <typename T, int LPR, bool IL>
__global__ void __launch_bounds__(kThreads)
k_norm_rope_back(NormRopeBackArgs a, int split) {
    __shared__ unsigned long long turns[kMaxHeadDim / 2];
    __shared__ float sums[kWarps][2][LPR * 8];
    const NormRopeArgs &f = a.f;
    load_turns(f.rot, turns);
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane % LPR, rg = lane / LPR;
    const bool live = c * 8 < f.D;
    const int src = partner_lane<IL>(f.rot, c, lane);
    const bool turned = c * 8 < f.rot.rotary_dim;
    const int nq = steps_of<LPR>(f.Hq), n = nq + steps_of<LPR>(f.Hk);
    const int64_t units = static_cast<int64_t>(f.T) * split;
    float dwq[8] = {}, dwk[8] = {};
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + warp; u < units;
         u += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t t = u / split;
        const int part = static_cast<int>(u - t * split);
        const int s0 = part * n / split, s1 = (part + 1) * n / split;
        float cs[8], sn[8];
        lane_cos_sin<IL>(f.rot, turns, t, c, cs, sn);
        if (s0 < nq)
            backward_rows<T, LPR, IL>(a.dq_out, f.q, f.q_out, t, f.Hq, s0, min(s1, nq), c, rg, live, src, turned, cs, sn,
                                      f.q_weight, f.D, f.eps, dwq);
        if (s1 > nq)
            backward_rows<T, LPR, IL>(a.dk_out, f.k, f.k_out, t, f.Hk, max(s0 - nq, 0), s1 - nq, c, rg, live, src, turned,
                                      cs, sn, f.k_weight, f.D, f.eps, dwk);
    }
    grid_dep_allow();
    if (!f.q_weight && !f.k_weight) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1) {
            dwq[i] += __shfl_xor_sync(0xffffffffu, dwq[i], o);
            dwk[i] += __shfl_xor_sync(0xffffffffu, dwk[i], o);
        }
        if (rg == 0) {
            sums[warp][0][c * 8 + i] = dwq[i];
            sums[warp][1][c * 8 + i] = dwk[i];
        }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < 2 * f.D; j += kThreads) {
        const int which = j >= f.D ? 1 : 0, d = j - which * f.D;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += sums[w][which][d];
        a.partial[static_cast<int64_t>(blockIdx.x) * 2 * f.D + j] = s;
    }
}

// dw[j] = sum over CTAs of partial[cta][j]; 32 columns a CTA, the CTAs' rows
// dealt to its warps.
__global__ void __launch_bounds__(kThreads)
k_sum_dw(const float *partial, int n, int D, float *dq_weight, float *dk_weight) {
    __shared__ float sums[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int j = blockIdx.x * 32 + lane;
    grid_dep_wait();
    float s = 0.0f;
    if (j < 2 * D) {
#pragma unroll 4
        for (int r = warp; r < n; r += kWarps) s += partial[static_cast<int64_t>(r) * 2 * D + j];
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && j < 2 * D) {
        s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += sums[w][lane];
        float *out = j < D ? dq_weight : dk_weight;
        if (out) out[j < D ? j : j - D] = s;
    }
}

// Warps a token: one, unless there are too few tokens to fill the GPU; then
// its rows are dealt to more (at most one step each).
int split_of(int64_t T, int steps) {
    constexpr int64_t want = 152 * 16;                     // warps that keep the GPU busy
    int64_t s = T > 0 ? div_up(want, T) : 1;
    if (s > steps) s = steps;
    return static_cast<int>(s < 1 ? 1 : s);
}

int lanes_per_row(int D) { return D <= 32 ? 4 : D <= 64 ? 8 : D <= 128 ? 16 : 32; }

int steps_for(int D, int H) {
    const int rows = 32 / lanes_per_row(D);
    return (H + rows - 1) / rows;
}

constexpr int64_t kForwardCtasMax = 152 * 8;               // 8 CTAs of 256 threads an SM
constexpr int64_t kBackCtasMax = 152 * 4;

template <typename F>
cudaError_t with_shape(int dtype, int D, bool il, F &&f) {
    auto by_il = [&](auto t, auto lpr) {
        return il ? f(t, lpr, std::true_type{}) : f(t, lpr, std::false_type{});
    };
    auto by_lpr = [&](auto t) {
        switch (lanes_per_row(D)) {
            case 4: return by_il(t, std::integral_constant<int, 4>{});
            case 8: return by_il(t, std::integral_constant<int, 8>{});
            case 16: return by_il(t, std::integral_constant<int, 16>{});
            default: return by_il(t, std::integral_constant<int, 32>{});
        }
    };
    return dtype == BEVPOOL_F16 ? by_lpr(__half{}) : by_lpr(__nv_bfloat16{});
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs &a) {
    const int split = split_of(a.T, steps_for(a.D, a.Hq) + steps_for(a.D, a.Hk));
    int64_t grid = div_up(static_cast<int64_t>(a.T) * split, kWarps);
    if (grid > kForwardCtasMax) grid = kForwardCtasMax;
    return with_shape(a.dtype, a.D, a.rot.interleaved != 0, [&](auto t, auto lpr, auto il) {
        k_norm_rope<decltype(t), decltype(lpr)::value, decltype(il)::value>
            <<<static_cast<int>(grid), kThreads, 0, a.stream>>>(a, split);
        count_launch();
        return cudaGetLastError();
    });
}

int norm_rope_back_ctas(int32_t T, int32_t Hq, int32_t Hk, int32_t D) {
    const int split = split_of(T, steps_for(D, Hq) + steps_for(D, Hk));
    const int64_t grid = div_up(static_cast<int64_t>(T) * split, kWarps);
    return static_cast<int>(grid < kBackCtasMax ? grid : kBackCtasMax);
}

cudaError_t launch_norm_rope_back(const NormRopeBackArgs &a) {
    const NormRopeArgs &f = a.f;
    const int split = split_of(f.T, steps_for(f.D, f.Hq) + steps_for(f.D, f.Hk));
    const int grid = norm_rope_back_ctas(f.T, f.Hq, f.Hk, f.D);
    if (grid > 0) {
        const cudaError_t e = with_shape(f.dtype, f.D, f.rot.interleaved != 0, [&](auto t, auto lpr, auto il) {
            k_norm_rope_back<decltype(t), decltype(lpr)::value, decltype(il)::value>
                <<<grid, kThreads, 0, f.stream>>>(a, split);
            count_launch();
            return cudaGetLastError();
        });
        if (e != cudaSuccess) return e;
    }
    if (!a.dq_weight && !a.dk_weight) return cudaSuccess;
    const cudaError_t e = launch_dependent(k_sum_dw, dim3(static_cast<unsigned>(div_up(2 * f.D, 32))), dim3(kThreads), 0,
                                           f.stream, static_cast<const float *>(a.partial), grid, f.D, a.dq_weight,
                                           a.dk_weight);
    if (e == cudaSuccess) count_launch();
    return e;
}

}  // namespace bevpool
