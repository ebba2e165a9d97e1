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
// folded into two factors an element, once for all rows of the token, so a row
// costs one reduction and two multiply-adds an element.  Its rows come through
// a ring of asynchronous copies that runs on over tensors and tokens (plain
// loads, some in registers ahead, left the memory idle at each token's start:
// backward 115 us against 86 below).  What is left over the bytes is
// instructions: about 130 a step of 512 bytes, 60 % of the issue slots; and the start of
// a CTA: the frequencies as turns, in FP64, come before its first copies and hold the
// FP64 unit for 4600 cycles an SM (forward, heads of 128; backward 3100).
//
// Measured on a GB300, q and k of one fused projection: forward of 20001 tokens,
// 40 heads of 128, bf16: 80 us (5.2 TB/s of 6.7 measured copy); backward of
// 32768 tokens, 18 heads of 128, bf16: 86 us in the kernel (5.2 TB/s).
#include "rotary.cuh"

namespace bevpool {

namespace {

constexpr int kForwardDepth = 8, kBackDepth = 4;  // steps in flight a warp

template <typename T, int LPR, bool IL, bool FULL>
__global__ void __launch_bounds__(kThreads, 3)
k_norm_rope(NormRopeArgs a, int split) {
    using Stream = RowStream<LPR, 2, 1, kForwardDepth>;
    __shared__ __align__(16) RowWeights weights;
    __shared__ __align__(16) uint8_t ring[kWarps * Stream::BYTES];
    __shared__ typename Stream::Part parts[2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rg = lane / LPR;
    weights.load(a.q_weight, a.k_weight, a.D);
    if (threadIdx.x == 0) {
        parts[0].set(0, a.q);
        parts[1].set(0, a.k);
        parts[0].H = a.Hq, parts[0].end = steps_of<LPR>(a.Hq);
        parts[1].H = a.Hk, parts[1].end = parts[0].end + steps_of<LPR>(a.Hk);
    }
    const LaneRow p = lane_row<IL>(a.rot, a.D, lane % LPR);
    LaneTurns<LPR> turns(a.rot, p, rg);
    __syncthreads();
    const Units units(a.T, split);
    if (units.first < units.n) turns.read(a.rot, units.token(units.first));
    Stream in(units, parts, static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + warp * Stream::BYTES, p, rg, a.D);
    const float inv_d = 1.0f / static_cast<float>(a.D);
    const int nq = parts[0].end, steps = parts[1].end;
    for (uint32_t u = units.first; u < units.n; u += units.stride) {
        const int64_t t = units.token(u);
        int s0, s1;
        units.steps(u, steps, &s0, &s1);
        float cs[4], sn[4];
        turns.cos_sin(p, cs, sn);
        if (units.n - u > units.stride) turns.read(a.rot, units.token(u + units.stride));
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            const int end = part ? s1 : min(s1, nq), first = part ? max(s0, nq) : s0;
            if (first >= end) continue;
            uint64_t fa[4], fb[4];
            float wu[4], wv[4];
            lane_weights(weights.w[part], p, wu, wv);
            lane_factors<IL>(cs, sn, wu, wv, fa, fb);
            const HeadRowsOut &o = part ? a.k_out : a.q_out;
            const bool norm = (part ? a.k_weight : a.q_weight) != nullptr;
            const int H = part ? a.Hk : a.Hq;
            const int h = (part ? first - nq : first) * Stream::RPS + rg;
            int rows = p.live ? (H - h + Stream::RPS - 1) / Stream::RPS : 0;   // steps in which this lane has a row
            T *op = static_cast<T *>(o.p) + t * o.token_stride + h * o.head_stride;
            const int64_t step = Stream::RPS * o.head_stride;
            for (int s = first; s < end; ++s) {
                LaneWords x;
                in.next(&x);
                uint64_t y[4];
                turn_row<T, LPR, IL, FULL>(x, p, fa, fb, norm, inv_d, a.eps, y);
                if (rows-- > 0) store_lane<IL, T>(op, p, y);
                op += step;
            }
        }
    }
}

// The weights' gradients are summed over a lane's rows in registers, over a
// warp by shuffles, over a CTA in shared memory, and over CTAs by k_sum_dw,
// always in the same order.
template <typename T, int LPR, bool IL, bool FULL>
__global__ void __launch_bounds__(kThreads, 2)
k_norm_rope_back(NormRopeBackArgs a, int split) {
    using Stream = RowStream<LPR, 2, 2, kBackDepth>;
    __shared__ __align__(16) RowWeights weights;
    __shared__ __align__(16) uint8_t ring[kWarps * Stream::BYTES];
    __shared__ typename Stream::Part parts[2];
    static_assert(sizeof(ring) >= kWarps * 2 * LPR * 8 * sizeof(float), "the warps' sums fit the ring");
    const NormRopeArgs &f = a.f;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rg = lane / LPR;
    weights.load(f.q_weight, f.k_weight, f.D);
    if (threadIdx.x == 0) {
        // without a norm the inputs are not needed: the gradient's rows stand in
        parts[0].set(0, a.dq_out);
        parts[0].set(1, f.q_weight ? f.q : a.dq_out);
        parts[1].set(0, a.dk_out);
        parts[1].set(1, f.k_weight ? f.k : a.dk_out);
        parts[0].H = f.Hq, parts[0].end = steps_of<LPR>(f.Hq);
        parts[1].H = f.Hk, parts[1].end = parts[0].end + steps_of<LPR>(f.Hk);
    }
    const LaneRow p = lane_row<IL>(f.rot, f.D, lane % LPR);
    LaneTurns<LPR> turns(f.rot, p, rg);
    __syncthreads();
    const Units units(f.T, split);
    if (units.first < units.n) turns.read(f.rot, units.token(units.first));
    Stream in(units, parts, static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + warp * Stream::BYTES, p, rg, f.D);
    const float inv_d = 1.0f / static_cast<float>(f.D);
    const int nq = parts[0].end, steps = parts[1].end;
    uint64_t dw[2][4] = {};                                // all bits zero: two FP32 zeros
    for (uint32_t u = units.first; u < units.n; u += units.stride) {
        const int64_t t = units.token(u);
        int s0, s1;
        units.steps(u, steps, &s0, &s1);
        float cs[4], sn[4];
        turns.cos_sin(p, cs, sn);
        if (units.n - u > units.stride) turns.read(f.rot, units.token(u + units.stride));
#pragma unroll
        for (int i = 0; i < 4; ++i) sn[i] = -sn[i];        // the turn by the negative angle
        const float one[4] = {1.0f, 1.0f, 1.0f, 1.0f};
        uint64_t fa[4], fb[4];
        lane_factors<IL>(cs, sn, one, one, fa, fb);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            const int end = part ? s1 : min(s1, nq), first = part ? max(s0, nq) : s0;
            if (first >= end) continue;
            float wu[4], wv[4];
            lane_weights(weights.w[part], p, wu, wv);
            const uint64_t wt[4] = {pair(wu[0], wu[1]), pair(wu[2], wu[3]), pair(wv[0], wv[1]), pair(wv[2], wv[3])};
            const HeadRowsOut &o = part ? f.k_out : f.q_out;
            const bool norm = (part ? f.k_weight : f.q_weight) != nullptr;
            const int H = part ? f.Hk : f.Hq;
            const int h = (part ? first - nq : first) * Stream::RPS + rg;
            int rows = p.live ? (H - h + Stream::RPS - 1) / Stream::RPS : 0;   // steps in which this lane has a row
            T *op = static_cast<T *>(o.p) + t * o.token_stride + h * o.head_stride;
            const int64_t step = Stream::RPS * o.head_stride;
            for (int s = first; s < end; ++s) {
                LaneWords r[2];
                in.next(r);
                uint64_t d[4], g[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = widen<T>(r[0].w[i]);
                turn_lane<IL, FULL>(d, fa, fb, p.turned, g);
                if (norm) {                                // the same for the whole grid
                    uint64_t x[4], m[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[i] = widen<T>(r[1].w[i]);
                        m[i] = mul2(g[i], wt[i]);
                    }
                    // both sums of the row at once: x^2, and g w x
                    float sq = lane_dot(x, x), dot = lane_dot(m, x);
#pragma unroll
                    for (int k = LPR / 2; k > 0; k >>= 1) {
                        sq += __shfl_xor_sync(0xffffffffu, sq, k);
                        dot += __shfl_xor_sync(0xffffffffu, dot, k);
                    }
                    // a lane without a row has read zeros: with eps = 0 their
                    // rsqrt is infinite, and 0 * inf would reach the sums
                    const float rs = rows > 0 ? rsqrtf(fmaf(sq, inv_d, f.eps)) : 0.0f;
                    const float c = -dot * inv_d * rs * rs;
                    const uint64_t r2 = pair(rs, rs), c2 = pair(c, c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        dw[part][i] = fma2(mul2(x[i], r2), g[i], dw[part][i]);
                        g[i] = mul2(fma2(x[i], c2, m[i]), r2);         // rs (g w - xh mean(g w xh))
                    }
                }
                if (rows-- > 0) store_lane<IL, T>(op, p, g);
                op += step;
            }
        }
    }
    grid_dep_allow();
    if (!f.q_weight && !f.k_weight) return;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    float *sums = reinterpret_cast<float *>(ring);         // [warp][2][LPR * 8]
#pragma unroll
    for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[2];
            unpair(dw[part][i], &v[0], &v[1]);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int k = LPR; k < 32; k <<= 1) v[x] += __shfl_xor_sync(0xffffffffu, v[x], k);
                if (rg == 0 && p.live) sums[(warp * 2 + part) * (LPR * 8) + (i < 2 ? p.e0 : p.e1) + 2 * (i & 1) + x] = v[x];
            }
        }
    __syncthreads();
    for (int j = threadIdx.x; j < 2 * f.D; j += kThreads) {
        const int part = j >= f.D ? 1 : 0, d = j - part * f.D;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += sums[(w * 2 + part) * (LPR * 8) + d];
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

constexpr int64_t kForwardCtasMax = 152 * 3;               // 3 CTAs of 256 threads an SM, one wave
constexpr int64_t kBackCtasMax = 152 * 2;

template <typename F>
cudaError_t with_shape(int dtype, int D, const RotaryArgs &r, F &&f) {
    auto by_full = [&](auto t, auto lpr, auto il) {
        return r.rotary_dim == D ? f(t, lpr, il, std::true_type{}) : f(t, lpr, il, std::false_type{});
    };
    auto by_il = [&](auto t, auto lpr) {
        return r.interleaved ? by_full(t, lpr, std::true_type{}) : by_full(t, lpr, std::false_type{});
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
    return with_shape(a.dtype, a.D, a.rot, [&](auto t, auto lpr, auto il, auto full) {
        k_norm_rope<decltype(t), decltype(lpr)::value, decltype(il)::value, decltype(full)::value>
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
        const cudaError_t e = with_shape(f.dtype, f.D, f.rot, [&](auto t, auto lpr, auto il, auto full) {
            k_norm_rope_back<decltype(t), decltype(lpr)::value, decltype(il)::value, decltype(full)::value>
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
