// attend_join.cu -- joins the partial results of a request's chunks of keys:
// with m the largest of the chunks' maxima, l = sum l_c 2^(m_c - m) and
// o = sum o_c 2^(m_c - m) / l, in a fixed order.
#include "paged_attention.cuh"

namespace bevpool {

namespace {

// A CTA a query row: its warps take the chunks in turn, and the first joins the
// warps' sums.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
k_attend_join(AttnArgs a, AttnPlan pl) {
    constexpr int E = D / 32;
    __shared__ float sums[kWarps][D + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, hk = blockIdx.y, b = blockIdx.z;
    const Request r = request_of(a, b);
    int32_t base;
    const int n = chunks_of(a, r, pl.chunk, pl.n_chunks, pl.align, &base);
    const int rows = r.q_rows * a.G;
    if (n == 1 || static_cast<int>(blockIdx.x) >= rows) return;
    grid_dep_wait();
    for (int row = blockIdx.x; row < rows; row += gridDim.x) {
        const int64_t at = part_row(a, pl, b, hk, 0, row);
        float m = -INFINITY;
        for (int c = lane; c < n; c += 32) {
            const float2 ml = *reinterpret_cast<const float2 *>(a.part_ml + (at + static_cast<int64_t>(c) * pl.rows) * 2);
            m = fmaxf(m, ml.x);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float from = m == -INFINITY ? 0.0f : m;
        float l = 0.0f, acc[E] = {};
#pragma unroll 4
        for (int c = warp; c < n; c += kWarps) {
            const int64_t p = at + static_cast<int64_t>(c) * pl.rows;
            const float2 ml = *reinterpret_cast<const float2 *>(a.part_ml + p * 2);
            const float *o = a.part_o + p * D + lane * E;
            if (ml.y != 0.0f) {                            // else nothing was seen there, and no O written
                const float f = pow2(ml.x - from);
                l = fmaf(ml.y, f, l);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = fmaf(o[e], f, acc[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) sums[warp][lane * E + e] = acc[e];
        if (lane == 0) sums[warp][D] = l;
        __syncthreads();
        if (warp == 0) {
#pragma unroll
            for (int w = 1; w < kWarps; ++w) {
                l += sums[w][D];
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] += sums[w][lane * E + e];
            }
            l = __shfl_sync(0xffffffffu, l, 0);
            store_row<T, E>(a, pl, r, b, hk, row / a.G, hk * a.G + row % a.G, row, 0, 1, m, l, acc);
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_attend_join(const AttnArgs &a, const AttnPlan &pl) {
    auto run = [&](auto t, auto d) {
        int64_t gx = pl.rows;
        if (gx > 1024) gx = 1024;
        const cudaError_t e =
            launch_dependent(k_attend_join<decltype(t), decltype(d)::value>,
                             dim3(static_cast<unsigned>(gx), static_cast<unsigned>(a.Hk), static_cast<unsigned>(a.pg.n_seqs)),
                             dim3(kThreads), 0, a.stream, a, pl);
        if (e == cudaSuccess) count_launch();
        return e;
    };
    auto by_d = [&](auto t) {
        return a.D == 64 ? run(t, std::integral_constant<int, 64>{}) : run(t, std::integral_constant<int, 128>{});
    };
    return a.dtype == BEVPOOL_F16 ? by_d(__half{}) : by_d(__nv_bfloat16{});
}

}  // namespace bevpool
