// attend_join.cu -- joins the partial results of a request's chunks of keys:
// with m the largest of the chunks' maxima, l = sum l_c 2^(m_c - m) and
// o = sum o_c 2^(m_c - m) / l, in a fixed order.
// Bound by the read of the partial results.  Measured: 67000 rows of 128 with two
// chunks 36 us (2.9 TB/s).
#include "paged_attention.cuh"

namespace bevpool {

namespace {

// W warps a query row: they take the chunks in turn, and the first joins their
// sums.
template <typename T, int D, int W>
__global__ void __launch_bounds__(kThreads)
k_attend_join(AttnArgs a, AttnPlan pl) {
    constexpr int E = D / 32, ROWS = kWarps / W;           // rows of a CTA
    __shared__ float sums[W > 1 ? kWarps : 1][D + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % W, hk = blockIdx.y, b = blockIdx.z;
    const Request r = request_of(a, b);
    int32_t base;
    const int n = chunks_of(a, r, pl.chunk, pl.n_chunks, pl.align, &base);
    const int rows = r.q_rows * a.G;
    if (n == 1 || static_cast<int>(blockIdx.x) * ROWS >= rows) return;
    grid_dep_wait();
    for (int row0 = blockIdx.x * ROWS; row0 < rows; row0 += gridDim.x * ROWS) {
        const int row = row0 + warp / W;
        float m = -INFINITY, l = 0.0f, acc[E] = {};
        if (row < rows) {
            const int64_t at = part_row(a, pl, b, hk, 0, row);
            for (int c = lane; c < n; c += 32) m = fmaxf(m, a.part_ml[(at + static_cast<int64_t>(c) * pl.rows) * 2]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float from = m == -INFINITY ? 0.0f : m;
#pragma unroll 4
            for (int c = part; c < n; c += W) {
                const int64_t p = at + static_cast<int64_t>(c) * pl.rows;
                const float2 ml = *reinterpret_cast<const float2 *>(a.part_ml + p * 2);
                if (ml.y != 0.0f) {                        // else nothing was seen there, and no O written
                    const float *o = a.part_o + p * D + lane * E;
                    const float f = pow2(ml.x - from);
                    l = fmaf(ml.y, f, l);
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] = fmaf(o[e], f, acc[e]);
                }
            }
        }
        if constexpr (W > 1) {
#pragma unroll
            for (int e = 0; e < E; ++e) sums[warp][lane * E + e] = acc[e];
            if (lane == 0) sums[warp][D] = l;
            __syncthreads();
            if (part == 0) {
#pragma unroll
                for (int w = 1; w < W; ++w) {
                    l += sums[warp + w][D];
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] += sums[warp + w][lane * E + e];
                }
            }
        }
        if (row < rows && part == 0)
            store_row<T, E>(a, pl, r, b, hk, row / a.G, hk * a.G + row % a.G, row, 0, 1, m, l, acc);
        if constexpr (W > 1) __syncthreads();
    }
}

}  // namespace

cudaError_t launch_attend_join(const AttnArgs &a, const AttnPlan &pl) {
    auto run = [&](auto t, auto d, auto w) {
        int64_t gx = div_up(pl.rows, kWarps / decltype(w)::value);
        if (gx > 1024) gx = 1024;
        const cudaError_t e =
            launch_dependent(k_attend_join<decltype(t), decltype(d)::value, decltype(w)::value>,
                             dim3(static_cast<unsigned>(gx), static_cast<unsigned>(a.Hk), static_cast<unsigned>(a.pg.n_seqs)),
                             dim3(kThreads), 0, a.stream, a, pl);
        if (e == cudaSuccess) count_launch();
        return e;
    };
    // A warp a row where a row has few chunks (a CTA then takes eight rows), all
    // of a CTA's where it has many.  The whole call, with 76 chunks of 64 rows:
    // 137 us with a warp a row, 103 with eight; with 3 chunks of 40000 rows: 185
    // and 232.
    auto by_w = [&](auto t, auto d) {
        if (pl.n_chunks <= 4) return run(t, d, std::integral_constant<int, 1>{});
        if (pl.n_chunks <= 16) return run(t, d, std::integral_constant<int, 4>{});
        return run(t, d, std::integral_constant<int, 8>{});
    };
    auto by_d = [&](auto t) {
        return a.D == 64 ? by_w(t, std::integral_constant<int, 64>{}) : by_w(t, std::integral_constant<int, 128>{});
    };
    return a.dtype == BEVPOOL_F16 ? by_d(__half{}) : by_d(__nv_bfloat16{});
}

}  // namespace bevpool
