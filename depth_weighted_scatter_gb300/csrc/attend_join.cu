// attend_join.cu -- joins the partial results of a request's chunks of keys:
// with m the largest of the chunks' maxima, l = sum l_c 2^(m_c - m) and
// o = sum o_c 2^(m_c - m) / l, in the order of the chunks.
#include "paged_attention.cuh"

namespace bevpool {

namespace {

// One warp a query row.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
k_attend_join(AttnArgs a, AttnPlan pl) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, hk = blockIdx.y, b = blockIdx.z;
    const Request r = request_of(a, b);
    int32_t base;
    const int n = chunks_of(a, r, pl.chunk, pl.n_chunks, pl.align, &base);
    if (n == 1) return;
    const int rows = r.q_rows * a.G;
    grid_dep_wait();
    for (int row = blockIdx.x * kWarps + (threadIdx.x >> 5); row < rows; row += gridDim.x * kWarps) {
        const int64_t at = part_row(a, pl, b, hk, 0, row);
        float m = -INFINITY;
        for (int c = lane; c < n; c += 32) m = fmaxf(m, a.part_ml[(at + static_cast<int64_t>(c) * pl.rows) * 2]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float from = m == -INFINITY ? 0.0f : m;
        float l = 0.0f, acc[E] = {};
#pragma unroll 4
        for (int c = 0; c < n; ++c) {
            const int64_t p = at + static_cast<int64_t>(c) * pl.rows;
            const float2 ml = *reinterpret_cast<const float2 *>(a.part_ml + p * 2);
            if (ml.y == 0.0f) continue;                    // nothing seen there, and no O written
            const float f = pow2(ml.x - from);
            l = fmaf(ml.y, f, l);
            const float *o = a.part_o + p * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(o[e], f, acc[e]);
        }
        store_row<T, E>(a, pl, r, b, hk, row / a.G, hk * a.G + row % a.G, row, 0, 1, m, l, acc);
    }
}

}  // namespace

cudaError_t launch_attend_join(const AttnArgs &a, const AttnPlan &pl) {
    auto run = [&](auto t, auto d) {
        int64_t gx = div_up(pl.rows, kWarps);
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
