// attend_join.cu -- joins the partial results of a request's chunks of keys:
// with m the largest of the chunks' maxima, l = sum l_c 2^(m_c - m) and
// o = sum o_c 2^(m_c - m) / l, in a fixed order.
// Bound by the read of the partial results and, where they are few, by its latency:
// with one row of a warp at a time 3 x 700 tokens over 1500 keys took 24.7 us in
// all, with four 22.6.  (Where a request has few rows that leaves warps idle: 64
// single tokens 234 and 239 us.)
#include "paged_attention.cuh"

namespace bevpool {

namespace {

// W warps a query row: they take the parts in turn, and the first joins their
// sums.  A warp takes R rows at a time, their loads in flight together.  SHARED:
// rows are those of a tile pair that several CTAs shared.  Every CTA waits for the
// attention kernel, also one that has nothing to join: where no request has more
// than one chunk that kernel alone writes the results, and what comes next in the
// stream is ordered after this kernel.
template <typename T, int D, int W, int R, bool SHARED>
__global__ void __launch_bounds__(kThreads)
k_attend_join(AttnArgs a, AttnPlan pl) {
    constexpr int E = D / 32, ROWS = kWarps / W * R;       // rows of a CTA
    static_assert(W == 1 || R == 1, "rows of several warps are one at a time");
    struct alignas(E * 4) Elements {
        float x[E];
    };
    __shared__ float sums[W > 1 ? kWarps : 1][D + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % W;
    int hk = blockIdx.y, b = blockIdx.z, n, row_end, first_row = 0;
    // Part i of row x is at base + x + i * step, the first `extra` further on.
    int64_t base, step, extra = 0;
    Request r;
    if constexpr (SHARED) {
        hk = blockIdx.y / pl.tiles % a.Hk;
        b = blockIdx.y / pl.tiles / a.Hk;
        r = request_of(a, b);
        first_row = blockIdx.y % pl.tiles * kPairRows;
        row_end = min(r.q_rows * a.G, first_row + kPairRows);
        grid_dep_wait();
        if (first_row >= row_end) return;
        const int2 cut = a.cut[blockIdx.y];
        if (cut.x < 0) return;
        n = cut.y - cut.x + 1;
        base = static_cast<int64_t>(cut.x) * (2 * kPairRows) - first_row;
        step = 2 * kPairRows;
        extra = kPairRows;
    } else {
        r = request_of(a, b);
        int32_t key0;
        n = chunks_of(a, r, pl, &key0);
        row_end = r.q_rows * a.G;
        grid_dep_wait();
        if (n == 1 || static_cast<int>(blockIdx.x) * ROWS >= row_end) return;
        base = part_row(a, pl, b, hk, 0, 0);
        step = pl.rows;
    }
    for (int row0 = first_row + blockIdx.x * ROWS; row0 < row_end; row0 += gridDim.x * ROWS) {
        const int row = row0 + warp / W * R;
        float m[R], l[R] = {}, acc[R][E] = {};
        const auto at = [&](int x, int i) {                // a row past the last reads the last one's
            return base + min(row + x, row_end - 1) + i * step + (i == 0 ? extra : 0);
        };
#pragma unroll
        for (int x = 0; x < R; ++x) m[x] = lane < n ? a.part_ml[at(x, lane) * 2] : -INFINITY;
        for (int i = lane + 32; i < n; i += 32)
#pragma unroll
            for (int x = 0; x < R; ++x) m[x] = fmaxf(m[x], a.part_ml[at(x, i) * 2]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int x = 0; x < R; ++x) m[x] = fmaxf(m[x], __shfl_xor_sync(0xffffffffu, m[x], o));
#pragma unroll(R == 1 ? 4 : 2)
        for (int i = part; i < n; i += W) {
#pragma unroll
            for (int x = 0; x < R; ++x) {
                const int64_t p = at(x, i);
                const float2 ml = *reinterpret_cast<const float2 *>(a.part_ml + p * 2);
                const Elements o = *reinterpret_cast<const Elements *>(a.part_o + p * D + lane * E);
                // no sum: nothing was seen there, and no O written
                const float f = pow2(ml.x - (m[x] == -INFINITY ? 0.0f : m[x]));
                if (ml.y != 0.0f) l[x] = fmaf(ml.y, f, l[x]);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[x][e] = ml.y != 0.0f ? fmaf(o.x[e], f, acc[x][e]) : acc[x][e];
            }
        }
        if constexpr (W > 1) {
#pragma unroll
            for (int e = 0; e < E; ++e) sums[warp][lane * E + e] = acc[0][e];
            if (lane == 0) sums[warp][D] = l[0];
            __syncthreads();
            if (part == 0) {
#pragma unroll
                for (int w = 1; w < W; ++w) {
                    l[0] += sums[warp + w][D];
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[0][e] += sums[warp + w][lane * E + e];
                }
            }
        }
#pragma unroll
        for (int x = 0; x < R; ++x)
            if (row + x < row_end && part == 0)
                store_row<T, E>(a, r, (row + x) / a.G, hk * a.G + (row + x) % a.G, -1, m[x], l[x], acc[x]);
        if constexpr (W > 1) __syncthreads();
    }
}

}  // namespace

cudaError_t launch_attend_join(const AttnArgs &a, const AttnPlan &pl) {
    auto launch = [&](auto kernel, dim3 grid) {
        const cudaError_t e = launch_dependent(kernel, grid, dim3(kThreads), 0, a.stream, a, pl);
        if (e == cudaSuccess) count_launch();
        return e;
    };
    auto by_rows = [&](auto t, auto d, auto w, auto r) {
        constexpr int D = decltype(d)::value, W = decltype(w)::value, R = decltype(r)::value, ROWS = kWarps / W * R;
        if (pl.share)
            return launch(k_attend_join<decltype(t), D, W, R, true>,
                          dim3(kPairRows / ROWS, static_cast<unsigned>(pl.tiles * a.Hk * a.pg.n_seqs)));
        int64_t gx = div_up(pl.rows, ROWS);
        if (gx > 1024) gx = 1024;
        return launch(k_attend_join<decltype(t), D, W, R, false>,
                      dim3(static_cast<unsigned>(gx), static_cast<unsigned>(a.Hk), static_cast<unsigned>(a.pg.n_seqs)));
    };
    auto run = [&](auto t, auto d, auto w) {
        if constexpr (decltype(w)::value == 1)
            if (!pl.few) return by_rows(t, d, w, std::integral_constant<int, 4>{});
        return by_rows(t, d, w, std::integral_constant<int, 1>{});
    };
    // A warp a row where a row has few chunks (a CTA then takes eight rows), all
    // of a CTA's where it has many.  The whole call, with 76 chunks of 64 rows:
    // 137 us with a warp a row, 103 with eight; with 3 chunks of 40000 rows: 185
    // and 232.  Shared tiles have as many parts as CTAs share one, and one more.
    const int64_t n = !pl.share ? pl.n_chunks : pl.share / (static_cast<int64_t>(pl.tiles) * a.Hk * a.pg.n_seqs) + 2;
    auto by_w = [&](auto t, auto d) {
        if (n <= 4) return run(t, d, std::integral_constant<int, 1>{});
        if (n <= 16) return run(t, d, std::integral_constant<int, 4>{});
        return run(t, d, std::integral_constant<int, 8>{});
    };
    auto by_d = [&](auto t) {
        return a.D == 64 ? by_w(t, std::integral_constant<int, 64>{}) : by_w(t, std::integral_constant<int, 128>{});
    };
    return a.dtype == BEVPOOL_F16 ? by_d(__half{}) : by_d(__nv_bfloat16{});
}

}  // namespace bevpool
