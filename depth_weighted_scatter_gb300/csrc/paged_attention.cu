// paged_attention.cu -- attention of new tokens over the paged cache: how a
// call is laid out, and its launches.
#include "paged_attention.cuh"

namespace bevpool {

namespace {

// One warp a token and query head.
template <typename T, bool E4M3, int D>
__global__ void __launch_bounds__(kThreads)
k_attend_rows(AttnArgs a, AttnPlan pl) {
    constexpr int E = D / 32;
    const int b = blockIdx.z;
    const Request r = request_of(a, b);
    const int64_t rows = static_cast<int64_t>(r.q_rows) * a.Hq;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < rows;
         u += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int32_t i = static_cast<int32_t>(u / a.Hq), h = static_cast<int32_t>(u % a.Hq);
        float acc[E], m, l;
        redo_row<T, E4M3, D>(a, r, b, h / a.G, i, h, 0, r.kv_len, &m, &l, acc);
        store_row<T, E>(a, pl, r, b, h / a.G, i, h, 0, 0, 1, m, l, acc);
    }
}

// CTAs that a call's chunks make of its longest requests: about four for each
// of the two places of an SM, so that ragged lengths even out; the partial
// results stay below 1 % of the cache's bytes.
constexpr int64_t kFewCtas = 152 * 2 * 4;

}  // namespace

AttnPlan attention_plan(int32_t n_seqs, int32_t Hq, int32_t Hk, int32_t max_q_len, int32_t max_kv_len, int32_t window) {
    AttnPlan pl = {};
    pl.rows = max_q_len * (Hq / Hk);
    pl.few = pl.rows <= 16;
    pl.n_chunks = 1;
    pl.chunk = INT32_MAX / 2;
    if (!pl.few) return pl;
    // Keys from the first that a request's rows see, rounded down, to the last.
    int64_t keys = max_kv_len;
    if (window > 0 && static_cast<int64_t>(window) + max_q_len + kChunkAlign < keys)
        keys = static_cast<int64_t>(window) + max_q_len + kChunkAlign;
    if (keys < 1) keys = 1;
    const int64_t per = div_up(keys * n_seqs * Hk, kFewCtas);
    int64_t chunk = align_up(static_cast<size_t>(per), kChunkAlign);
    if (chunk > keys) chunk = align_up(static_cast<size_t>(keys), kChunkAlign);
    pl.chunk = static_cast<int32_t>(chunk);
    pl.n_chunks = static_cast<int32_t>(div_up(keys, chunk));
    return pl;
}

size_t attention_workspace_bytes(int32_t n_seqs, int32_t, int32_t Hq, int32_t Hk, int32_t D, int32_t max_q_len,
                                 int32_t max_kv_len) {
    // The most chunks of any window: a chunk holds kChunkAlign keys at least, and
    // keys * n_seqs * Hk / kFewCtas.
    const AttnPlan pl = attention_plan(n_seqs, Hq, Hk, max_q_len, max_kv_len, 0);
    if (!pl.few) return 0;
    const int64_t pairs = static_cast<int64_t>(n_seqs) * Hk;
    int64_t n = div_up(max_kv_len, kChunkAlign);
    if (n > div_up(kFewCtas, pairs)) n = div_up(kFewCtas, pairs);
    return n <= 1 ? 0 : static_cast<size_t>(pairs * n * pl.rows * (D + 2)) * sizeof(float);
}

cudaError_t launch_paged_attention(const AttnArgs &args, void *workspace) {
    AttnArgs a = args;
    const AttnPlan pl = attention_plan(a.pg.n_seqs, a.Hq, a.Hk, a.max_q_len, a.max_kv_len, a.window);
    if (pl.few) {
        a.part_o = static_cast<float *>(workspace);
        a.part_ml = a.part_o + static_cast<int64_t>(a.pg.n_seqs) * a.Hk * pl.n_chunks * pl.rows * a.D;
        const cudaError_t e = launch_attend_few(a, pl);
        if (e != cudaSuccess || pl.n_chunks == 1) return e;
        return launch_attend_join(a, pl);
    }
    auto run = [&](auto t, auto e4m3, auto d) {
        int64_t gx = div_up(static_cast<int64_t>(a.max_q_len) * a.Hq, kWarps);
        if (gx > 65535) gx = 65535;
        k_attend_rows<decltype(t), decltype(e4m3)::value, decltype(d)::value>
            <<<dim3(static_cast<unsigned>(gx), 1, static_cast<unsigned>(a.pg.n_seqs)), kThreads, 0, a.stream>>>(a, pl);
        count_launch();
        return cudaGetLastError();
    };
    auto by_d = [&](auto t, auto e4m3) {
        return a.D == 64 ? run(t, e4m3, std::integral_constant<int, 64>{})
                         : run(t, e4m3, std::integral_constant<int, 128>{});
    };
    auto by_e = [&](auto t) { return a.cache_e4m3 ? by_d(t, std::true_type{}) : by_d(t, std::false_type{}); };
    return a.dtype == BEVPOOL_F16 ? by_e(__half{}) : by_e(__nv_bfloat16{});
}

}  // namespace bevpool
