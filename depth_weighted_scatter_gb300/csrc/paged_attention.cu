// paged_attention.cu -- attention of new tokens over the paged cache: the
// launch.
#include "paged_attention.cuh"

namespace bevpool {

namespace {

// One warp a token and query head.
template <typename T, bool E4M3, int D>
__global__ void __launch_bounds__(kThreads)
k_attend_rows(AttnArgs a) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int b = blockIdx.z;
    const Request r = request_of(a, b);
    const int64_t rows = static_cast<int64_t>(r.q_rows) * a.Hq;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < rows;
         u += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int32_t i = static_cast<int32_t>(u / a.Hq), h = static_cast<int32_t>(u % a.Hq);
        const int64_t t = r.q0 + i;
        float q[E], acc[E] = {}, m = -INFINITY, l = 0.0f;
        const T *qp = static_cast<const T *>(a.q.p) + t * a.q.token_stride + h * a.q.head_stride + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) q[e] = static_cast<float>(qp[e]);
        int32_t lo, hi;
        seen_keys(a, r, i, &lo, &hi);
        attend_row<T, E4M3, D>(a, b, h / a.G, q, lo, hi, &m, &l, acc);
        const float inv = l > 0.0f || l != l ? a.v_scale / l : 0.0f;
        T *op = static_cast<T *>(a.out.p) + t * a.out.token_stride + h * a.out.head_stride + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) op[e] = static_cast<T>(acc[e] * inv);
        if (a.lse && lane == 0) a.lse[t * a.Hq + h] = l > 0.0f || l != l ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
}

}  // namespace

size_t attention_workspace_bytes(int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t) { return 0; }

cudaError_t launch_paged_attention(const AttnArgs &a) {
    auto run = [&](auto t, auto e4m3, auto d) {
        int64_t gx = div_up(static_cast<int64_t>(a.max_q_len) * a.Hq, kWarps);
        if (gx > 65535) gx = 65535;
        k_attend_rows<decltype(t), decltype(e4m3)::value, decltype(d)::value>
            <<<dim3(static_cast<unsigned>(gx), 1, static_cast<unsigned>(a.pg.n_seqs)), kThreads, 0, a.stream>>>(a);
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
