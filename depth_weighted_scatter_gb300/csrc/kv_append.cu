// kv_append.cu -- keys and values of new tokens into the paged cache, with
// the keys' norm and rotation (and the queries', optionally) on the way.
//
// Bound by memory: each row is read once and written once, straight to its
// slot.  The lane layout and the coefficients are those of the norm and
// rotation kernel (rotary.cuh); a warp takes one token, or a slice of its
// rows when there are few tokens, and finds the token's request with one
// 32-wide search of cu_q.
#include "rotary.cuh"

namespace bevpool {

namespace {

template <int LPR>
__host__ __device__ __forceinline__ int steps_of(int H) {
    return (H + 32 / LPR - 1) / (32 / LPR);
}

// The request of token t: the number of b in [1, n] with cu[b] <= t (n when t
// is past the last request).  cu ascends.
__device__ __forceinline__ int find_request(const int32_t *cu, int n, int32_t t, int lane) {
    int b = 0;
    for (int base = 1; base <= n; base += 32) {
        const int i = base + lane;
        const unsigned m = __ballot_sync(0xffffffffu, i <= n && cu[i] <= t);
        b += __popc(m);
        if (m != 0xffffffffu) break;
    }
    return b;
}

// Rows of one kind.  MODE 0: queries to q_out; 1: keys, 2: values to the cache
// (values are neither normed nor turned).
template <typename T, int LPR, bool IL, bool E4M3, int MODE>
__device__ __forceinline__ void append_rows(const AppendArgs &g, const HeadRows &in, int64_t t, int H, int s0, int s1,
                                            int c, int rg, bool live, int src, bool turned, const float *cs,
                                            const float *sn, const float *w, int cp, int64_t slot, float inv_scale) {
    constexpr int U = 4, RPS = 32 / LPR;
    const NormRopeArgs &f = g.f;
    float a[8], b[8];
    if (MODE != 2 && live) row_coefs(cs, sn, w, c, cp, IL, a, b);
    const T *ip = static_cast<const T *>(in.p) + t * in.token_stride + c * 8;
    const float inv_d = 1.0f / static_cast<float>(f.D);
    for (int s = s0; s < s1; s += U) {
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = (s + u) * RPS + rg;
            const bool on = live && s + u < s1 && h < H;
            x[u] = on ? *reinterpret_cast<const uint4 *>(ip + h * in.head_stride) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u >= s1) break;                        // the same for the whole warp
            const int h = (s + u) * RPS + rg;
            const bool on = live && h < H;
            if (MODE == 2 && !E4M3) {
                if (on) *reinterpret_cast<uint4 *>(static_cast<T *>(g.v_cache) + slot + h * g.pg.head_stride + c * 8) = x[u];
                continue;
            }
            float y[8];
            if constexpr (MODE == 2)
                unpack8<T>(x[u], y);
            else
                turn_row<T, LPR, IL>(x[u], src, turned, a, b, w != nullptr, inv_d, f.eps, y);
            if (MODE == 0) {
                if (on)
                    *reinterpret_cast<uint4 *>(static_cast<T *>(f.q_out.p) + t * f.q_out.token_stride +
                                               h * f.q_out.head_stride + c * 8) = pack8<T>(y);
            } else if (E4M3) {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] *= inv_scale;
                uint8_t *cache = static_cast<uint8_t *>(MODE == 1 ? g.k_cache : g.v_cache);
                if (on) *reinterpret_cast<uint2 *>(cache + slot + h * g.pg.head_stride + c * 8) = pack8_e4m3(y);
            } else {
                if (on)
                    *reinterpret_cast<uint4 *>(static_cast<T *>(g.k_cache) + slot + h * g.pg.head_stride + c * 8) =
                        pack8<T>(y);
            }
        }
    }
}

template <typename T, int LPR, bool IL, bool E4M3>
__global__ void __launch_bounds__(kThreads)
k_kv_append(AppendArgs g, int split) {
    __shared__ unsigned long long turns[kMaxHeadDim / 2];
    const NormRopeArgs &f = g.f;
    load_turns(f.rot, turns);
    __syncthreads();
    const int lane = threadIdx.x & 31, c = lane % LPR, rg = lane / LPR;
    const bool live = c * 8 < f.D;
    const int src = partner_lane<IL>(f.rot, c, lane), cp = c + src - lane;
    const bool turned = c * 8 < f.rot.rotary_dim;
    const int nq = f.q.p ? steps_of<LPR>(f.Hq) : 0, nk = steps_of<LPR>(f.Hk), n = nq + 2 * nk;
    const float k_inv = 1.0f / g.k_scale, v_inv = 1.0f / g.v_scale;
    const int64_t units = static_cast<int64_t>(f.T) * split;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units;
         u += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t t = u / split;
        const int part = static_cast<int>(u - t * split);
        const int s0 = part * n / split, s1 = (part + 1) * n / split;
        float cs[8], sn[8];
        if (s0 < nq + nk) lane_cos_sin<IL>(f.rot, turns, t, c, cs, sn);
        if (s0 < nq)
            append_rows<T, LPR, IL, E4M3, 0>(g, f.q, t, f.Hq, s0, min(s1, nq), c, rg, live, src, turned, cs, sn,
                                             f.q_weight, cp, 0, 1.0f);
        if (s1 <= nq) continue;
        const int b = find_request(g.pg.cu_q, g.pg.n_seqs, static_cast<int32_t>(t), lane);
        if (b >= g.pg.n_seqs) continue;
        const int64_t place = static_cast<int64_t>(g.pg.kv_len[b]) - g.pg.cu_q[b + 1] + t;
        if (place < 0 || (place >> g.pg.page_shift) >= g.pg.table_pages) continue;
        const int32_t page = g.pg.block_table[static_cast<int64_t>(b) * g.pg.table_pages + (place >> g.pg.page_shift)];
        if (page < 0 || page >= g.pg.n_pages) continue;
        const int64_t slot = page * g.pg.page_stride + (place & (g.pg.page_size - 1)) * g.pg.slot_stride;
        if (s0 < nq + nk)
            append_rows<T, LPR, IL, E4M3, 1>(g, f.k, t, f.Hk, max(s0 - nq, 0), min(s1 - nq, nk), c, rg, live, src, turned,
                                             cs, sn, f.k_weight, cp, slot, k_inv);
        if (s1 > nq + nk)
            append_rows<T, LPR, IL, E4M3, 2>(g, g.v, t, f.Hk, max(s0 - nq - nk, 0), s1 - nq - nk, c, rg, live, src,
                                             turned, cs, sn, nullptr, cp, slot, v_inv);
    }
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs &g) {
    const NormRopeArgs &f = g.f;
    auto run = [&](auto t, auto lpr, auto il, auto e4m3) {
        constexpr int LPR = decltype(lpr)::value;
        const int steps = (f.q.p ? steps_of<LPR>(f.Hq) : 0) + 2 * steps_of<LPR>(f.Hk);
        // Warps a token: as in the norm and rotation kernel.
        int64_t split = div_up(152 * 16, f.T);
        if (split > steps) split = steps;
        int64_t grid = div_up(static_cast<int64_t>(f.T) * split, kWarps);
        if (grid > 152 * 8) grid = 152 * 8;
        k_kv_append<decltype(t), LPR, decltype(il)::value, decltype(e4m3)::value>
            <<<static_cast<int>(grid), kThreads, 0, f.stream>>>(g, static_cast<int>(split));
        count_launch();
        return cudaGetLastError();
    };
    auto by_e = [&](auto t, auto lpr, auto il) {
        return g.cache_e4m3 ? run(t, lpr, il, std::true_type{}) : run(t, lpr, il, std::false_type{});
    };
    auto by_il = [&](auto t, auto lpr) {
        return f.rot.interleaved ? by_e(t, lpr, std::true_type{}) : by_e(t, lpr, std::false_type{});
    };
    auto by_lpr = [&](auto t) {
        if (f.D <= 32) return by_il(t, std::integral_constant<int, 4>{});
        if (f.D <= 64) return by_il(t, std::integral_constant<int, 8>{});
        if (f.D <= 128) return by_il(t, std::integral_constant<int, 16>{});
        return by_il(t, std::integral_constant<int, 32>{});
    };
    return f.dtype == BEVPOOL_F16 ? by_lpr(__half{}) : by_lpr(__nv_bfloat16{});
}

}  // namespace bevpool
