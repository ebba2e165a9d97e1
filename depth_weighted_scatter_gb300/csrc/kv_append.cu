// kv_append.cu -- keys and values of new tokens into the paged cache, with
// the keys' norm and rotation (and the queries', optionally) on the way.
//
// Bound by memory: each row is read once and written once, straight to its
// slot.  The lane layout, the factors and the ring of rows read ahead are those
// of the norm and rotation kernel (rotary.cuh); a warp takes one token, or a
// slice of its rows when there are few tokens, and finds the token's request
// with one 32-wide search of cu_q.
//
// Measured on a GB300: 65536 tokens of 8 + 8 + 8 heads of 64, fp16 to E4M3: 65 us
// (3.8 TB/s of 6.7 measured copy; 71 % of the issue slots, as a token has but six
// steps to share its angles and its place; the frequencies' FP64 at the start of a
// CTA takes 2300 cycles an SM); 64 single tokens of 32 + 8 + 8 heads
// of 128, bf16: 8.2 us a call, bound by the launch.
#include "rotary.cuh"

namespace bevpool {

namespace {

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

// Where token t goes in the cache (elements), or -1: nowhere.
__device__ __forceinline__ int64_t slot_of(const PagedArgs &pg, int64_t t, int lane) {
    const int b = find_request(pg.cu_q, pg.n_seqs, static_cast<int32_t>(t), lane);
    if (b >= pg.n_seqs) return -1;
    const int64_t place = static_cast<int64_t>(pg.kv_len[b]) - pg.cu_q[b + 1] + t;
    if (place < 0 || (place >> pg.page_shift) >= pg.table_pages) return -1;
    const int32_t page = pg.block_table[static_cast<int64_t>(b) * pg.table_pages + (place >> pg.page_shift)];
    if (page < 0 || page >= pg.n_pages) return -1;
    return page * pg.page_stride + (place & (pg.page_size - 1)) * pg.slot_stride;
}

// x / scale of two values, rounded once but for 2^-46 of it.  (Times the rounded
// inverse an exact value halfway between two codes goes the wrong way for some
// scales: half of them for 63 / 4096.  The second product costs 65536 tokens of 24 heads
// of 64 1.4 us of 65.)
__device__ __forceinline__ uint64_t quotient(uint64_t x, const AppendArgs::Inverse &inv) {
    return fma2(x, pair(inv.hi, inv.hi), mul2(x, pair(inv.lo, inv.lo)));
}

constexpr int kAppendDepth = 8;                        // steps in flight a warp

template <typename T, int LPR, bool IL, bool FULL, bool E4M3>
__global__ void __launch_bounds__(kThreads, 3)
k_kv_append(AppendArgs g, int split) {
    using Stream = RowStream<LPR, 3, 1, kAppendDepth>;
    __shared__ __align__(16) RowWeights weights;
    __shared__ __align__(16) uint8_t ring[kWarps * Stream::BYTES];
    __shared__ typename Stream::Part parts[3];
    const NormRopeArgs &f = g.f;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rg = lane / LPR;
    weights.load(f.q_weight, f.k_weight, f.D);
    if (threadIdx.x == 0) {
        parts[0].set(0, f.q.p ? f.q : f.k);                // without queries: no steps, but an address
        parts[1].set(0, f.k);
        parts[2].set(0, g.v);
        parts[0].H = f.Hq, parts[0].end = steps_of<LPR>(f.Hq);
        parts[1].H = f.Hk, parts[1].end = parts[0].end + steps_of<LPR>(f.Hk);
        parts[2].H = f.Hk, parts[2].end = parts[1].end + steps_of<LPR>(f.Hk);
    }
    const LaneRow p = lane_row<IL>(f.rot, f.D, lane % LPR);
    LaneTurns<LPR> turns(f.rot, p, rg);
    __syncthreads();
    const Units units(f.T, split);
    if (units.first < units.n) turns.read(f.rot, units.token(units.first));
    Stream in(units, parts, static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + warp * Stream::BYTES, p, rg, f.D);
    const float inv_d = 1.0f / static_cast<float>(f.D);
    const int nq = parts[0].end, nk = parts[1].end, steps = parts[2].end;
    for (uint32_t u = units.first; u < units.n; u += units.stride) {
        const int64_t t = units.token(u);
        int s0, s1;
        units.steps(u, steps, &s0, &s1);
        const int64_t slot = s1 > nq ? slot_of(g.pg, t, lane) : -1;
        float cs[4], sn[4];
        turns.cos_sin(p, cs, sn);
        if (units.n - u > units.stride) turns.read(f.rot, units.token(u + units.stride));
#pragma unroll
        for (int part = 0; part < 3; ++part) {             // queries, keys, values
            const int begin = part == 0 ? 0 : part == 1 ? nq : nk;
            const int first = max(s0, begin), end = min(s1, part == 0 ? nq : part == 1 ? nk : steps);
            if (first >= end) continue;
            uint64_t fa[4], fb[4];
            if (part < 2) {
                float wu[4], wv[4];
                lane_weights(weights.w[part], p, wu, wv);
                lane_factors<IL>(cs, sn, wu, wv, fa, fb);
            }
            const bool norm = (part == 0 ? f.q_weight : f.k_weight) != nullptr;
            const int H = part == 0 ? f.Hq : f.Hk;
            const AppendArgs::Inverse &inv = part == 1 ? g.k_inv : g.v_inv;
            const int h = (first - begin) * Stream::RPS + rg;
            // steps in which this lane has a row to keep
            int rows_left = p.live && (part == 0 || slot >= 0) ? (H - h + Stream::RPS - 1) / Stream::RPS : 0;
            const int64_t stride = part == 0 ? f.q_out.head_stride : g.pg.head_stride, step = Stream::RPS * stride;
            int64_t at = (part == 0 ? t * f.q_out.token_stride : slot) + h * stride;
            void *dst = part == 0 ? f.q_out.p : part == 1 ? g.k_cache : g.v_cache;
            for (int s = first; s < end; ++s) {
                LaneWords x;
                in.next(&x);
                uint64_t y[4];
                if (part < 2) {
                    turn_row<T, LPR, IL, FULL>(x, p, fa, fb, norm, inv_d, f.eps, y);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = widen<T>(x.w[i]);
                }
                if (E4M3 && part > 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = quotient(y[i], inv);
                }
                if (rows_left-- > 0) {
                    if (E4M3 && part > 0)
                        store_lane_e4m3<IL>(static_cast<uint8_t *>(dst) + at, p, y);
                    else if (part == 2)
                        store_words<IL, T>(static_cast<T *>(dst) + at, p, x);
                    else
                        store_lane<IL, T>(static_cast<T *>(dst) + at, p, y);
                }
                at += step;
            }
        }
    }
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs &g) {
    const NormRopeArgs &f = g.f;
    auto run = [&](auto t, auto lpr, auto il, auto full, auto e4m3) {
        constexpr int LPR = decltype(lpr)::value;
        const int steps = steps_of<LPR>(f.Hq) + 2 * steps_of<LPR>(f.Hk);
        // Warps a token: as in the norm and rotation kernel.
        int64_t split = div_up(152 * 16, f.T);
        if (split > steps) split = steps;
        int64_t grid = div_up(static_cast<int64_t>(f.T) * split, kWarps);
        if (grid > 152 * 3) grid = 152 * 3;
        k_kv_append<decltype(t), LPR, decltype(il)::value, decltype(full)::value, decltype(e4m3)::value>
            <<<static_cast<int>(grid), kThreads, 0, f.stream>>>(g, static_cast<int>(split));
        count_launch();
        return cudaGetLastError();
    };
    auto by_e = [&](auto t, auto lpr, auto il, auto full) {
        return g.cache_e4m3 ? run(t, lpr, il, full, std::true_type{}) : run(t, lpr, il, full, std::false_type{});
    };
    auto by_full = [&](auto t, auto lpr, auto il) {
        return f.rot.rotary_dim == f.D ? by_e(t, lpr, il, std::true_type{}) : by_e(t, lpr, il, std::false_type{});
    };
    auto by_il = [&](auto t, auto lpr) {
        return f.rot.interleaved ? by_full(t, lpr, std::true_type{}) : by_full(t, lpr, std::false_type{});
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
