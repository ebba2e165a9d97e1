// kv_append_scaled.cu -- keys and values of new tokens into a paged E4M3 cache
// with a scale for each page and key head, worked out on the way: with top the
// largest finite magnitude that a page gets,
//     scale = top / 448                        (a page whose first token is new)
//     scale = old * 2^n, the least n >= 0 with top <= 448 * old * 2^n
//                                              (a page that holds earlier tokens)
// and the earlier tokens' codes times 2^-n.  The keys' norm and rotation (and the
// queries', optionally) are those of the norm and rotation kernel (rotary.cuh).
//
// A page's tokens are one group's: it reads a head's rows once, keeps what it
// stores of them in registers as FP32, finds the largest, and only then rounds.
// Powers of two move the earlier codes, so that they are rounded again only where
// they fall among E4M3's subnormal ones.
//
// Two layouts.  Pages with many new tokens: a group is a CTA, a thread has a lane's
// place in STEPS rows, whose angles it keeps for all of the part of the heads that
// the CTA takes.  Few tokens (a decoding step): a group is a warp, with one head of
// one page.  A page with more tokens than a group has rows is read twice.
#include "rotary.cuh"

namespace bevpool {

namespace {

constexpr float kLargest = 448.0f;
constexpr float kScaleLo = 0x1p-48f, kScaleHi = 0x1p48f;

// The request of token t: the last b in [0, n] with cu[b] <= t (n past the last
// one).  cu ascends from 0; 32 places are asked at a time.
__device__ __forceinline__ int request_of_token(const int32_t *cu, int n, int32_t t, int lane) {
    int lo = 0, hi = n + 1;                                // cu[lo] <= t; hi: the first known to be above, or n + 1
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, i = lo + (lane + 1) * step;
        const unsigned m = __ballot_sync(0xffffffffu, i < hi && cu[i] <= t);
        const int k = __popc(m);
        hi = min(hi, lo + (k + 1) * step);
        lo += k * step;
    }
    return lo;
}

// Tokens [t0, t1) of request b that go to the same page.
struct PageRun {
    int32_t b, t0, t1;
    int32_t page, slot;        // page < 0: nowhere; slot of t0
    bool held;                 // the page holds earlier tokens of the request
};

__device__ __forceinline__ PageRun page_run(const PagedArgs &pg, int b, int32_t c0, int32_t c1, int64_t start, int64_t page_i) {
    PageRun r;
    const int64_t p0 = page_i << pg.page_shift, place = max(p0, start);
    r.b = b;
    r.t0 = static_cast<int32_t>(c0 + place - start);
    r.t1 = static_cast<int32_t>(min(static_cast<int64_t>(c1), c0 + p0 + pg.page_size - start));
    r.slot = static_cast<int32_t>(place - p0);
    r.held = r.slot > 0;
    r.page = -1;
    if (b < pg.n_seqs && page_i >= 0 && page_i < pg.table_pages) {
        const int32_t p = pg.block_table[static_cast<int64_t>(b) * pg.table_pages + page_i];
        if (p >= 0 && p < pg.n_pages) r.page = p;
    }
    return r;
}

// Bounds of request b among T tokens; b = n_seqs: the tokens past the last request.
__device__ __forceinline__ void bounds_of(const PagedArgs &pg, int32_t T, int b, int32_t *c0, int32_t *c1, int64_t *start) {
    *c0 = min(max(pg.cu_q[b], 0), T);
    *c1 = b < pg.n_seqs ? min(max(pg.cu_q[b + 1], *c0), T) : T;
    *start = b < pg.n_seqs ? static_cast<int64_t>(pg.kv_len[b]) - (*c1 - *c0) : 0;
}

// CTAs for pages: request b has places for cu_q[b] / page_size + 2 b on, as many
// as its tokens can touch pages.
__device__ __forceinline__ int64_t first_place(const PagedArgs &pg, int32_t T, int b) {
    return (min(max(pg.cu_q[b], 0), T) >> pg.page_shift) + 2 * static_cast<int64_t>(b);
}

// 1 / s in two parts of one sign (the lower one is never zero: an infinite value
// times either has its sign).  s is in [2^-48, 2^48].
__device__ __forceinline__ AppendArgs::Inverse inverse_of(float s) {
    const float hi = __frcp_rz(s);
    return {hi, fmaxf(fmaf(-s, hi, 1.0f) * hi, hi * 0x1p-60f)};
}

__device__ __forceinline__ uint64_t quotient(uint64_t x, const AppendArgs::Inverse &inv) {
    return fma2(x, pair(inv.hi, inv.hi), mul2(x, pair(inv.lo, inv.lo)));
}

// A scale as it is used, whatever the array holds.
__device__ __forceinline__ float clamp_scale(float s) { return fminf(fmaxf(s, kScaleLo), kScaleHi); }

// The scale after new tokens of largest magnitude top (finite), and the power of
// two that the earlier codes are to be multiplied by.
__device__ __forceinline__ float new_scale(float top, bool held, float old, float *move) {
    *move = 1.0f;
    if (!held) return clamp_scale(__fdiv_rn(top, kLargest));
    const float was = clamp_scale(old), x = __fdiv_rn(top, kLargest * was);
    if (!(x > 1.0f)) return was;
    const uint32_t u = __float_as_uint(x);
    const int n = static_cast<int>(u >> 23) - 127 + ((u & 0x7fffff) != 0 ? 1 : 0);
    const float now = fminf(__uint_as_float(static_cast<uint32_t>(min(n, 127) + 127) << 23) * was, kScaleHi);
    *move = was / now;
    return now;
}

// 16 codes times a power of two (0 < move < 1).
__device__ __forceinline__ uint4 move_codes(uint4 w, float move) {
    const uint64_t m = pair(move, move);
    uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint64_t y[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>((u[i] >> (16 * j)) & 0xffff), __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            y[j] = mul2(pair(f.x, f.y), m);
        }
        u[i] = pack4_e4m3(y[0], y[1]);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

template <bool FINITE>
__device__ __forceinline__ float largest(float m, const uint64_t *y) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        unpair(y[i], &a, &b);
        a = fabsf(a), b = fabsf(b);
        if (FINITE) a = a < INFINITY ? a : 0.0f, b = b < INFINITY ? b : 0.0f;
        m = max3(m, a, b);                                 // NaN is passed over
    }
    return m;
}

struct TurnTable {             // of the pairs, in shared memory
    unsigned long long turns[kMaxHeadDim / 2];
    int32_t axis[kMaxHeadDim / 2];
};

// GROUP: warps of a group, all of the CTA's (pages) or one (tokens).
template <typename T, int LPR, bool IL, bool FULL, int GROUP, int STEPS>
__global__ void __launch_bounds__(kThreads, GROUP == 1 ? 4 : STEPS == 2 ? 3 : 2)
k_append_scaled(ScaledAppendArgs a, int parts) {
    constexpr bool PAGES = GROUP > 1;
    constexpr int RPS = 32 / LPR, ROWS = GROUP * RPS * STEPS, D = LPR * 8;
    __shared__ __align__(16) RowWeights weights;
    __shared__ TurnTable table;
    __shared__ uint32_t tops[2][kWarps];
    const NormRopeArgs &f = a.g.f;
    const PagedArgs &pg = a.g.pg;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rg = lane / LPR;
    const int jobs = f.Hq + 2 * f.Hk;

    // This group's tokens and heads: [job0, job1) of queries, keys, values.
    PageRun run = {0, 0, 0, -1, 0, false};
    int job0 = 0, job1 = 0;
    if constexpr (PAGES) {
        const int64_t place = blockIdx.x / parts;
        const int part = static_cast<int>(blockIdx.x % parts);
        int lo = 0, hi = pg.n_seqs + 1;                    // first_place(lo) <= place
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32, i = lo + (lane + 1) * step;
            const int k = __popc(__ballot_sync(0xffffffffu, i < hi && first_place(pg, f.T, i) <= place));
            hi = min(hi, lo + (k + 1) * step);
            lo += k * step;
        }
        int32_t c0, c1;
        int64_t start;
        bounds_of(pg, f.T, lo, &c0, &c1, &start);
        run = page_run(pg, lo, c0, c1, start, (start >> pg.page_shift) + place - first_place(pg, f.T, lo));
        if (run.t0 >= run.t1) return;                      // the same for the whole CTA
        job0 = part * jobs / parts;
        job1 = (part + 1) * jobs / parts;
    } else {
        const int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
        if (u < static_cast<int64_t>(f.T) * jobs) {
            const int32_t t = static_cast<int32_t>(u / jobs);
            const int b = request_of_token(pg.cu_q, pg.n_seqs, t, lane);
            int32_t c0, c1;
            int64_t start;
            bounds_of(pg, f.T, b, &c0, &c1, &start);
            const int64_t at = start + t - c0;
            // a page's first token takes the others along
            if (t >= c0 && t < c1 && (t == c0 || (at & (pg.page_size - 1)) == 0)) {
                run = page_run(pg, b, c0, c1, start, at >> pg.page_shift);
                job0 = static_cast<int>(u % jobs);
                job1 = job0 + 1;
            }
        }
    }
    weights.load(f.q_weight, f.k_weight, f.D);
    for (int i = threadIdx.x; i < f.rot.rotary_dim / 2; i += kThreads) {
        table.turns[i] = turn_of(f.rot.inv_freq[i]);
        table.axis[i] = pair_axis(f.rot, i);
    }
    const LaneRow p = lane_row<IL>(f.rot, D, lane % LPR);
    __syncthreads();
    if (run.t0 >= run.t1) return;
    const int n = run.t1 - run.t0, batches = (n + ROWS - 1) / ROWS;
    const int row0 = (PAGES ? warp * RPS : 0) + rg;        // this thread's first row; the others RPS * GROUP apart
    const float inv_d = 1.0f / static_cast<float>(D);

    // Angles of the rows of a batch.
    float cs[STEPS][4], sn[STEPS][4];
    const auto angles = [&](int batch) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int row = batch * ROWS + s * (GROUP * RPS) + row0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                cs[s][i] = 1.0f;
                sn[s][i] = 0.0f;
                if (p.turned && row < n) {
                    const int pr = p.c * 4 + i;
                    turn_cos_sin(table.turns[pr], f.rot.positions[static_cast<int64_t>(run.t0 + row) * f.rot.n_axes + table.axis[pr]], &cs[s][i],
                                 &sn[s][i]);
                }
            }
        }
    };
    LaneWords raw[STEPS];
    const auto read = [&](int job, int batch) {
        const bool q = job < f.Hq, k = !q && job < f.Hq + f.Hk;
        const HeadRows &src = q ? f.q : k ? f.k : a.g.v;
        const int h = q ? job : k ? job - f.Hq : job - f.Hq - f.Hk;
        const T *at = static_cast<const T *>(src.p) + h * src.head_stride;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int row = batch * ROWS + s * (GROUP * RPS) + row0;
            if (row < n) {
                const T *x = at + static_cast<int64_t>(run.t0 + row) * src.token_stride;
                if constexpr (IL) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(x + p.e0);
                    raw[s].w[0] = w.x, raw[s].w[1] = w.y, raw[s].w[2] = w.z, raw[s].w[3] = w.w;
                } else {
                    const uint2 w = *reinterpret_cast<const uint2 *>(x + p.e0), v = *reinterpret_cast<const uint2 *>(x + p.e1);
                    raw[s].w[0] = w.x, raw[s].w[1] = w.y, raw[s].w[2] = v.x, raw[s].w[3] = v.y;
                }
            } else {
                raw[s].w[0] = raw[s].w[1] = raw[s].w[2] = raw[s].w[3] = 0;
            }
        }
    };
    // The largest of a group's threads' magnitudes.
    int flip = 0;
    const auto over_group = [&](float m) {
        uint32_t u = __reduce_max_sync(0xffffffffu, __float_as_uint(m));   // not below 0: the order of the bits
        if constexpr (PAGES) {
            if (lane == 0) tops[flip][warp] = u;
            __syncthreads();
            u = tops[flip][0];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) u = max(u, tops[flip][w]);
            flip ^= 1;
        }
        return __uint_as_float(u);
    };

    angles(0);
    if (batches == 1) read(job0, 0);
    for (int job = job0; job < job1; ++job) {
        const bool is_q = job < f.Hq, is_k = !is_q && job < f.Hq + f.Hk;
        const int h = is_q ? job : is_k ? job - f.Hq : job - f.Hq - f.Hk;
        uint64_t y[STEPS][4];
        // The rows of a batch as they are stored, but for the scale.
        const auto work_out = [&]() {
            if (!is_q && !is_k) {
#pragma unroll
                for (int s = 0; s < STEPS; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[s][i] = widen<T>(raw[s].w[i]);
                return;
            }
            float wu[4], wv[4];
            lane_weights(weights.w[is_k], p, wu, wv);
            const bool norm = (is_q ? f.q_weight : f.k_weight) != nullptr;
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                uint64_t fa[4], fb[4];
                lane_factors<IL>(cs[s], sn[s], wu, wv, fa, fb);
                turn_row<T, LPR, IL, FULL>(raw[s], p, fa, fb, norm, inv_d, f.eps, y[s]);
            }
        };
        const auto store_q = [&](int batch) {
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int row = batch * ROWS + s * (GROUP * RPS) + row0;
                if (row < n)
                    store_lane<IL, T>(static_cast<T *>(f.q_out.p) + static_cast<int64_t>(run.t0 + row) * f.q_out.token_stride + h * f.q_out.head_stride, p, y[s]);
            }
        };
        // A pass over the batches for the largest (queries: all there is), one to store.
        const bool once = batches == 1;
        float top = 0.0f;
        bool again = false;                                // an infinity was met: the largest finite one is wanted
        AppendArgs::Inverse inv = {};
        const int64_t head = run.page * pg.page_stride + h * pg.head_stride;
        uint8_t *cache = static_cast<uint8_t *>(is_k ? a.g.k_cache : a.g.v_cache) + head;
        for (int pass = 0; pass < 2; ++pass) {
            for (int batch = 0; batch < batches; ++batch) {
                if (!once) {
                    if (is_q || is_k) angles(batch);
                    read(job, batch);
                }
                if (!once || (pass == 0 && !again)) work_out();
                if (once && pass == 0 && !again && job + 1 < job1) read(job + 1, 0);
                if (is_q) {
                    store_q(batch);
                } else if (pass == 0) {
#pragma unroll
                    for (int s = 0; s < STEPS; ++s) top = again ? largest<true>(top, y[s]) : largest<false>(top, y[s]);
                } else if (run.page >= 0) {
#pragma unroll
                    for (int s = 0; s < STEPS; ++s) {
                        const int row = batch * ROWS + s * (GROUP * RPS) + row0;
                        uint64_t z[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) z[i] = quotient(y[s][i], inv);
                        if (row < n) store_lane_e4m3<IL>(cache + (run.slot + row) * pg.slot_stride, p, z);
                    }
                }
            }
            if (is_q) break;
            if (pass == 0) {
                top = over_group(top);
                if (!again && top == INFINITY) {           // the same for the group
                    again = true;
                    top = 0.0f;
                    pass = -1;
                    continue;
                }
                if (run.page < 0) break;
                float *scale = (is_k ? a.k_scales : a.v_scales) + static_cast<int64_t>(run.page) * f.Hk + h;
                float move;
                const float old = run.held ? *scale : 0.0f;
                const float now = new_scale(top, run.held, old, &move);
                inv = inverse_of(now);
                if (run.held) {
                    if constexpr (PAGES) __syncthreads(); else __syncwarp();       // all have read the old one
                }
                if (PAGES ? threadIdx.x == 0 : lane == 0) *scale = now;
                if (move != 1.0f) {                        // the earlier tokens' codes
                    constexpr int CPR = D / 16;
                    for (int i = PAGES ? threadIdx.x : lane; i < run.slot * CPR; i += GROUP * 32) {
                        uint4 *c = reinterpret_cast<uint4 *>(cache + (i / CPR) * pg.slot_stride + (i % CPR) * 16);
                        *c = move_codes(*c, move);
                    }
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_append_scaled(const ScaledAppendArgs &a) {
    const NormRopeArgs &f = a.g.f;
    const int jobs = f.Hq + 2 * f.Hk;
    const auto run = [&](auto t, auto lpr, auto il, auto full, auto group, auto steps) {
        constexpr int LPR = decltype(lpr)::value, GROUP = decltype(group)::value, STEPS = decltype(steps)::value;
        int64_t grid, parts = 1;
        if constexpr (GROUP > 1) {
            const int64_t places = (f.T >> a.g.pg.page_shift) + 2 * (static_cast<int64_t>(a.g.pg.n_seqs) + 1);
            const int64_t pages = (f.T >> a.g.pg.page_shift) + a.g.pg.n_seqs;
            parts = div_up(152 * 8, pages);
            if (parts > jobs) parts = jobs;
            grid = places * parts;
        } else {
            grid = div_up(static_cast<int64_t>(f.T) * jobs, kWarps);
        }
        if (grid > INT32_MAX) return cudaErrorInvalidValue;
        k_append_scaled<decltype(t), LPR, decltype(il)::value, decltype(full)::value, GROUP, STEPS>
            <<<static_cast<unsigned>(grid), kThreads, 0, f.stream>>>(a, static_cast<int>(parts));
        count_launch();
        return cudaGetLastError();
    };
    using std::integral_constant;
    const auto by_group = [&](auto t, auto lpr, auto il, auto full) {
        if (f.T <= 4 * static_cast<int64_t>(a.g.pg.n_seqs)) return run(t, lpr, il, full, integral_constant<int, 1>{}, integral_constant<int, 1>{});
        return run(t, lpr, il, full, integral_constant<int, kWarps>{}, integral_constant<int, decltype(lpr)::value == 8 ? 2 : 4>{});
    };
    const auto by_full = [&](auto t, auto lpr, auto il) {
        return f.rot.rotary_dim == f.D ? by_group(t, lpr, il, std::true_type{}) : by_group(t, lpr, il, std::false_type{});
    };
    const auto by_il = [&](auto t, auto lpr) {
        return f.rot.interleaved ? by_full(t, lpr, std::true_type{}) : by_full(t, lpr, std::false_type{});
    };
    const auto by_lpr = [&](auto t) {
        return f.D == 64 ? by_il(t, integral_constant<int, 8>{}) : by_il(t, integral_constant<int, 16>{});
    };
    return f.dtype == BEVPOOL_F16 ? by_lpr(__half{}) : by_lpr(__nv_bfloat16{});
}

}  // namespace bevpool
