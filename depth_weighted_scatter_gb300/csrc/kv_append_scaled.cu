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
// Two layouts.  Pages with many new tokens: a group is as many warps as a page's
// rows fill (2, 4 or 8), a thread has a lane's place in STEPS rows, whose angles it
// keeps for all of the heads that its group takes.  Few tokens (a decoding step): a
// group is a warp, with one head of one page.  A page with more tokens than a group
// has rows is read twice, its angles kept in shared memory.
//
// Measured on a GB300: 65536 tokens of 8 + 8 + 8 heads of 64, fp16, pages of 64: 63 us
// (4.0 TB/s of 6.8 measured copy; with one scale for the cache 65); six chunks of up to
// 1501 tokens of 32 + 8 + 8 heads of 128, bf16: 46 us, 104 pages being too few CTAs to
// cover what a head's rows wait for (a sum over lanes, a largest over warps) with each
// other; 64 single tokens: 6.2 us a call, the launch and its call. The rows through
// registers a head ahead instead of asynchronous copies: 74 and 51 us; sincospif for
// the angles and factors anew for each head: 112 and 78.  Pages of 128 and 256, which are
// read twice: the chunks 86 and 147 us (heads' split pairs, positions of one axis; 43 with
// pages of 64), the frames 122 and 129 (69).
//
#include <algorithm>

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
// times either has its sign).  s is in [2^-48, 2^48].  One Newton step leaves the
// approximate reciprocal within a unit in the last place of 1 / s, two units below
// that it is less than 1 / s, and what is left is a positive number.
__device__ __forceinline__ AppendArgs::Inverse inverse_of(float s) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    r = fmaf(fmaf(-s, r, 1.0f), r, r);
    const float hi = __uint_as_float(__float_as_uint(r) - 2);
    return {hi, fmaf(-s, hi, 1.0f) * hi};
}

// top / 448, rounded to nearest: the remainder of the rounded product corrects it
// (top is at least 448 * 2^-48 where that counts, so nothing is subnormal).
__device__ __forceinline__ float over_largest(float top) {
    constexpr float inv = 1.0f / kLargest;
    const float q = top * inv;
    return fmaf(fmaf(-kLargest, q, top), inv, q);
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
    if (!held) return clamp_scale(over_largest(top));
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

// CTAs a page: its heads are shared out so that the waves of CTAs (slots: what the
// GPU holds at a time) take least, a CTA costing what its heads' rows cost and about
// kSetUp heads besides (its request, its rows' angles).  Measured with 1 / 2 / 3 / 4 / 5
// parts, nothing in L2: 1024 pages of 64 slots and 24 heads of 64 76 / 76 / 79 / 83 / 89
// us, 104 of 48 heads of 128 60 / 48 / 56 / 50 / 48; the same tokens over pages of 128
// slots 128 / 132 / 152 / 140 / 146 and 232 / 140 / 124 / 95 / 89, of 256 203 / 133 / 181 /
// 152 / 158 and 443 / 263 / 199 / 148 / 181.  Taken: 1, 2; 1, 5; 2, 4.
int64_t append_parts(int64_t pages, int jobs, int groups, int64_t slots) {
    constexpr int64_t kSetUp = 4, kMost = 4096;
    int64_t best = 1, least = INT64_MAX;
    for (int64_t parts = 1; parts <= jobs && parts <= kMost; ++parts) {
        const int64_t cost = div_up(pages * parts, slots) * (div_up(jobs, parts * groups) + kSetUp);
        if (cost < least) {
            least = cost;
            best = parts;
        }
    }
    return best;
}

struct TurnTable {             // of the pairs, in shared memory
    unsigned long long turns[128 / 2];
    int32_t axis[128 / 2];
};

// cos and sin of position * inv_freq, off by 2^-20 at most: the angle, reduced exactly
// (rotary.cuh), goes to the hardware's functions.  They are off by up to 2^-21.19 in
// [-pi, pi]; the angle by 2^-23.3 (64 of 2^31 half turns, of its conversion), 2^-23 (its
// product) and 2^-23.5 (its factor).  (sincospif's last four bits cost as much as ten
// heads' rows where a group has few heads.)
__device__ __forceinline__ float2 cos_sin_fast(unsigned long long turns, int32_t pos) {
    const uint32_t top = static_cast<uint32_t>((turns * static_cast<unsigned long long>(static_cast<long long>(pos))) >> 32);
    const float angle = static_cast<float>(static_cast<int32_t>(top)) * 1.4629180792671596e-9f;      // pi 2^-31
    return make_float2(__cosf(angle), __sinf(angle));
}

// A row's cos and sin of a lane's four pairs, and the row turned by them.
template <bool IL>
struct RowTurn {
    uint64_t c[2], s[2];                                   // pairs 0 1 and 2 3
    __device__ __forceinline__ void set(const float2 *cs) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            c[i] = pair(cs[2 * i].x, cs[2 * i + 1].x);
            s[i] = pair(cs[2 * i].y, cs[2 * i + 1].y);
        }
    }
    __device__ __forceinline__ void turn(uint64_t *y) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (IL) {                            // words 2i, 2i + 1 hold a pair each
                float cc[2], ss[2];
                unpair(c[i], &cc[0], &cc[1]);
                unpair(s[i], &ss[0], &ss[1]);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float a, b;
                    unpair(y[2 * i + k], &a, &b);
                    y[2 * i + k] = pair(fmaf(a, cc[k], -(b * ss[k])), fmaf(b, cc[k], a * ss[k]));
                }
            } else {                                       // word i holds the first elements, word i + 2 the second
                const uint64_t u = y[i], v = y[i + 2];
                float u0, u1, c0, c1, t0, t1;
                unpair(u, &u0, &u1);
                unpair(c[i], &c0, &c1);
                unpair(mul2(v, s[i]), &t0, &t1);
                y[i] = pair(fmaf(u0, c0, -t0), fmaf(u1, c1, -t1));
                y[i + 2] = fma2(v, c[i], mul2(u, s[i]));
            }
        }
    }
};

// Shared memory of an SM, and what a CTA takes of it besides the dynamic part (its
// weights, its pairs, 1 KB of the system's).
constexpr int kSmShared = 228 * 1024, kFixedShared = 4 * 1024;

// Heads whose rows are on their way: 32 KB a CTA where an SM holds three, 48 KB where
// it holds two (one head more or less: 63 to 64 us and 47 to 56 of the cases below).
constexpr int append_ahead(int steps) { return steps == 2 ? 4 : 3; }

// Groups of one warp (tokens), or of `group_warps` (pages).
template <typename T, int LPR, bool IL, bool PAGES, int STEPS>
__global__ void __launch_bounds__(kThreads, PAGES ? (STEPS == 2 ? 3 : 2) : 3)
k_append_scaled(ScaledAppendArgs a, int parts, int group_warps) {
    constexpr int RPS = 32 / LPR, D = LPR * 8, AHEAD = append_ahead(STEPS);
    __shared__ __align__(16) RowWeights weights;
    __shared__ TurnTable table;
    __shared__ uint32_t tops[PAGES ? kWarps : 1][3];
    extern __shared__ __align__(16) uint8_t dynamic[];     // pages: rows on their way; of several batches, their angles instead
    float2 *angles = reinterpret_cast<float2 *>(dynamic);  // [row][pair]
    const NormRopeArgs &f = a.g.f;
    const PagedArgs &pg = a.g.pg;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rg = lane / LPR;
    const int jobs = f.Hq + 2 * f.Hk;
    const int apart = PAGES ? group_warps * RPS : RPS, rows = apart * STEPS;       // rows between a thread's, and of a group
    const int group = PAGES ? warp / group_warps : warp, group_warp = PAGES ? warp % group_warps : 0;

    // This group's tokens and heads: [job0, job1) of queries, keys, values.
    PageRun run = {0, 0, 0, -1, 0, false};
    int job0 = 0, job1 = 0;
    if constexpr (PAGES) {
        const int64_t place = blockIdx.x / parts;
        const int groups = kWarps / group_warps, part = static_cast<int>(blockIdx.x % parts) * groups + group;
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
        job0 = static_cast<int>(static_cast<int64_t>(part) * jobs / (parts * groups));
        job1 = static_cast<int>((static_cast<int64_t>(part) + 1) * jobs / (parts * groups));
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
    const int n = run.t1 - run.t0, batches = (n + rows - 1) / rows;
    const int pairs = f.rot.rotary_dim / 2;
    weights.load(f.q_weight, f.k_weight, f.D);
    for (int i = threadIdx.x; i < pairs; i += kThreads) {
        table.turns[i] = turn_of(f.rot.inv_freq[i]);
        table.axis[i] = pair_axis(f.rot, i);
    }
    if (PAGES && threadIdx.x < kWarps * 3) tops[threadIdx.x / 3][threadIdx.x % 3] = 0;
    const LaneRow p = lane_row<IL>(f.rot, D, lane % LPR);
    __syncthreads();
    if (PAGES && batches > 1) {                            // the same for the whole CTA
        for (int i = threadIdx.x; i < n * pairs; i += kThreads) {
            const int row = i / pairs, pr = i - row * pairs;
            angles[i] = cos_sin_fast(table.turns[pr], f.rot.positions[static_cast<int64_t>(run.t0 + row) * f.rot.n_axes + table.axis[pr]]);
        }
        __syncthreads();
    }
    if (job0 >= job1) return;
    const int row0 = group_warp * RPS + rg;                // this thread's first row
    const float inv_d = 1.0f / static_cast<float>(D);
    const auto sync_group = [&]() {
        if constexpr (!PAGES)
            __syncwarp();
        else if (group_warps == kWarps)
            __syncthreads();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(group_warps * 32) : "memory");
    };

    RowTurn<IL> turns[STEPS];
    const auto set_turns = [&](int batch) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int row = batch * rows + s * apart + row0;
            float2 cs[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                cs[i] = make_float2(1.0f, 0.0f);
                if (p.turned && row < n) {
                    const int pr = p.c * 4 + i;
                    cs[i] = PAGES && batches > 1
                                ? angles[row * pairs + pr]
                                : cos_sin_fast(table.turns[pr], f.rot.positions[static_cast<int64_t>(run.t0 + row) * f.rot.n_axes + table.axis[pr]]);
                }
            }
            turns[s].set(cs);
        }
    };
    int turn_slot = 0;                                     // of tops
    // The largest magnitude of a group's rows.
    const auto over_group = [&](float m) {
        uint32_t u = __reduce_max_sync(0xffffffffu, __float_as_uint(m));   // not below 0: the order of the bits
        if constexpr (PAGES) {
            uint32_t *top = tops[group];
            if (lane == 0) atomicMax(&top[turn_slot], u);
            sync_group();
            u = top[turn_slot];
            // the place before this one was read before the barrier, and is written again after the next
            const int before = turn_slot == 0 ? 2 : turn_slot - 1;
            if (group_warp == 0 && lane == 0) top[before] = 0;
            turn_slot = turn_slot == 2 ? 0 : turn_slot + 1;
        }
        return __uint_as_float(u);
    };

    // One of the three tensors: PART 0 queries, 1 keys, 2 values; its heads [h0, h1).
    const auto part_of = [&](auto part_c, int h0, int h1) {
        constexpr int PART = decltype(part_c)::value;
        if (h0 >= h1 || (PART > 0 && run.page < 0)) return;
        const HeadRows &src = PART == 0 ? f.q : PART == 1 ? f.k : a.g.v;
        const int64_t head_bytes = src.head_stride * 2, step_bytes = static_cast<int64_t>(apart) * src.token_stride * 2;
        const char *from = static_cast<const char *>(src.p) + (static_cast<int64_t>(run.t0 + row0) * src.token_stride + h0 * src.head_stride) * 2;
        const float *weight = PART == 0 ? f.q_weight : f.k_weight;
        uint64_t w[4];
        if constexpr (PART < 2) {
            float u[4], v[4];
            lane_weights(weights.w[PART], p, u, v);
            w[0] = pair(u[0], u[1]), w[1] = pair(u[2], u[3]), w[2] = pair(v[0], v[1]), w[3] = pair(v[2], v[3]);
        }
        // where this thread's first row goes
        const int64_t to_step = static_cast<int64_t>(apart) * (PART == 0 ? f.q_out.token_stride * 2 : pg.slot_stride);
        const int64_t to_head = PART == 0 ? f.q_out.head_stride * 2 : pg.head_stride;
        char *to = PART == 0 ? static_cast<char *>(f.q_out.p) + static_cast<int64_t>(run.t0 + row0) * f.q_out.token_stride * 2
                             : static_cast<char *>(PART == 1 ? a.g.k_cache : a.g.v_cache) + run.page * pg.page_stride +
                                   (run.slot + row0) * pg.slot_stride;
        to += h0 * to_head;
        float *scales = PART == 0 ? nullptr : (PART == 1 ? a.k_scales : a.v_scales) + static_cast<int64_t>(run.page) * f.Hk;
        LaneWords raw[STEPS];
        const auto read = [&](const char *x, int first) {
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                if (first + s * apart < n) {
                    const T *row = reinterpret_cast<const T *>(x + s * step_bytes);
                    if constexpr (IL) {
                        const uint4 q = *reinterpret_cast<const uint4 *>(row + p.e0);
                        raw[s].w[0] = q.x, raw[s].w[1] = q.y, raw[s].w[2] = q.z, raw[s].w[3] = q.w;
                    } else {
                        const uint2 q = *reinterpret_cast<const uint2 *>(row + p.e0), v = *reinterpret_cast<const uint2 *>(row + p.e1);
                        raw[s].w[0] = q.x, raw[s].w[1] = q.y, raw[s].w[2] = v.x, raw[s].w[3] = v.y;
                    }
                } else {
                    raw[s].w[0] = raw[s].w[1] = raw[s].w[2] = raw[s].w[3] = 0;
                }
            }
        };
        uint64_t y[STEPS][4];
        // The rows read, as they are stored but for the scale.
        const auto work_out = [&]() {
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
#pragma unroll
                for (int i = 0; i < 4; ++i) y[s][i] = widen<T>(raw[s].w[i]);
                if constexpr (PART < 2) {
                    float r = 1.0f;
                    if (weight) r = rsqrtf(fmaf(row_sum<LPR>(lane_dot(y[s], y[s])), inv_d, f.eps));
                    if (weight) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) y[s][i] = mul2(mul2(y[s][i], pair(r, r)), w[i]);
                    }
                    if (p.turned) turns[s].turn(y[s]);
                }
            }
        };
        // Once a head's largest is known: its scale, the earlier tokens' codes; what the
        // new ones are divided by.
        const auto settle = [&](int h, float top, float old) {
            float move;
            const float now = new_scale(top, run.held, old, &move);
            if (group_warp == 0 && lane == 0) scales[h] = now;             // after all have read the old one
            if (run.held && move != 1.0f) {
                constexpr int CPR = D / 16;
                uint8_t *page = static_cast<uint8_t *>(PART == 1 ? a.g.k_cache : a.g.v_cache) + run.page * pg.page_stride + h * pg.head_stride;
                for (int i = group_warp * 32 + lane; i < run.slot * CPR; i += (PAGES ? group_warps : 1) * 32) {
                    uint4 *c = reinterpret_cast<uint4 *>(page + (i / CPR) * pg.slot_stride + (i % CPR) * 16);
                    *c = move_codes(*c, move);
                }
            }
            return inverse_of(now);
        };
        const auto store = [&](int batch, const AppendArgs::Inverse &inv) {
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                if (batch * rows + s * apart + row0 >= n) continue;
                char *x = to + (batch * STEPS + s) * to_step;
                if constexpr (PART == 0) {
                    store_lane<IL, T>(reinterpret_cast<T *>(x), p, y[s]);
                } else {
                    uint64_t z[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) z[i] = quotient(y[s][i], inv);
                    store_lane_e4m3<IL>(reinterpret_cast<uint8_t *>(x), p, z);
                }
            }
        };
        if (batches == 1) {
            // Pages: a thread's own pieces of the next heads' rows come by asynchronous
            // copies to its own place.
            const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(dynamic)) + threadIdx.x * 16;
            const auto fetch = [&](int h, int slot) {
                if (h < h1) {
#pragma unroll
                    for (int s = 0; s < STEPS; ++s) {
                        const bool on = row0 + s * apart < n;              // else zeros
                        const T *row = reinterpret_cast<const T *>(on ? from + (h - h0) * head_bytes + s * step_bytes : from);
                        const uint32_t d = ring + (slot * STEPS + s) * (kThreads * 16);
                        if constexpr (IL) {
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(row + p.e0), "r"(on ? 16 : 0) : "memory");
                        } else {
                            asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(d), "l"(row + p.e0), "r"(on ? 8 : 0) : "memory");
                            asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(d + 8), "l"(row + p.e1), "r"(on ? 8 : 0) : "memory");
                        }
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            [[maybe_unused]] int slot = 0;
            if constexpr (PAGES) {
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) fetch(h0 + i, i);
            } else {
                read(from, row0);
            }
            float old_next = PART > 0 && run.held ? scales[h0] : 0.0f;
#pragma unroll 1
            for (int h = h0; h < h1; ++h, to += to_head) {
                const float old = old_next;
                if constexpr (PAGES) {
                    asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
#pragma unroll
                    for (int s = 0; s < STEPS; ++s)
                        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                     : "=r"(raw[s].w[0]), "=r"(raw[s].w[1]), "=r"(raw[s].w[2]), "=r"(raw[s].w[3])
                                     : "r"(ring + (slot * STEPS + s) * (kThreads * 16))
                                     : "memory");
                }
                work_out();
                if constexpr (PAGES) {
                    fetch(h + AHEAD, slot);
                    slot = slot == AHEAD - 1 ? 0 : slot + 1;
                }
                if (PART > 0 && run.held && h + 1 < h1) old_next = scales[h + 1];
                if constexpr (PART == 0) {
                    store(0, {});
                } else {
                    float top = 0.0f;
#pragma unroll
                    for (int s = 0; s < STEPS; ++s) top = largest<false>(top, y[s]);
                    top = over_group(top);
                    if (top == INFINITY) {                 // the same for the group: the largest finite one
                        top = 0.0f;
#pragma unroll
                        for (int s = 0; s < STEPS; ++s) top = largest<true>(top, y[s]);
                        top = over_group(top);
                    }
                    store(0, settle(h, top, old));
                }
            }
            return;
        }
        // A pass over the batches for the largest (queries: all there is; once more where
        // an infinity was met), one to store.
#pragma unroll 1
        for (int h = h0; h < h1; ++h, from += head_bytes, to += to_head) {
            const float old = PART > 0 && run.held ? scales[h] : 0.0f;
            float top = 0.0f;
            AppendArgs::Inverse inv = {};
            int pass = 0;                                  // 0: the largest, 1: the largest finite one, 2: store
            do {
                top = 0.0f;
#pragma unroll 1
                for (int batch = 0; batch < batches; ++batch) {
                    if (PART < 2) set_turns(batch);
                    read(from + batch * STEPS * step_bytes, batch * rows + row0);
                    work_out();
                    if (PART == 0 || pass == 2) {
                        store(batch, inv);
                    } else {
#pragma unroll
                        for (int s = 0; s < STEPS; ++s) top = pass == 1 ? largest<true>(top, y[s]) : largest<false>(top, y[s]);
                    }
                }
                if (PART == 0 || pass == 2) break;
                top = over_group(top);
                if (pass == 0 && top == INFINITY) {
                    pass = 1;
                } else {
                    inv = settle(h, top, old);
                    pass = 2;
                }
            } while (true);
        }
    };
    const int q1 = f.Hq, k1 = q1 + f.Hk;
    if (batches == 1 && job0 < k1) set_turns(0);
    part_of(std::integral_constant<int, 0>{}, job0, min(job1, q1));
    part_of(std::integral_constant<int, 1>{}, max(job0, q1) - q1, min(job1, k1) - q1);
    part_of(std::integral_constant<int, 2>{}, max(job0, k1) - k1, job1 - k1);
}

}  // namespace

cudaError_t launch_append_scaled(const ScaledAppendArgs &a) {
    const NormRopeArgs &f = a.g.f;
    const PagedArgs &pg = a.g.pg;
    const int jobs = f.Hq + 2 * f.Hk;
    using std::integral_constant;
    const auto run = [&](auto t, auto lpr, auto il, auto pages_c) {
        constexpr int LPR = decltype(lpr)::value, STEPS = !decltype(pages_c)::value ? 1 : LPR == 8 ? 2 : 4;
        constexpr bool IL = decltype(il)::value, PAGES = decltype(pages_c)::value;
        int64_t grid, parts = 1;
        int group_warps = 1, smem = 0;
        if constexpr (PAGES) {
            group_warps = pg.page_size >= 64 ? 8 : pg.page_size / 8;       // 64 rows at most
            const int groups = kWarps / group_warps;
            const int64_t full = f.T >> pg.page_shift, places = full + 2 * (static_cast<int64_t>(pg.n_seqs) + 1), pages = full + pg.n_seqs;
            // a CTA has the rows on their way or its angles in shared memory, never both
            constexpr int ring = append_ahead(STEPS) * STEPS * kThreads * 16, most = 256 * (LPR * 4) * static_cast<int>(sizeof(float2));
            smem = ring;
            if (pg.page_size > 64) smem = std::max(smem, pg.page_size * (f.rot.rotary_dim / 2) * static_cast<int>(sizeof(float2)));
            const int held = std::min(STEPS == 2 ? 3 : 2, kSmShared / (smem + kFixedShared));      // CTAs of an SM
            parts = append_parts(pages, jobs, groups, 152 * held);
            grid = places * parts;
            const cudaError_t e = allow_smem<&k_append_scaled<decltype(t), LPR, IL, PAGES, STEPS>>(std::max(ring, most));
            if (e != cudaSuccess) return e;
        } else {
            grid = div_up(static_cast<int64_t>(f.T) * jobs, kWarps);
        }
        if (grid > INT32_MAX) return cudaErrorInvalidValue;
        k_append_scaled<decltype(t), LPR, IL, PAGES, STEPS>
            <<<static_cast<unsigned>(grid), kThreads, smem, f.stream>>>(a, static_cast<int>(parts), group_warps);
        count_launch();
        return cudaGetLastError();
    };
    // A warp a page and head or a CTA a page, by the tokens of a request on average (the
    // host knows no more).  Measured with 1 / 2 / 4 / 6 / 8 tokens for each of 64 requests, 48
    // heads: 128 elements, pages of 64: 5 / 7 / 12 / 17 / 21 us and 21 to 22; of 16: the same
    // and 11 to 13; 64 elements, pages of 64: 5 / 7 / 9 / 15 / 17 and 16.  A chunk of 190
    // tokens beside 63 single ones, which the average hides, takes 42 us for 22 (64 elements:
    // 23 for 16).
    const auto by_group = [&](auto t, auto lpr, auto il) {
        return f.T <= 4 * static_cast<int64_t>(pg.n_seqs) ? run(t, lpr, il, std::false_type{}) : run(t, lpr, il, std::true_type{});
    };
    const auto by_il = [&](auto t, auto lpr) {
        return f.rot.interleaved ? by_group(t, lpr, std::true_type{}) : by_group(t, lpr, std::false_type{});
    };
    const auto by_lpr = [&](auto t) {
        return f.D == 64 ? by_il(t, integral_constant<int, 8>{}) : by_il(t, integral_constant<int, 16>{});
    };
    return f.dtype == BEVPOOL_F16 ? by_lpr(__half{}) : by_lpr(__nv_bfloat16{});
}

}  // namespace bevpool
