// attend_codes.cu -- attention of at most eight query rows a request and key head
// over E4M3 codes with a scale for each page and key head (single tokens above all;
// nine to sixteen rows: attend_few.cuh).
//
// Laid out as the few-rows kernel: the keys are cut into chunks, one a CTA, whose
// four warps take tiles in turn, each with its own ring and its own running softmax.
// What bounds it is the read of the cache, and next the instructions between a
// tile's arrival and its sums, so these are kept few:
//   - a tile's pages come by TMA, a box a page, issued by the lanes that looked the
//     pages up; each tile has a barrier;
//   - S = Q K^T takes the keys' codes as they are, in E4M3 products.  The queries are
//     split into codes too, q = hi + lo / 32 (+ least / 1024 for fp16), scaled by the
//     power of two that brings a row's largest element to [128, 256): each part takes
//     four bits more, so a bf16 (fp16) element keeps all of its bits down to 2^-14
//     (2^-17) of the largest, and what a smaller one loses is 2^-22 (2^-27) of that.
//     Rows 8 to 15 of a product are the lo parts of rows 0 to 7, joined in FP32;
//   - O^T += V^T P^T: the head's elements are the product's rows and the query rows
//     its columns, half as many products as the other way round.  Codes are widened
//     to fp16 on the way, weights are fp16 times 2^14 as in the few-rows kernel.
//
// Measured on a GB300, 32 query and 8 key heads of 128, bf16: 64 requests of up to 8192
// keys, pages of 16: 137 us (5.6 TB/s, 82 % of measured copy; the few-rows kernel 154);
// two requests of up to 131072 keys, pages of 64: 76 us (5.4 TB/s, 80 %; 94): what is
// left is mostly a CTA's start (four lookups that wait for each other), the shorter
// request's idle places and the join; one request of 777 keys, 8 heads of 64: 10.5 to 12.5
// us a call (13.5).  Two CTAs an SM with three tiles a ring instead of three with two:
// 144 and 91 us where these took 137 and 86; four with tiles of 2 KB: 142 and 85.
#include "tcgen05.cuh"
#include "tensor_map.cuh"
#include "warp_mma.cuh"

namespace bevpool {

namespace {

__device__ unsigned long long g_timeouts;

constexpr int kCodesWarps = 4, kCodesStages = 2, kCodesRows = 8;

template <int D>
struct CodesShape {
    static constexpr int TILE = 4096, STAGE = 2 * TILE;    // bytes of keys, and with the values
    static constexpr int KT = TILE / D, GROUPS = KT / 16;  // keys of a tile, groups of 16
    static constexpr int CPR = D / 16;                     // 16-byte pieces of a row
    static constexpr int SMEM = 1024 + kCodesWarps * kCodesStages * STAGE;
    // Place of a piece in its row: the 128-byte (64-byte) swizzle.
    static __device__ __forceinline__ int swz(int row, int c) { return D == 64 ? c ^ ((row >> 1) & 3) : c ^ (row & 7); }
};

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) { return pack4_e4m3(pair(a, b), pair(c, d)); }

// Four values less their codes, times 32.
__device__ __forceinline__ void rest4(uint32_t codes, float *x) {
    const uint32_t u = widen2<__half>(codes & 0xffffu), v = widen2<__half>(codes >> 16);
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u)), g = __half22float2(*reinterpret_cast<const __half2 *>(&v));
    x[0] = (x[0] - f.x) * 32.0f, x[1] = (x[1] - f.y) * 32.0f, x[2] = (x[2] - g.x) * 32.0f, x[3] = (x[3] - g.y) * 32.0f;
}

template <typename T, int D>
__global__ void __launch_bounds__(kCodesWarps * 32, kCodesCtas)
k_attend_codes(AttnArgs a, AttnPlan pl, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    using S = CodesShape<D>;
    constexpr bool FINE = std::is_same<T, __half>::value;  // a third part
    constexpr int KS = D / 32, NT = S::KT / 8, CH = D / 16;
    constexpr float kLift = 14.0f;
    extern __shared__ uint8_t raw_smem[];
    __shared__ uint64_t full[kCodesWarps][kCodesStages];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, qd = lane & 3;
    const int hk = blockIdx.y, b = blockIdx.z;
    const Request r = request_of(a, b);
    if (r.q_rows == 0) return;
    int32_t base;
    const int n_used = chunks_of(a, r, pl, &base);
    if (static_cast<int>(blockIdx.x) >= n_used) return;
    const int rows = r.q_rows * a.G;
    int32_t first, last, tmp;                              // keys that any row sees
    seen_keys(a, r, 0, &first, &tmp);
    seen_keys(a, r, r.q_rows - 1, &tmp, &last);
    const int32_t c0 = base + static_cast<int32_t>(blockIdx.x) * pl.chunk;
    const int32_t c1 = static_cast<int32_t>(min(static_cast<int64_t>(c0) + pl.chunk, static_cast<int64_t>(last)));
    const uint32_t smem = (shared_addr(raw_smem) + 1023) & ~1023u, ring = smem + warp * kCodesStages * S::STAGE;
    const int32_t *table = a.pg.block_table + static_cast<int64_t>(b) * a.pg.table_pages;

    // Pages of a tile: box x, of `high` slots, is lane x's.
    const int high = min(a.pg.page_size, S::KT), boxes = S::KT / high;
    auto page_of = [&](int32_t j) {                        // n_pages (the box fills with zeros): none
        const int32_t k = j + lane * high;
        int32_t p = a.pg.n_pages;
        if (lane < boxes && k < c1) {
            const int32_t x = table[k >> a.pg.page_shift];
            if (x >= 0 && x < a.pg.n_pages) p = x;
        }
        return p;
    };
    auto fetch = [&](int stage, int32_t j, int32_t page) {
        const uint32_t bar = shared_addr(&full[warp][stage]), dst = ring + stage * S::STAGE + lane * high * D;
        if (lane == 0) bar_expect(bar, S::STAGE);
        __syncwarp();
        if (lane < boxes) {
            const int32_t slot = (j + lane * high) & (a.pg.page_size - 1);
            tma_load_4d(dst, &k_map, bar, 0, slot, hk, page);
            tma_load_4d(dst + S::TILE, &v_map, bar, 0, slot, hk, page);
        }
    };
    float ks = 1.0f, vs = 1.0f;                            // of this lane's box of the tile at work
    auto scales_of = [&](int32_t p) {
        const int64_t i = static_cast<int64_t>(p < a.pg.n_pages ? p : 0) * a.Hk + hk;
        if (lane < boxes) {
            ks = a.k_scales[i];
            vs = a.v_scales[i];
        }
    };
    if (lane == 0) {
        for (int s = 0; s < kCodesStages; ++s) bar_init(shared_addr(&full[warp][s]), 1);
        bar_init_fence();
    }
    __syncwarp();
    const int32_t step = kCodesWarps * S::KT;
    int32_t j = c0 + warp * S::KT;
    int32_t pages[kCodesStages + 1];                       // of the tile at work and of those after it
#pragma unroll
    for (int s = 0; s <= kCodesStages; ++s) pages[s] = page_of(j + s * step);
#pragma unroll
    for (int s = 0; s < kCodesStages - 1; ++s)
        if (j + s * step < c1) fetch(s, j + s * step, pages[s]);
    scales_of(pages[0]);

    // Row g: what it sees, and its query in parts.
    int32_t lo = 0, hi = INT32_MAX;
    uint32_t qa[KS][4] = {}, qc[FINE ? KS : 1][4] = {};
    float scale = 0.0f;                                    // of its scores (base 2)
    {
        float x[KS][8] = {};
        float top = 0.0f;
        bool fine = true;
        if (g < rows) {
            const int i = g / a.G, h = hk * a.G + g % a.G;
            seen_keys(a, r, i, &lo, &hi);
            const T *qp = static_cast<const T *>(a.q.p) + static_cast<int64_t>(r.q0 + i) * a.q.token_stride + h * a.q.head_stride + 4 * qd;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(qp + 32 * k + 16 * y);
                    unpair(widen<T>(w.x), &x[k][4 * y], &x[k][4 * y + 1]);
                    unpair(widen<T>(w.y), &x[k][4 * y + 2], &x[k][4 * y + 3]);
                }
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    top = fmaxf(top, fabsf(x[k][y]));
                    fine = fine && x[k][y] - x[k][y] == 0.0f;
                }
            }
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const unsigned bad = __ballot_sync(0xffffffffu, !fine);
        const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -113), 127);         // its exponent
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 7 - e) << 23);                    // 2^(7 - e)
        scale = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - 7 + e) << 23);
        if ((bad >> (4 * g)) & 15) scale = NAN;            // codes hold no infinity
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float *z = x[k] + 4 * y;
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] *= up;
                qa[k][2 * y] = codes4(z[0], z[1], z[2], z[3]);
                rest4(qa[k][2 * y], z);
                qa[k][2 * y + 1] = codes4(z[0], z[1], z[2], z[3]);
                if constexpr (FINE) {
                    rest4(qa[k][2 * y + 1], z);
                    qc[k][2 * y] = codes4(z[0], z[1], z[2], z[3]);
                }
            }
    }

    float o[CH][4] = {}, m = -INFINITY, l = 0.0f;
    uint32_t phase = 0;
    bool ok = true;
    for (int stage = 0; j < c1; j += step) {
        const int fill = stage == 0 ? kCodesStages - 1 : stage - 1;
        if (j + (kCodesStages - 1) * step < c1) fetch(fill, j + (kCodesStages - 1) * step, pages[kCodesStages - 1]);
        const PageFactors mine = page_factors(1.0f, ks, vs);
        const uint32_t hole = __ballot_sync(0xffffffffu, lane < boxes && pages[0] >= a.pg.n_pages);
#pragma unroll
        for (int s = 0; s < kCodesStages; ++s) pages[s] = pages[s + 1];
        pages[kCodesStages] = page_of(j + (kCodesStages + 1) * step);
        scales_of(pages[0]);
        ok = bar_wait(shared_addr(&full[warp][stage]), phase);
        if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
        }
        const uint32_t kt = ring + stage * S::STAGE, vt = kt + S::TILE;
        if (j < first || j + S::KT > c1) {                 // values that no row sees: 0 * NaN is not 0
            for (int i = lane; i < S::KT * S::CPR; i += 32) {
                const int32_t k = j + i / S::CPR;
                if (k < first || k >= c1) asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(vt + i * 16), "r"(0) : "memory");
            }
            fence_shared_async();                          // before the next copy to this place
            __syncwarp();
        }

        // S = Q K^T
        float s[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int row = n * 8 + (lane & 7), piece = lane >> 3;
            float c[4] = {}, d[4] = {};
#pragma unroll
            for (int p = 0; p < S::CPR; p += 4) {
                uint32_t w[4];
                ldm4(kt + row * D + S::swz(row, p + piece) * 16, w);
                mma_e4m3(c, qa[p / 2], w[0], w[1]);
                mma_e4m3(c, qa[p / 2 + 1], w[2], w[3]);
                if constexpr (FINE) {
                    mma_e4m3(d, qc[p / 2], w[0], w[1]);
                    mma_e4m3(d, qc[p / 2 + 1], w[2], w[3]);
                }
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) s[n][x] = fmaf(FINE ? fmaf(d[x], 0x1p-5f, c[x + 2]) : c[x + 2], 0x1p-5f, c[x]);
        }
        float sums[S::GROUPS];
#pragma unroll
        for (int x = 0; x < S::GROUPS; ++x) {
            const int from = x * 16 / high;
            const float up = scale * __shfl_sync(0xffffffffu, mine.score, from), lift = __shfl_sync(0xffffffffu, mine.lift, from);
            sums[x] = __shfl_sync(0xffffffffu, mine.sum, from);
#pragma unroll
            for (int n = 2 * x; n < 2 * x + 2; ++n)
#pragma unroll
                for (int y = 0; y < 2; ++y) s[n][y] = fmaf(s[n][y], up, lift);
        }
        if (!__all_sync(0xffffffffu, hole == 0 && j >= lo && j + S::KT <= hi)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int32_t k = j + n * 8 + 2 * qd + x;
                    if (k < lo || k >= hi || ((hole >> (n * 8 / high)) & 1)) s[n][x] = -INFINITY;
                }
        }
        // running maximum, weights, sum
        float mn = m;
#pragma unroll
        for (int n = 0; n < NT; ++n) mn = max3(mn, s[n][0], s[n][1]);
        mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 1));
        mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 2));
        const float from = (mn == -INFINITY ? 0.0f : mn) - kLift;
        if (__any_sync(0xffffffffu, mn != m)) {
            const float keep = pow2(m - kLift - from);
            l *= keep;
            const float k0 = __shfl_sync(0xffffffffu, keep, 8 * qd), k1 = __shfl_sync(0xffffffffu, keep, 8 * qd + 4);     // rows 2 qd, 2 qd + 1
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                o[c][0] *= k0;
                o[c][1] *= k1;
                o[c][2] *= k0;
                o[c][3] *= k1;
            }
        }
        m = mn;
        // O^T += V^T P^T, 16 keys at a time.  The sum takes the weights before their
        // rounding to 16 bits.
#pragma unroll
        for (int x = 0; x < S::GROUPS; ++x) {
            uint32_t pf[2];
            float lx = 0.0f;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float p0 = pow2(s[2 * x + n][0] - from), p1 = pow2(s[2 * x + n][1] - from);
                lx += p0 + p1;
                pf[n] = pack2<__half>(p0, p1);
            }
            l = fmaf(lx, sums[x], l);
            const int row = 16 * x + (lane & 15), piece = lane >> 4;
#pragma unroll
            for (int c = 0; c < CH; c += 2) {
                uint32_t w[4];
                ldm4t(vt + row * D + S::swz(row, c + piece) * 16, w);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const uint32_t w0 = w[2 * y], w1 = w[2 * y + 1];
                    const uint32_t va[4] = {widen2<__half>(__byte_perm(w0, 0, 0x4420)), widen2<__half>(__byte_perm(w0, 0, 0x4431)),
                                            widen2<__half>(__byte_perm(w1, 0, 0x4420)), widen2<__half>(__byte_perm(w1, 0, 0x4431))};
                    mma<__half>(o[c + y], va, pf[0], pf[1]);
                }
            }
        }
        __syncwarp();
        if (stage == kCodesStages - 1) {
            stage = 0;
            phase ^= 1;
        } else {
            ++stage;
        }
    }
    if (!ok) {                                             // a wait ran out: NaN, and what is still on its way is waited for
        l = NAN;
        for (int s = 0; s < kCodesStages; ++s) bar_wait(shared_addr(&full[warp][s]), phase);
        if (lane == 0) atomicAdd(&g_timeouts, 1ull);
    }
    __syncthreads();

    // Join the four warps: each leaves its maximum, sum and O in shared memory.
    constexpr int LD = D + 4;
    float *so = reinterpret_cast<float *>(raw_smem + (smem - shared_addr(raw_smem)));     // [warp][8][D + 4]
    float *sm = so + kCodesWarps * kCodesRows * LD;                                        // [warp][8][2]
    static_assert(kCodesWarps * kCodesRows * (D + 6) * 4 <= S::SMEM - 1024, "the join fits the ring");
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (qd == 0) {
        sm[(warp * kCodesRows + g) * 2] = m - kLift;
        sm[(warp * kCodesRows + g) * 2 + 1] = l;
    }
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int x = 0; x < 2; ++x)
            *reinterpret_cast<float2 *>(so + (warp * kCodesRows + 2 * qd + x) * LD + 16 * c + 2 * g) = make_float2(o[c][x], o[c][x + 2]);
    __syncthreads();
    constexpr int E = D / 32;
    for (int row = warp; row < rows; row += kCodesWarps) {
        float mt = -INFINITY, lt = 0.0f, acc[E] = {};
#pragma unroll
        for (int w = 0; w < kCodesWarps; ++w) mt = fmaxf(mt, sm[(w * kCodesRows + row) * 2]);
        const float from = mt == -INFINITY ? 0.0f : mt;
#pragma unroll
        for (int w = 0; w < kCodesWarps; ++w) {
            const float f = pow2(sm[(w * kCodesRows + row) * 2] - from);
            lt = fmaf(sm[(w * kCodesRows + row) * 2 + 1], f, lt);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(so[(w * kCodesRows + row) * LD + lane * E + e], f, acc[e]);
        }
        const int i = row / a.G, h = hk * a.G + row % a.G;
        bool fine = lt - lt == 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) fine = fine && acc[e] - acc[e] == 0.0f;
        // A NaN may come from a key that another token of the chunk sees and this one
        // does not (its weight 0 times the value): the row is then taken again element
        // by element.
        if (r.q_rows > 1 && !__all_sync(0xffffffffu, fine))
            redo_row<T, kCacheScaled, D>(a, r, b, hk, i, h, c0, c1, &mt, &lt, acc);
        store_row<T, E>(a, r, i, h, n_used > 1 ? part_row(a, pl, b, hk, static_cast<int>(blockIdx.x), row) : -1, mt, lt, acc);
    }
    grid_dep_allow();
}

template <typename T, int D>
cudaError_t run(const AttnArgs &a, const AttnPlan &pl) {
    using S = CodesShape<D>;
    CUtensorMap k_map, v_map;
    if (!code_map(a, a.k_cache, S::KT, true, &k_map) || !code_map(a, a.v_cache, S::KT, true, &v_map)) return cudaErrorInvalidValue;
    const cudaError_t e = allow_smem<&k_attend_codes<T, D>>(S::SMEM);
    if (e != cudaSuccess) return e;
    k_attend_codes<T, D><<<dim3(static_cast<unsigned>(pl.n_chunks), static_cast<unsigned>(a.Hk), static_cast<unsigned>(a.pg.n_seqs)),
                           kCodesWarps * 32, S::SMEM, a.stream>>>(a, pl, k_map, v_map);
    count_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t attend_codes_timeouts(int64_t *count) {
    unsigned long long n = 0;
    const cudaError_t e = cudaMemcpyFromSymbol(&n, g_timeouts, sizeof(n));
    if (e == cudaSuccess) *count += static_cast<int64_t>(n);
    return e;
}

cudaError_t launch_attend_codes(const AttnArgs &a, const AttnPlan &pl) {
    if (a.dtype == BEVPOOL_F16) return a.D == 64 ? run<__half, 64>(a, pl) : run<__half, 128>(a, pl);
    return a.D == 64 ? run<__nv_bfloat16, 64>(a, pl) : run<__nv_bfloat16, 128>(a, pl);
}

}  // namespace bevpool
