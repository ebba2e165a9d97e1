// attend_few.cuh -- attention of few query rows (single tokens above all): at
// most 16 rows a request and key head, the query heads of a group being rows
// too, so that each key and value is read once for all of them.
//
// Bound by the read of the cache.  The keys are cut into chunks, one a CTA,
// so that few requests still fill the GPU; inside a CTA four warps take tiles
// in turn, each with its own ring of tiles filled by asynchronous copies and
// its own running softmax, so nothing synchronises the warps until the end.
// S = Q K^T and O += P V run on warp-level matrix instructions (16 rows by 8
// columns by 16): their rate is far above what the copies deliver, and a
// 128-row tile would be empty but for a few rows.
//
// E4M3 codes stay codes in shared memory and are widened in registers.  For
// K a thread's four consecutive codes serve as its four places along the
// product's inner axis (Q is loaded in the same order); for V a transposed
// load of 2-byte units yields two columns at once.  Both products are then of
// fp16, which holds every code and is one conversion away (bf16 would be four):
// a bf16 query row is first scaled by the power of two that brings its largest
// element to 2^14 (elements 2^-31 of it and more keep all their bits), and its
// scores by the inverse.
//
// fp16 weights carry a factor of 2^14, so that they keep 11 bits down to 2^-28
// of the largest.
//
// Page scales (nine to sixteen rows; fewer: attend_codes.cu): a tile's scales come with
// it, by copies of 4 bytes, and go into its scores, weights and sums (PageFactors).
//
// Measured on a GB300, 32 query and 8 key heads of 128: 64 requests of up to 8192
// keys, bf16: 233 us (6.6 TB/s, 98 % of measured copy); two requests of up to
// 131072 keys in E4M3: 91 us (4.6 TB/s, 68 %: no unit is saturated (ALU 44 %, issue
// slots 36 %), eight warps an SM do not cover the way from the copies through the
// conversions to the products); one request of 777 keys, 8 heads of 64: 8.3 us on
// the GPU, 10 to 12 a call.
#pragma once

#include "paged_attention.cuh"
#include "warp_mma.cuh"

namespace bevpool {

namespace {

constexpr int kFewWarps = 4;
constexpr int kFewStages = 3;

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}

template <bool E4M3, int D>
struct FewShape {
    static constexpr int EB = E4M3 ? 1 : 2;
    static constexpr int RB = D * EB;                      // bytes of a cache row
    static constexpr int CPR = RB / 16;                    // 16-byte pieces of it
    static constexpr int KT = 4096 / RB;                   // keys of a tile: 4 KB of K, 4 KB of V
    static constexpr int TILE = KT * RB;
    static constexpr int STAGE = 2 * TILE;
    static constexpr int SMEM = kFewWarps * kFewStages * STAGE;
    // Place of a piece in its row, so that eight rows of a piece fall on
    // different banks.
    static __device__ __forceinline__ int swz(int row, int c) {
        return RB == 64 ? c ^ ((row >> 1) & 3) : c ^ (row & 7);
    }
};

template <typename T, int C, int D>
__global__ void __launch_bounds__(kFewWarps * 32, 2)
k_attend_few(AttnArgs a, AttnPlan pl) {
    constexpr bool E4M3 = C != kCacheSame, SCALED = C == kCacheScaled;
    using S = FewShape<E4M3, D>;
    using M = typename std::conditional<E4M3, __half, T>::type;             // type of both products
    constexpr float kLift = std::is_same<M, __half>::value ? 14.0f : 0.0f;  // log2 of the weights' factor
    constexpr int KS = D / 16, NT = D / 8, KG = S::KT / 16;                // k steps of S, columns tiles of O, 16-key groups
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, qd = lane & 3;
    const int hk = blockIdx.y, b = blockIdx.z;
    const Request r = request_of(a, b);
    if (r.q_rows == 0) return;
    int32_t base;
    const int n_used = chunks_of(a, r, pl, &base);
    if (static_cast<int>(blockIdx.x) >= n_used) return;
    const int rows = r.q_rows * a.G;

    // Rows g and g + 8 of this thread: what they see and their query (places
    // past the last row see all and are not kept).
    int32_t lo[2] = {0, 0}, hi[2] = {INT32_MAX, INT32_MAX};
    uint32_t qf[KS][4] = {};
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int row = g + 8 * x;
        if (row >= rows) continue;
        const int i = row / a.G, h = hk * a.G + row % a.G;
        seen_keys(a, r, i, &lo[x], &hi[x]);
        const T *qp = static_cast<const T *>(a.q.p) + static_cast<int64_t>(r.q0 + i) * a.q.token_stride +
                      h * a.q.head_stride;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            qf[k][x] = *reinterpret_cast<const uint32_t *>(qp + 16 * k + (E4M3 ? 4 * qd : 2 * qd));
            qf[k][x + 2] = *reinterpret_cast<const uint32_t *>(qp + 16 * k + (E4M3 ? 4 * qd + 2 : 2 * qd + 8));
        }
    }
    // scale of a row's scores (base 2)
    float scale[2] = {a.scale_log2, a.scale_log2};
    if constexpr (E4M3 && !std::is_same<T, __half>::value) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float top = 0.0f;
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int y = x; y < 4; y += 2)
                    top = fmaxf(top, fmaxf(fabsf(__uint_as_float(qf[k][y] << 16)), fabsf(__uint_as_float(qf[k][y] & 0xffff0000u))));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -112), 127);     // its exponent
            const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);               // 2^(14 - e)
            scale[x] *= __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23);
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int y = x; y < 4; y += 2)
                    qf[k][y] = pack2<__half>(__uint_as_float(qf[k][y] << 16) * up, __uint_as_float(qf[k][y] & 0xffff0000u) * up);
        }
    }
    int32_t first, last, tmp;                              // keys that any row sees
    seen_keys(a, r, 0, &first, &tmp);
    seen_keys(a, r, r.q_rows - 1, &tmp, &last);
    const int32_t c0 = base + static_cast<int32_t>(blockIdx.x) * pl.chunk;
    const int32_t c1 = static_cast<int32_t>(min(static_cast<int64_t>(c0) + pl.chunk, static_cast<int64_t>(last)));

    const uint32_t ring = smem_addr(smem) + warp * kFewStages * S::STAGE;
    // past the rings: the scales of a tile's 16-key groups, keys' then values'
    const uint32_t scale_ring = smem_addr(smem) + S::SMEM + warp * kFewStages * 2 * KG * 4;
    const int32_t *table = a.pg.block_table + static_cast<int64_t>(b) * a.pg.table_pages;
    const char *kc = static_cast<const char *>(a.k_cache), *vc = static_cast<const char *>(a.v_cache);
    const int64_t head_off = hk * a.pg.head_stride;

    // Pages of a tile's 16-key groups (a group lies inside a page); -1 where
    // there is none.
    auto pages_of = [&](int32_t j, int32_t *pg) {
#pragma unroll
        for (int x = 0; x < KG; ++x) {
            const int32_t k = j + 16 * x;
            pg[x] = -1;
            if (k < c1) {
                const int32_t p = table[k >> a.pg.page_shift];
                if (p >= 0 && p < a.pg.n_pages) pg[x] = p;
            }
        }
    };
    auto fetch = [&](int stage, int32_t j, const int32_t *pg) {
        const uint32_t dst = ring + stage * S::STAGE;
        constexpr int RPI = 32 / S::CPR;                   // rows a copy of the warp covers
        const int c = lane % S::CPR, r0 = lane / S::CPR;
#pragma unroll
        for (int i = 0; i < S::KT / RPI; ++i) {
            const int row = i * RPI + r0;
            const int32_t k = j + row, p = pg[i * RPI / 16];
            const bool on = p >= 0 && k >= first && k < c1;
            const int64_t at = on ? (p * a.pg.page_stride + (k & (a.pg.page_size - 1)) * a.pg.slot_stride + head_off) *
                                            S::EB + c * 16
                                  : 0;
            const uint32_t d = dst + row * S::RB + S::swz(row, c) * 16;
            copy16(d, kc + at, on);
            copy16(d + S::TILE, vc + at, on);
        }
        if constexpr (SCALED) {
            if (lane < 2 * KG) {
                int32_t p = pg[0];
#pragma unroll
                for (int x = 1; x < KG; ++x) p = lane % KG == x ? pg[x] : p;
                const float *scales = lane < KG ? a.k_scales : a.v_scales;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(scale_ring + (stage * 2 * KG + lane) * 4),
                             "l"(scales + (p >= 0 ? static_cast<int64_t>(p) * a.Hk + hk : 0)), "r"(p >= 0 ? 4 : 0)
                             : "memory");
            }
        }
    };

    float o[NT][4] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    const int32_t step = kFewWarps * S::KT;
    int32_t j = c0 + warp * S::KT;
    uint32_t holes = 0;                                    // bit s * KG + x: group x of ring place s has no page
    int32_t pg[KG];
    auto note = [&](int stage) {
        uint32_t h = 0;
#pragma unroll
        for (int x = 0; x < KG; ++x) h |= (pg[x] < 0 ? 1u : 0u) << x;
        holes = (holes & ~(((1u << KG) - 1) << (stage * KG))) | (h << (stage * KG));
    };
#pragma unroll
    for (int s = 0; s < kFewStages - 1; ++s) {
        if (j + s * step < c1) {
            pages_of(j + s * step, pg);
            fetch(s, j + s * step, pg);
            note(s);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    pages_of(j + (kFewStages - 1) * step, pg);
    for (int stage = 0; j < c1; j += step) {
        const int fill = stage == 0 ? kFewStages - 1 : stage - 1;
        if (j + (kFewStages - 1) * step < c1) {
            fetch(fill, j + (kFewStages - 1) * step, pg);
            note(fill);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        pages_of(j + kFewStages * step, pg);               // for the next round, so that its copies need not wait
        asm volatile("cp.async.wait_group %0;" ::"n"(kFewStages - 1) : "memory");
        __syncwarp();
        const uint32_t kt = ring + stage * S::STAGE, vt = kt + S::TILE;

        // S = Q K^T
        float s[S::KT / 8][4] = {};
#pragma unroll
        for (int n = 0; n < S::KT / 8; ++n) {
            const int row = n * 8 + (lane & 7), piece = lane >> 3;
#pragma unroll
            for (int c = 0; c < S::CPR; c += 4) {
                uint32_t w[4];
                ldm4(kt + row * S::RB + S::swz(row, c + piece) * 16, w);
                if constexpr (E4M3) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) mma<M>(s[n], qf[c + x], widen2<M>(w[x] & 0xffff), widen2<M>(w[x] >> 16));
                } else {
                    mma<M>(s[n], qf[c / 2], w[0], w[1]);
                    mma<M>(s[n], qf[c / 2 + 1], w[2], w[3]);
                }
            }
        }
        const uint32_t hole = (holes >> (stage * KG)) & ((1u << KG) - 1);
        const bool whole = hole == 0 && j >= max(lo[0], lo[1]) && j + S::KT <= min(hi[0], hi[1]);
        float sums[KG];                                    // SCALED: factors of the groups' sums
        if constexpr (SCALED) {
#pragma unroll
            for (int x = 0; x < KG; ++x) {
                float ks, vs;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(ks) : "r"(scale_ring + (stage * 2 * KG + x) * 4) : "memory");
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(vs) : "r"(scale_ring + (stage * 2 * KG + KG + x) * 4) : "memory");
                const PageFactors f = page_factors(1.0f, ks, vs);
                sums[x] = f.sum;
                const float up[2] = {scale[0] * f.score, scale[1] * f.score};
#pragma unroll
                for (int n = 2 * x; n < 2 * x + 2; ++n)
#pragma unroll
                    for (int y = 0; y < 4; ++y) s[n][y] = fmaf(s[n][y], up[y >> 1], f.lift);
            }
        } else {
#pragma unroll
            for (int n = 0; n < S::KT / 8; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[n][x] *= scale[x >> 1];
        }
        if (!__all_sync(0xffffffffu, whole)) {
#pragma unroll
            for (int n = 0; n < S::KT / 8; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int32_t k = j + n * 8 + 2 * qd + (x & 1);
                    if (k < lo[x >> 1] || k >= hi[x >> 1] || ((hole >> (n / 2)) & 1)) s[n][x] = -INFINITY;
                }
        }
        // running maximum, weights, sum
        float mn[2] = {m[0], m[1]};
#pragma unroll
        for (int n = 0; n < S::KT / 8; ++n) {
            mn[0] = fmaxf(mn[0], fmaxf(s[n][0], s[n][1]));
            mn[1] = fmaxf(mn[1], fmaxf(s[n][2], s[n][3]));
        }
        float keep[2], from[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            mn[x] = fmaxf(mn[x], __shfl_xor_sync(0xffffffffu, mn[x], 1));
            mn[x] = fmaxf(mn[x], __shfl_xor_sync(0xffffffffu, mn[x], 2));
            from[x] = (mn[x] == -INFINITY ? 0.0f : mn[x]) - kLift;
            keep[x] = pow2(m[x] - kLift - from[x]);
            l[x] *= keep[x];
        }
        if (__any_sync(0xffffffffu, mn[0] != m[0] || mn[1] != m[1])) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                o[n][0] *= keep[0];
                o[n][1] *= keep[0];
                o[n][2] *= keep[1];
                o[n][3] *= keep[1];
            }
        }
        m[0] = mn[0];
        m[1] = mn[1];
        // O += P V, 16 keys at a time.  The sum l takes the weights before
        // their rounding to 16 bits.
#pragma unroll
        for (int x = 0; x < KG; ++x) {
            uint32_t pf[4];
            float lx[2] = {0.0f, 0.0f};
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float p0 = pow2(s[2 * x + n][0] - from[0]), p1 = pow2(s[2 * x + n][1] - from[0]);
                const float p2 = pow2(s[2 * x + n][2] - from[1]), p3 = pow2(s[2 * x + n][3] - from[1]);
                lx[0] += p0 + p1;
                lx[1] += p2 + p3;
                pf[2 * n] = pack2<M>(p0, p1);
                pf[2 * n + 1] = pack2<M>(p2, p3);
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) l[y] = SCALED ? fmaf(lx[y], sums[x], l[y]) : l[y] + lx[y];
            const int row = 16 * x + (lane & 15), piece = lane >> 4;
#pragma unroll
            for (int c = 0; c < S::CPR; c += 2) {
                uint32_t w[4];
                ldm4t(vt + row * S::RB + S::swz(row, c + piece) * 16, w);
                if constexpr (E4M3) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t w0 = w[2 * y], w1 = w[2 * y + 1];
                        mma<M>(o[2 * (c + y)], pf, widen2<M>(__byte_perm(w0, 0, 0x4420)), widen2<M>(__byte_perm(w1, 0, 0x4420)));
                        mma<M>(o[2 * (c + y) + 1], pf, widen2<M>(__byte_perm(w0, 0, 0x4431)),
                               widen2<M>(__byte_perm(w1, 0, 0x4431)));
                    }
                } else {
                    mma<M>(o[c], pf, w[0], w[1]);
                    mma<M>(o[c + 1], pf, w[2], w[3]);
                }
            }
        }
        __syncwarp();
        stage = stage == kFewStages - 1 ? 0 : stage + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();

    // Join the four warps: each leaves its maximum, sum and O in shared memory.
    float *so = reinterpret_cast<float *>(smem);                           // [warp][16][D + 4]
    constexpr int LD = D + 4;
    float *sm = so + kFewWarps * 16 * LD;                                  // [warp][16][2]
    static_assert((kFewWarps * 16 * (D + 6) + 1) * 4 <= S::SMEM, "the join fits the ring");
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
        const int row = g + 8 * x;
        if (qd == 0) {
            sm[(warp * 16 + row) * 2] = m[x] - kLift;
            sm[(warp * 16 + row) * 2 + 1] = l[x];
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float *d = so + (warp * 16 + row) * LD;
            if constexpr (E4M3) {
                const int at = 16 * (n >> 1) + 4 * qd + (n & 1);
                d[at] = o[n][2 * x];
                d[at + 2] = o[n][2 * x + 1];
            } else {
                d[8 * n + 2 * qd] = o[n][2 * x];
                d[8 * n + 2 * qd + 1] = o[n][2 * x + 1];
            }
        }
    }
    __syncthreads();
    constexpr int E = D / 32;
    for (int row = warp; row < rows; row += kFewWarps) {
        float mt = -INFINITY, lt = 0.0f, acc[E] = {};
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) mt = fmaxf(mt, sm[(w * 16 + row) * 2]);
        const float from = mt == -INFINITY ? 0.0f : mt;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
            const float f = pow2(sm[(w * 16 + row) * 2] - from);
            lt = fmaf(sm[(w * 16 + row) * 2 + 1], f, lt);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(so[(w * 16 + row) * LD + lane * E + e], f, acc[e]);
        }
        const int i = row / a.G, h = hk * a.G + row % a.G;
        bool fine = lt - lt == 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) fine = fine && acc[e] - acc[e] == 0.0f;
        // An infinity or NaN may come from a key that another token of the
        // chunk sees and this one does not (its weight 0 times the value): the
        // row is then taken again element by element.
        if (r.q_rows > 1 && !__all_sync(0xffffffffu, fine))
            redo_row<T, C, D>(a, r, b, hk, i, h, c0, c1, &mt, &lt, acc);
        store_row<T, E>(a, r, i, h, n_used > 1 ? part_row(a, pl, b, hk, static_cast<int>(blockIdx.x), row) : -1, mt, lt, acc);
    }
    grid_dep_allow();
}

// The launch of one of the caches' kernels.
template <typename T, int C, int D>
cudaError_t run_attend_few(const AttnArgs &a, const AttnPlan &pl) {
    using S = FewShape<C != kCacheSame, D>;
    constexpr int smem = S::SMEM + (C == kCacheScaled ? kFewWarps * kFewStages * 2 * (S::KT / 16) * 4 : 0);
    const cudaError_t e = allow_smem<&k_attend_few<T, C, D>>(smem);
    if (e != cudaSuccess) return e;
    k_attend_few<T, C, D><<<dim3(static_cast<unsigned>(pl.n_chunks), static_cast<unsigned>(a.Hk), static_cast<unsigned>(a.pg.n_seqs)),
                            kFewWarps * 32, smem, a.stream>>>(a, pl);
    count_launch();
    return cudaGetLastError();
}

template <int C>
cudaError_t launch_attend_few_of(const AttnArgs &a, const AttnPlan &pl) {
    if (a.dtype == BEVPOOL_F16) return a.D == 64 ? run_attend_few<__half, C, 64>(a, pl) : run_attend_few<__half, C, 128>(a, pl);
    return a.D == 64 ? run_attend_few<__nv_bfloat16, C, 64>(a, pl) : run_attend_few<__nv_bfloat16, C, 128>(a, pl);
}

}  // namespace

}  // namespace bevpool
