// attend_tile.cu -- attention of many query rows on the tcgen05 tensor cores.
//
// The rows of a request and key head are its new tokens times the query heads
// of the group, so that a tile of 128 rows is full even for short chunks and
// each key is read once for the whole group.  A CTA holds two row tiles and
// walks the keys in blocks of 128:
//   warps 0-3, 4-7   softmax of tile 0, 1 (one row a thread): S from tensor
//                    memory, running maximum and sum, P (16 bits) back over S
//   warps 8, 9       issue the products of tile 0, 1: S = Q K^T (both from shared
//                    memory) and O += P V (P from tensor memory), O in tensor memory
//   warp 10          loads K and V: a TMA box for each page and 64 elements of
//                    the head, into a ring of 128-byte-swizzled blocks
//   warps 12-15      (E4M3 cache instead) load codes, widen them to 16 bits and
//                    store them in the same layout
// While one tile is in its softmax the tensor core works on the other.
//
// Where there are few pairs of row tiles they may be shared out (AttnPlan::share): each
// CTA works its part of all pairs' blocks, pieces of pairs at its ends leave their
// sums, maxima and O to a second kernel.  A piece starts with every barrier set up
// anew; warp 11 looks the next one up meanwhile.
//
// O is only rescaled when a row's maximum has grown by more than 2^8 since the
// scale in use was set; FP32 sums lose nothing by that.  bf16 weights are then 1 to
// 2^8 at the maximum.  fp16 weights carry a factor of 2^7 besides, all that fp16 has
// room for above 2^8: they keep 11 bits down to 2^-21 of the scale in use and end at
// 2^-32 of it, so that 2^17 keys can lose 2^-15 of a row's sum at most.  (A factor of
// 2^11 that leaves room for a growth of 2^4 rescales oftener: with scores of standard
// deviation 4, a prompt of 8192 tokens took 522 us for 490 in fp16, 2 x 2500 rows of 8
// heads of 64 over 12500 keys 154 for 147; with scores of 1 there is no difference.)
// At head_dim 128 P takes S's place in tensor memory, and the completion of
// S(j+1) also says that O += P V of block j is done, as they are issued in that
// order.  At 64 there is room for both, S(j+1) is made during block j's softmax,
// and O and P have a barrier of their own.
//
// What bounds it.  At head_dim 128 the products: a block pair (both tiles) is
// 2048 cycles of tensor core, but S takes both operands from shared memory, 8 KB
// for each 64 cycles, all that it gives beside the copies, so about 2500; 2850 to
// 2950 are measured, as the waits between the steps of a tile are not all covered
// by the other's.  At 64 the softmax warps: 2300 cycles of dependent instructions
// against 1024 of products and as many of exponentials.  A CTA's start and end
// take 7 us beside that, a piece of a share 10 (at 64: 5.5): its queries, the first
// keys, the masked block, O.
//
// Measured on a GB300 (2.0 GHz), 32 query and 8 key heads of 128, bf16: a prompt of
// 8192 tokens 380 to 400 us (1445 to 1375 TFLOP/s of 1900 measured; whole blocks make
// 1.6 % more products than are counted); six ragged chunks of up to 500 tokens over up
// to 12000 keys 258 to 269 us (1330 to 1270 TFLOP/s); 2500 tokens of 8 heads of 64 over 12500 keys in
// E4M3, two requests: 131 us (654 TFLOP/s; chunks of equal length instead of shares:
// 158).  Two threads a row gave no gain (they share the exponentials' unit: 471 us
// for the prompt against 473 at the time), nor did going on with other places of the
// grid in one CTA (423 against 417).
//
// A wait that runs out (it never should) ends the CTA: its rows become NaN and
// bevpool_attention_timeouts counts it.
#include <cuda.h>

#include "paged_attention.cuh"
#include "packed.cuh"
#include "tcgen05.cuh"

namespace bevpool {

__device__ unsigned long long g_attention_timeouts;

namespace {

constexpr int kBlock = 128;                // keys of a block
constexpr int kTileRows = 128;
// log2 of the weight of a row's maximum when its scale is set, and of the largest
// weight before it is set anew.
template <typename T>
constexpr float kLift = std::is_same<T, __half>::value ? 7.0f : 0.0f;
template <typename T>
constexpr float kMost = std::is_same<T, __half>::value ? 15.0f : 8.0f;

template <bool E4M3, int D>
struct TileShape {
    // Warpgroups: two of softmax, one of products and TMA, and with E4M3 codes
    // one of loaders.  Registers a thread, by setmaxnreg; their sum is within
    // what the launch gives (168 a thread of 384, 128 of 512).
    static constexpr int LOADERS = E4M3 ? 4 : 1;                           // warps
    static constexpr int THREADS = E4M3 ? 512 : 384;
    static constexpr int LAUNCH_REGS = E4M3 ? 128 : 168;
    static constexpr int SOFTMAX_REGS = E4M3 ? 184 : 208;
    static constexpr int PRODUCT_REGS = E4M3 ? 56 : 80;
    static constexpr int LOADER_REGS = 88;
    static_assert(256 * SOFTMAX_REGS + 128 * PRODUCT_REGS + (E4M3 ? 128 * LOADER_REGS : 0) <= THREADS * LAUNCH_REGS,
                  "the split is within the launch's registers");
    static_assert(SOFTMAX_REGS >= LAUNCH_REGS && PRODUCT_REGS <= LAUNCH_REGS && (!E4M3 || LOADER_REGS <= LAUNCH_REGS),
                  "softmax threads gain registers, the others lose some");
    // At head_dim 64 tensor memory has room for P beside S: the next block's S is
    // then made while this block is in its softmax.
    static constexpr bool AHEAD = D == 64;
    static constexpr int P_COL = AHEAD ? 2 * kBlock + 2 * D : 0;           // P's first column; tile t's are 64 t (128 t over S) on
    static constexpr int P_STEP = AHEAD ? kBlock / 2 : kBlock;
    static constexpr int HALVES = D / 64;                                  // 128-byte columns of a block
    static constexpr int BLOCK_BYTES = kBlock * D * 2;
    static constexpr int STAGES = D == 64 ? 8 : E4M3 ? 4 : 5;              // K and V blocks in turn
    static constexpr int RAW_BYTES = E4M3 ? 2 * kBlock * D : 0;            // two blocks of codes on their way
    static constexpr int Q_BYTES = kTileRows * D * 2;
    static constexpr int SMEM = 1024 + 2 * Q_BYTES + STAGES * BLOCK_BYTES + RAW_BYTES;     // 1024: alignment
};

// What a CTA does at a time: a pair of row tiles over the blocks [p0, p1).
struct TilePiece {
    int32_t b, hk, row0;                   // b < 0: none
    int32_t p0, p1;
    int32_t part;                          // first row of its partial results; below 0: it has all of the pair's blocks
};

// Shared tiles.  All pairs in order lie on one axis, each kStart units (what its
// start and end take, in blocks) and then its blocks; a CTA's share is [from, to).
struct TileWalk {
    int64_t from, to, total, at;           // at: where the next pair starts
    int32_t place, ctas;                   // the next pair; CTAs with a share
};
constexpr int32_t kStart = 4, kLeast = 6;  // kLeast: units of a share, at least

struct TileBars {                          // shared memory
    uint64_t full[8], empty[8];            // ring
    uint64_t q_full[2], s_full[2], p_full[2][2], s_read[2], o_full[2], turn[2], drain[2];
    uint32_t tmem, failed;
    TilePiece piece[2];                    // the one at work and the next
    TileWalk walk;
    int64_t scan[16];
};

// What a row tile sees of the blocks [p0, p1): [b0, b1).
struct TileRange {
    int32_t b0, b1;
};

__device__ __forceinline__ TileRange tile_range(const AttnArgs &a, const Request &r, int32_t row0, int32_t rows, int32_t p0,
                                                int32_t p1) {
    if (row0 >= rows) return {0, 0};
    int32_t lo, hi, x;
    seen_keys(a, r, row0 / a.G, &lo, &x);
    seen_keys(a, r, (min(row0 + kTileRows, rows) - 1) / a.G, &x, &hi);
    if (hi <= lo) return {0, 0};
    const int32_t b0 = max(lo / kBlock, p0), b1 = min((hi - 1) / kBlock + 1, p1);
    return b1 > b0 ? TileRange{b0, b1} : TileRange{0, 0};
}

// What either tile of a pair sees.
__device__ __forceinline__ TileRange pair_range(TileRange t0, TileRange t1) {
    return {t0.b1 == 0 ? t1.b0 : t1.b1 == 0 ? t0.b0 : min(t0.b0, t1.b0), max(t0.b1, t1.b1)};
}

// The pair at a place on the axis; its blocks, or {0, -kStart} where it has no rows.
__device__ __forceinline__ TileRange pair_at(const AttnArgs &a, const AttnPlan &pl, int32_t place, TilePiece *pc) {
    pc->row0 = place % pl.tiles * kPairRows;
    pc->hk = place / pl.tiles % a.Hk;
    pc->b = place / pl.tiles / a.Hk;
    const Request r = request_of(a, pc->b);
    const int32_t rows = r.q_rows * a.G;
    if (pc->row0 >= rows) return {0, -kStart};
    return pair_range(tile_range(a, r, pc->row0, rows, 0, INT32_MAX), tile_range(a, r, pc->row0 + kTileRows, rows, 0, INT32_MAX));
}

// This CTA's share, by all of its threads (two places each).
template <int THREADS>
__device__ __forceinline__ void find_share(const AttnArgs &a, const AttnPlan &pl, TileBars &bars) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t places = pl.tiles * a.Hk * a.pg.n_seqs;
    int64_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int32_t place = 2 * threadIdx.x + i;
        w[i] = 0;
        if (place < places) {
            TilePiece pc;
            const TileRange x = pair_at(a, pl, place, &pc);
            w[i] = kStart + x.b1 - x.b0;
        }
    }
    int64_t sum = w[0] + w[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t below = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += below;
    }
    if (lane == 31) bars.scan[warp] = sum;
    __syncthreads();
    int64_t at = sum - w[0] - w[1], total = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        if (i < warp) at += bars.scan[i];
        total += bars.scan[i];
    }
    const int64_t most = total / kLeast;
    const int32_t ctas = static_cast<int32_t>(most < 1 ? 1 : most < gridDim.x ? most : gridDim.x);
    const int32_t me = min(static_cast<int32_t>(blockIdx.x), ctas);
    const int64_t from = me * total / ctas, to = min(me + 1, ctas) * total / ctas;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (from < to && at <= from && from < at + w[i]) {
            bars.walk.at = at;
            bars.walk.place = 2 * threadIdx.x + i;
        }
        at += w[i];
    }
    if (threadIdx.x == 0) {
        bars.walk.from = from;
        bars.walk.to = to;
        bars.walk.total = total;
        bars.walk.ctas = ctas;
        if (from >= to) bars.walk.at = to;                                 // no share
    }
}

// The next piece of this CTA's share, by one thread.
__device__ __forceinline__ TilePiece next_piece(const AttnArgs &a, const AttnPlan &pl, TileWalk &walk) {
    TilePiece pc = {-1, 0, 0, 0, 0, -1};
    while (walk.at < walk.to) {
        const int32_t place = walk.place;
        const TileRange x = pair_at(a, pl, place, &pc);
        const int64_t at = walk.at, first = at + kStart;                   // of its first block
        const int32_t n = x.b1 - x.b0;
        // a request's later pairs have no rows either
        walk.place = n >= 0 ? place + 1 : place - place % pl.tiles + (pc.row0 == 0 ? pl.tiles * (a.Hk - pc.hk) : pl.tiles);
        if (n < 0) continue;
        walk.at = first + n;
        const int32_t from = static_cast<int32_t>(min(max(walk.from - first, static_cast<int64_t>(0)), static_cast<int64_t>(n)));
        const int32_t to = static_cast<int32_t>(min(max(walk.to - first, static_cast<int64_t>(0)), static_cast<int64_t>(n)));
        if (n == 0 ? at < walk.from : from >= to) continue;
        pc.p0 = x.b0 + from;
        pc.p1 = x.b0 + to;
        if (from > 0 || to < n) {
            pc.part = static_cast<int32_t>(blockIdx.x) * (2 * kPairRows);
            if (from == 0) {                                               // others end it
                pc.part += kPairRows;
                const int64_t last = ((first + n) * walk.ctas - 1) / walk.total;           // whose share its last block is in
                a.cut[place] = make_int2(blockIdx.x, static_cast<int32_t>(last));
            }
        } else {
            pc.part = -1;
            a.cut[place] = make_int2(-1, 0);
        }
        return pc;
    }
    pc.b = -1;
    return pc;
}

// Every barrier, set up; `again`: once more, with nothing left that arrives.
template <int STAGES, int FULL>
__device__ __forceinline__ void init_bars(TileBars &bars, bool again) {
    const auto init = [&](uint64_t *bar, uint32_t n) {
        if (again) bar_end(shared_addr(bar));
        bar_init(shared_addr(bar), n);
    };
    for (int i = 0; i < STAGES; ++i) {
        init(&bars.full[i], FULL);
        init(&bars.empty[i], 2);
    }
    for (int t = 0; t < 2; ++t) {
        init(&bars.q_full[t], kTileRows);
        init(&bars.s_full[t], 1);
        init(&bars.p_full[t][0], kTileRows);
        init(&bars.p_full[t][1], kTileRows);
        init(&bars.s_read[t], kTileRows);
        init(&bars.o_full[t], 1);
        init(&bars.turn[t], 1);
        init(&bars.drain[t], 1);
    }
    bar_init_fence();
}

enum { kSoftmax, kProducts, kLoads };

// A role's part of one piece; false where a wait ran out.
template <typename T, bool E4M3, int D, bool SHARED, int ROLE>
__device__ __forceinline__ bool attend_piece(const AttnArgs &a, const AttnPlan &pl, const CUtensorMap &k_map,
                                             const CUtensorMap &v_map, TileBars &bars, int piece, uint32_t smem) {
    using S = TileShape<E4M3, D>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const TilePiece pc = bars.piece[piece];
    const int hk = pc.hk, b = pc.b;
    const Request r = request_of(a, b);
    const int32_t rows = r.q_rows * a.G, row0 = pc.row0;
    const TileRange t0 = tile_range(a, r, row0, rows, pc.p0, pc.p1), t1 = tile_range(a, r, row0 + kTileRows, rows, pc.p0, pc.p1);
    const TileRange both = pair_range(t0, t1);
    const int32_t j0 = both.b0, j1 = both.b1;
    const int32_t *table = a.pg.block_table + static_cast<int64_t>(b) * a.pg.table_pages;
    const uint32_t q_smem = smem, ring = smem + 2 * S::Q_BYTES;
    const uint32_t tmem = bars.tmem;
    bool ok = true;

    if constexpr (ROLE == kSoftmax) {
        // ------------------------------------------------------------ softmax
        const int t = warp >> 2, tid = threadIdx.x & 127;
        const TileRange tr = t == 0 ? t0 : t1;
        const int32_t tile0 = row0 + t * kTileRows;
        const int32_t row = tile0 + tid, warp0 = tile0 + (warp & 3) * 32;  // this thread's row, the warp's first
        const bool used = row < rows;
        int32_t lo = 0, hi = INT32_MAX;                                    // a place past the last row sees all, and is not kept
        int64_t token = 0;
        int32_t h = 0;
        if (used) {
            const int32_t i = row / a.G;
            token = r.q0 + i;
            h = hk * a.G + row - i * a.G;
            seen_keys(a, r, i, &lo, &hi);
        }
        if (tr.b1 > tr.b0) {
            // The warp's 32 rows of queries, copied 16 bytes a lane; where a row
            // starts is known to its own lane.  (Through registers a prompt of 8192
            // tokens took 402 us for 388.)
            constexpr int CPR = D / 8, RPI = 32 / CPR, N = 32 / RPI;       // 16-byte pieces of a row; rows a load
            const int64_t at = token * a.q.token_stride + h * a.q.head_stride;
            const int c = lane % CPR;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int y = i * RPI + lane / CPR, x = (warp & 3) * 32 + y;
                const int64_t at_x = __shfl_sync(0xffffffffu, at, y);
                const bool on = warp0 + y < rows;
                const uint32_t d = q_smem + t * S::Q_BYTES + (c >> 3) * (kTileRows * 128) + x * 128 + (((c & 7) ^ (x & 7)) << 4);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d),
                             "l"(static_cast<const T *>(a.q.p) + (on ? at_x : 0) + c * 8), "r"(on ? 16 : 0)
                             : "memory");
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_shared_async();
            bar_arrive(shared_addr(&bars.q_full[t]));
        }
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_mem = tmem + lanes + t * kBlock, p_mem = tmem + lanes + S::P_COL + t * S::P_STEP, o_mem = tmem + lanes + 2 * kBlock + t * D;
        float m = -INFINITY;                                               // the scale in use (base 2)
        uint64_t sum = pair(0.0f, 0.0f);
        // Groups of 16 keys that lie on no page, one bit each; read a block ahead.
        auto holes_of = [&](int32_t j) {
            bool hole = false;
            if (lane < kBlock / 16) {
                const int32_t k = j * kBlock + lane * 16;
                if (k < r.kv_len) {
                    const int32_t p = table[k >> a.pg.page_shift];
                    hole = p < 0 || p >= a.pg.n_pages;
                }
            }
            return hole;
        };
        bool hole = tr.b1 > tr.b0 ? holes_of(tr.b0) : false;
        uint32_t phase = 0;
        for (int32_t j = tr.b0; j < tr.b1; ++j, phase ^= 1) {
            const uint32_t holes = __ballot_sync(0xffffffffu, hole);
            if (j + 1 < tr.b1) hole = holes_of(j + 1);
            ok = bar_wait(shared_addr(&bars.s_full[t]), phase);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            tmem_fence_after();
            uint32_t s[kBlock];
#pragma unroll
            for (int c = 0; c < kBlock; c += 32) tmem_ld32(s_mem + c, s + c);
            tmem_wait_ld();
            if constexpr (S::AHEAD) {                                      // S may be made again
                tmem_fence_before();
                bar_arrive(shared_addr(&bars.s_read[t]));
            }
            const int32_t k0 = j * kBlock;
            if (!__all_sync(0xffffffffu, holes == 0 && lo <= k0 && hi - kBlock >= k0)) {
                // seen keys of the block, 32 a word
#pragma unroll
                for (int w = 0; w < kBlock / 32; ++w) {
                    const int from = min(max(lo - k0 - 32 * w, 0), 32), to = min(max(hi - k0 - 32 * w, 0), 32);
                    uint32_t seen = static_cast<uint32_t>((1ull << to) - 1) & ~static_cast<uint32_t>((1ull << from) - 1);
                    if ((holes >> (2 * w)) & 1) seen &= 0xffff0000u;
                    if ((holes >> (2 * w)) & 2) seen &= 0x0000ffffu;
#pragma unroll
                    for (int c = 0; c < 32; ++c) s[32 * w + c] = (seen >> c) & 1 ? s[32 * w + c] : 0xff800000u;   // -inf
                }
            }
            // P of one half and its sum, at the scale m.
            const uint64_t scale2 = pair(a.scale_log2, a.scale_log2);
            auto weights = [&](int h, uint32_t *p) {
                const float base2 = m == -INFINITY ? 0.0f : -m;
                const uint64_t from2 = pair(base2, base2);
                uint64_t u = pair(0.0f, 0.0f), v = u;
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const int at = h * 64 + 2 * c;
                    float x, y;
                    unpair(fma2(pair(__uint_as_float(s[at]), __uint_as_float(s[at + 1])), scale2, from2), &x, &y);
                    x = pow2(x);
                    y = pow2(y);
                    if (c & 1)
                        v = add2(v, pair(x, y));
                    else
                        u = add2(u, pair(x, y));
                    p[c] = pack2<T>(x, y);
                }
                return add2(u, v);
            };
            // Each half is released by itself: its product with V runs during
            // the exponentials of the other.
            auto release = [&](int h, const uint32_t *p) {
#pragma unroll
                for (int g = 0; g < 4; ++g) tmem_st8(p_mem + h * 32 + g * 8, p + g * 8);
                tmem_wait_st();
                tmem_fence_before();
                bar_arrive(shared_addr(&bars.p_full[t][h]));
            };
            // The first half's weights are worked out at the scale in use while
            // the row's maximum is still being found (other units do that), and
            // again in the rare case that the maximum has outgrown the scale.
            uint32_t p[32];
            const uint32_t o_free = S::AHEAD ? bar_test(shared_addr(&bars.o_full[t]), phase ^ 1) : 0;
            uint64_t part = weights(0, p);
            float mx[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) mx[x] = __uint_as_float(s[x]);
#pragma unroll
            for (int c = 4; c < kBlock - 4; c += 8)
#pragma unroll
                for (int x = 0; x < 4; ++x) mx[x] = max3(mx[x], __uint_as_float(s[c + x]), __uint_as_float(s[c + 4 + x]));
#pragma unroll
            for (int x = 0; x < 4; ++x) mx[x] = fmaxf(mx[x], __uint_as_float(s[kBlock - 4 + x]));
            const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * a.scale_log2;
            // O and P are free once the last block's O += P V is done (where S and
            // P share their place, S says so)
            if (S::AHEAD && j > tr.b0) {
                if (!o_free) ok = bar_wait(shared_addr(&bars.o_full[t]), phase ^ 1);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                tmem_fence_after();
            }
            const bool grown = top > m + kMost<T> || (m == -INFINITY && top > m);
            if (__any_sync(0xffffffffu, grown)) {
                const float mn = grown ? top - kLift<T> : m;
                const float f = grown ? pow2(m - mn) : 1.0f;               // m = -inf: 0
                m = mn;
                if (j > tr.b0) {
                    sum = mul2(sum, pair(f, f));
#pragma unroll 1
                    for (int c = 0; c < D; c += 8) {                       // few registers: S is held beside
                        uint32_t o[8];
                        tmem_ld8(o_mem + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 8; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                        tmem_st8(o_mem + c, o);
                    }
                }
                part = weights(0, p);
            }
            release(0, p);
            sum = add2(sum, part);
            part = weights(1, p);
            release(1, p);
            sum = add2(sum, part);
        }
        float l, l1;
        unpair(sum, &l, &l1);
        l += l1;
        if (ok && tr.b1 > tr.b0) ok = bar_wait(shared_addr(&bars.o_full[t]), S::AHEAD ? phase ^ 1 : 0);
        if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
        } else {
            tmem_fence_after();
            const bool some = !(l == 0.0f);
            const float inv = some ? a.v_scale / l : 0.0f;
            const int64_t part = pc.part >= 0 ? pc.part + t * kTileRows + tid : -1;
            bool fine = l - l == 0.0f;
            // O leaves through shared memory (over the queries, read by now), so
            // that a warp's stores cover whole rows.
            const uint32_t stage = q_smem + t * S::Q_BYTES + (warp & 3) * 32 * (D * 2);
            if (part < 0) {
                constexpr int CPR = D / 8;                                 // 16-byte pieces of a row
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32] = {};
                    if (tr.b1 > tr.b0) {
                        tmem_ld32(o_mem + c, o);
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int x = 0; x < 32; x += 8) {
                        float f[8];
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            f[y] = some ? __uint_as_float(o[x + y]) * inv : 0.0f;
                            fine = fine && f[y] - f[y] == 0.0f;
                        }
                        const uint4 w = pack8<T>(f);
                        const uint32_t d = stage + lane * (D * 2) + ((((c + x) / 8) ^ (lane & 7)) << 4);
                        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(d), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w)
                                     : "memory");
                    }
                }
                __syncwarp();
                const int c = lane % CPR;
                const int64_t at = token * a.out.token_stride + h * a.out.head_stride;
#pragma unroll 4
                for (int x = lane / CPR; x < 32; x += 32 / CPR) {
                    uint4 w;
                    const uint32_t d = stage + x * (D * 2) + ((c ^ (x & 7)) << 4);
                    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(d)
                                 : "memory");
                    const int64_t at_x = __shfl_sync(0xffffffffu, at, x);
                    if (warp0 + x < rows) *reinterpret_cast<uint4 *>(static_cast<T *>(a.out.p) + at_x + c * 8) = w;
                }
                __syncwarp();
            } else if (tr.b1 > tr.b0) {
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(o_mem + c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int x = 0; x < 32; ++x) fine = fine && __uint_as_float(o[x]) - __uint_as_float(o[x]) == 0.0f;
                    // 64 bytes of a row at a time
                    const uint32_t d0 = stage + lane * 64;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(d0 + ((x ^ ((lane >> 1) & 3)) << 4)),
                                         "r"(o[half * 16 + 4 * x]), "r"(o[half * 16 + 4 * x + 1]),
                                         "r"(o[half * 16 + 4 * x + 2]), "r"(o[half * 16 + 4 * x + 3])
                                         : "memory");
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int x = i * 8 + lane / 4, y = lane & 3;
                            uint4 w;
                            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                         : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                                         : "r"(stage + x * 64 + ((y ^ ((x >> 1) & 3)) << 4))
                                         : "memory");
                            if (warp0 + x < rows)
                                *reinterpret_cast<uint4 *>(a.part_o + (part - lane + x) * D + c + half * 16 + y * 4) = w;
                        }
                        __syncwarp();
                    }
                }
            }
            if (used) {
                if (part >= 0)
                    *reinterpret_cast<float2 *>(a.part_ml + part * 2) = make_float2(m, l);
                else if (a.lse)
                    a.lse[token * a.Hq + h] = some ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
            }
            // An infinity or NaN may come from a key in the block that the row
            // does not see (its weight 0 times the value): such rows are taken
            // again element by element.
            uint32_t again = __ballot_sync(0xffffffffu, used && !fine);
            __syncwarp();
            while (again) {
                const int x = __ffs(again) - 1;
                again &= again - 1;
                const int32_t rr = tile0 + (warp & 3) * 32 + x;
                float acc[D / 32], m1, s1;
                redo_row<T, E4M3, D>(a, r, b, hk, rr / a.G, hk * a.G + rr % a.G, pc.p0 * kBlock,
                                     static_cast<int32_t>(min(pc.p1 * static_cast<int64_t>(kBlock), static_cast<int64_t>(r.kv_len))),
                                     &m1, &s1, acc);
                store_row<T, D / 32>(a, r, rr / a.G, hk * a.G + rr % a.G, part < 0 ? -1 : part - lane + x, m1, s1, acc);
            }
        }
    } else if (ROLE == kProducts && warp < 10) {
        // ------------------------------------------------------------ products
        // A warp a tile: while one waits the other's products run.
        const int t = warp - 8;
        const TileRange tr = t == 0 ? t0 : t1;
        constexpr int format = std::is_same<T, __half>::value ? 0 : 1;
        constexpr uint32_t s_desc = mma_desc(format, kBlock, false), o_desc = mma_desc(format, D, true);
        auto in = [&](int32_t j) { return j >= tr.b0 && j < tr.b1; };
        const uint32_t s_bar = shared_addr(&bars.s_full[t]), p_bar = shared_addr(&bars.p_full[t][0]);
        const uint32_t your_turn = shared_addr(&bars.turn[t ^ 1]);
        auto scores = [&](uint32_t k_smem, bool pass) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                if (pass && k == D / 16 - 3) bar_arrive(your_turn);
                const uint32_t off = (k >> 2) * (kBlock * 128) + (k & 3) * 32;
                mma_ss(tmem + t * kBlock, operand_desc(q_smem + t * S::Q_BYTES + off, 16, 1024),
                       operand_desc(k_smem + off, 16, 1024), s_desc, k > 0);
            }
            mma_commit(s_bar);
        };
        uint32_t at = 0, lap = 0;                                          // place in the ring and its phase
        auto next = [&]() {
            if (++at == S::STAGES) {
                at = 0;
                lap ^= 1;
            }
        };
        uint32_t p_phase = 0;
        // A wait that ran out ends the products, not the walk: both warps meet at
        // the tail's barrier.
        auto wait = [&](uint32_t bar, uint32_t parity) {
            if (ok) ok = bar_wait(bar, parity);
        };
        // The next two places of the ring (a block's V, the next one's K): asked
        // for before the waits that they are needed after.
        uint32_t here = 0, after = 0;
        auto ask_ring = [&]() {
            const uint32_t at1 = at + 1 == S::STAGES ? 0 : at + 1, lap1 = at + 1 == S::STAGES ? lap ^ 1 : lap;
            here = bar_test(shared_addr(&bars.full[at]), lap);
            after = bar_test(shared_addr(&bars.full[at1]), lap1);
        };
        // Every block's K and V are let go by both warps, used or not.
        if (j1 > j0) {
            if (tr.b1 > 0) wait(shared_addr(&bars.q_full[t]), 0);
            wait(shared_addr(&bars.full[at]), lap);
            if (ok && elect_one()) {
                if (in(j0)) scores(ring + at * S::BLOCK_BYTES, false);
                mma_commit(shared_addr(&bars.empty[at]));
            }
            __syncwarp();
            next();
        }
        // V's rows: groups of `high` (a page's, or a block's) of all of the head's
        // 64-element columns in turn, so that a page's V is one box.
        const int high = E4M3 || a.pg.page_size > kBlock ? kBlock : a.pg.page_size;
        auto v_row = [&](int row) {                                        // its first column's bytes
            return ((row & ~(high - 1)) * S::HALVES + (row & (high - 1))) * 128;
        };
        // Values past the request's last key are whatever the page holds: zeros in
        // their place (the weights there are 0, but 0 * NaN is not).
        auto clear_tail = [&](int32_t j, uint32_t v_smem) {
            if (E4M3 || (j + 1) * static_cast<int64_t>(kBlock) <= r.kv_len) return;
            if (t == 0 && ok) {
                const int dead = r.kv_len - j * kBlock;                    // first row to clear
                for (int x = dead * 8 + lane; x < kBlock * 8; x += 32)
#pragma unroll
                    for (int h = 0; h < S::HALVES; ++h)
                        asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(v_smem + v_row(x / 8) + h * (high * 128) +
                                                                                  (x & 7) * 16),
                                     "r"(0)
                                     : "memory");
                fence_shared_async();
            }
            asm volatile("bar.sync 1, 64;" ::: "memory");                  // both product warps
        };
        uint32_t v_off[kBlock / 16];
#pragma unroll
        for (int k = 0; k < kBlock / 16; ++k) v_off[k] = v_row(16 * k);
        // O += P V, half of the keys as soon as their weights are there.
        auto half_product = [&](int h, uint32_t v_smem, bool first) {
            tmem_fence_after();
            if (ok && elect_one()) {
#pragma unroll
                for (int k = h * (kBlock / 32); k < (h + 1) * (kBlock / 32); ++k)
                    mma_ts(tmem + 2 * kBlock + t * D, tmem + S::P_COL + t * S::P_STEP + k * 8,
                           operand_desc(v_smem + v_off[k], high * 128, 1024), o_desc, !(first && k == 0));
            }
            __syncwarp();
        };
        if constexpr (S::AHEAD) {
            uint32_t read_phase = 0;
            for (int32_t j = j0; j < j1; ++j) {
                const uint32_t v_at = at, v_lap = lap, v_smem = ring + at * S::BLOCK_BYTES, v_here = here;
                const bool now = in(j), then = j + 1 < j1;
                next();
                if (then) {                                                // the next block's S first
                    if (!after) wait(shared_addr(&bars.full[at]), lap);
                    if (now) {
                        wait(shared_addr(&bars.s_read[t]), read_phase);
                        read_phase ^= 1;
                    }
                    tmem_fence_after();
                    if (ok && elect_one()) {
                        if (in(j + 1)) scores(ring + at * S::BLOCK_BYTES, false);
                        mma_commit(shared_addr(&bars.empty[at]));
                    }
                    __syncwarp();
                    next();
                }
                if (!v_here) wait(shared_addr(&bars.full[v_at]), v_lap);
                clear_tail(j, v_smem);
                if (now) {
                    wait(p_bar, p_phase);
                    half_product(0, v_smem, j == tr.b0);
                    wait(p_bar + 8, p_phase);
                    half_product(1, v_smem, j == tr.b0);
                    p_phase ^= 1;
                }
                ask_ring();
                if (ok && elect_one()) {
                    if (now) mma_commit(shared_addr(&bars.o_full[t]));
                    mma_commit(shared_addr(&bars.empty[v_at]));
                }
                __syncwarp();
            }
        } else {
            // They take turns, a block's products of one tile after those of the
            // other, so that one tile is in its softmax while the other's products
            // run; left to themselves both tiles fell into step and the tensor core
            // idled in both softmaxes (8192-token prompt: 496 us against 473).
            // The turn passes before the last products are issued, as issuing
            // waits for the queue.
            const uint32_t my_turn = shared_addr(&bars.turn[t]);
            uint32_t turn_phase = 0;
            for (int32_t j = j0; j < j1; ++j) {
                if (!here) wait(shared_addr(&bars.full[at]), lap);
                const uint32_t v_at = at, v_smem = ring + at * S::BLOCK_BYTES;
                next();
                clear_tail(j, v_smem);
                const bool then = j + 1 < j1, now = in(j);
                if (then && !after) wait(shared_addr(&bars.full[at]), lap);
                if (now) wait(p_bar, p_phase);
                if (j > j0 || t == 1) {
                    wait(my_turn, turn_phase);
                    turn_phase ^= 1;
                }
                if (now) {
                    half_product(0, v_smem, j == tr.b0);
                    wait(p_bar + 8, p_phase);
                    half_product(1, v_smem, j == tr.b0);
                    p_phase ^= 1;
                }
                if (ok && elect_one()) {
                    mma_commit(shared_addr(&bars.empty[v_at]));
                    if (then && in(j + 1)) {
                        scores(ring + at * S::BLOCK_BYTES, true);
                    } else {
                        bar_arrive(your_turn);
                        if (now) mma_commit(shared_addr(&bars.o_full[t]));
                    }
                    if (then) mma_commit(shared_addr(&bars.empty[at]));
                }
                __syncwarp();
                if (then) next();
                ask_ring();
            }
        }
        // All products done before the CTA ends.
        if (elect_one()) mma_commit(shared_addr(&bars.drain[t]));
        __syncwarp();
        ok = bar_wait(shared_addr(&bars.drain[t]), 0) && ok;
    } else if (ROLE == kProducts && (E4M3 || warp == 11)) {
        if (SHARED && warp == 11 && lane == 0) bars.piece[piece ^ 1] = next_piece(a, pl, bars.walk);
    } else if constexpr (!E4M3) {
        // ------------------------------------------------------------ TMA
        const int per = a.pg.page_size < kBlock ? kBlock / a.pg.page_size : 1;         // pages of a block
        const int high = kBlock / per;                                                 // rows of a box
        const int boxes = per * S::HALVES;
        const int page_i = lane / S::HALVES, half = lane % S::HALVES;
        uint32_t at = 0, lap = 0;
        // Page of this lane's box in block j; n_pages (past the pool: the box
        // fills with zeros) where there is none.
        auto page_of = [&](int32_t j) {
            const int32_t k = j * kBlock + page_i * high;
            int32_t p = a.pg.n_pages;
            if (lane < boxes && j < j1 && k < r.kv_len) {
                const int32_t x = table[k >> a.pg.page_shift];
                if (x >= 0 && x < a.pg.n_pages) p = x;
            }
            return p;
        };
        int32_t page = page_of(j0);
        int issued = 0;
        for (int32_t j = j0; j < j1 && ok; ++j) {
            const int32_t now = page;
            page = page_of(j + 1);
            const int32_t slot = (j * kBlock + page_i * high) & (a.pg.page_size - 1);
            const int32_t v_now = __shfl_sync(0xffffffffu, now, lane * S::HALVES);   // V's boxes: a lane a page
            const int32_t v_slot = (j * kBlock + lane * high) & (a.pg.page_size - 1);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                ok = bar_wait(shared_addr(&bars.empty[at]), lap ^ 1);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                const uint32_t full = shared_addr(&bars.full[at]);
                if (lane == 0) bar_expect(full, S::BLOCK_BYTES);
                __syncwarp();
                const uint32_t dst = ring + at * S::BLOCK_BYTES;
                if (kv == 0 && lane < boxes)
                    tma_load_4d(dst + half * (kBlock * 128) + page_i * high * 128, &k_map, full, half * 64, slot, hk, now);
                if (kv == 1 && lane < per)
                    tma_load_5d(dst + lane * high * (S::HALVES * 128), &v_map, full, 0, v_slot, 0, hk, v_now);
                ++issued;
                if (++at == S::STAGES) {
                    at = 0;
                    lap ^= 1;
                }
            }
        }
        // All copies landed before the CTA ends, and every place let go of before
        // the barriers are set up anew.
        for (int i = 0; i < S::STAGES && i < issued; ++i) {
            if (at == 0) lap ^= 1;
            at = at == 0 ? S::STAGES - 1 : at - 1;
            ok = bar_wait(shared_addr(&bars.full[at]), lap) && ok;
            if (SHARED) ok = ok && bar_wait(shared_addr(&bars.empty[at]), lap);
        }
    } else {
        // ------------------------------------------------------------ E4M3 codes
        constexpr int CPR = D / 16;                                        // 16-byte pieces of a row of codes
        constexpr int RPI = S::LOADERS * 32 / CPR;                         // rows in one step of all loader warps
        constexpr int N = kBlock / RPI;
        const int tid = threadIdx.x - 12 * 32, c = tid % CPR, row_i = tid / CPR;
        uint32_t at = 0, lap = 0;
        // Codes arrive by asynchronous copies two blocks ahead, each thread's own
        // pieces at its own place, so that it needs no other to widen them.
        const uint32_t raw = ring + S::STAGES * S::BLOCK_BYTES + tid * 16;
        uint4 w[N];
        int32_t pages[N], ahead[N];                                        // of the rows that this thread loads
        auto look_up = [&](int32_t j, int32_t *p) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int32_t k = j * kBlock + i * RPI + row_i;
                p[i] = j < j1 && k < r.kv_len ? table[k >> a.pg.page_shift] : -1;
            }
        };
        auto fetch = [&](int32_t j, int kv) {
            const uint8_t *cache = static_cast<const uint8_t *>(kv ? a.v_cache : a.k_cache);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int32_t k = j * kBlock + i * RPI + row_i;
                const bool on = pages[i] >= 0 && pages[i] < a.pg.n_pages;                  // else zeros
                const int64_t at_i = on ? pages[i] * a.pg.page_stride + (k & (a.pg.page_size - 1)) * a.pg.slot_stride +
                                              hk * a.pg.head_stride + c * 16
                                        : 0;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(raw + kv * (kBlock * D) + i * (S::LOADERS * 512)),
                             "l"(cache + at_i), "r"(on ? 16 : 0)
                             : "memory");
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        auto take = [&](int kv) {                                          // the older of the two blocks on their way
            asm volatile("cp.async.wait_group 1;" ::: "memory");
#pragma unroll
            for (int i = 0; i < N; ++i)
                asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                             : "r"(raw + kv * (kBlock * D) + i * (S::LOADERS * 512))
                             : "memory");
        };
        auto store = [&](int kv) {
            const uint32_t dst = ring + at * S::BLOCK_BYTES + (c >> 2) * (kBlock * 128);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int row = i * RPI + row_i;
                const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                uint32_t x[8];
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    const uint32_t codes = (u[y >> 1] >> (16 * (y & 1))) & 0xffffu;
                    x[y] = widen2<T>(codes);
                }
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(
                                     dst + row * 128 + ((((c & 3) * 2 + y) ^ (row & 7)) << 4)),
                                 "r"(x[4 * y]), "r"(x[4 * y + 1]), "r"(x[4 * y + 2]), "r"(x[4 * y + 3])
                                 : "memory");
            }
        };
        if (j1 > j0) {
            look_up(j0, pages);
            fetch(j0, 0);
            fetch(j0, 1);
            look_up(j0 + 1, pages);
            look_up(j0 + 2, ahead);                                        // a block ahead, off the path of its loads
        }
        for (int32_t j = j0; j < j1 && ok; ++j) {
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                take(kv);
                ok = bar_wait(shared_addr(&bars.empty[at]), lap ^ 1);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                store(kv);
                fetch(j + 1, kv);                                          // in place of the codes just used; none past the last block
                fence_shared_async();
                bar_arrive(shared_addr(&bars.full[at]));
                if (++at == S::STAGES) {
                    at = 0;
                    lap ^= 1;
                }
            }
#pragma unroll
            for (int i = 0; i < N; ++i) pages[i] = ahead[i];
            look_up(j + 3, ahead);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        for (int i = 0; SHARED && i < S::STAGES && i < 2 * (j1 - j0) && ok; ++i) {     // every place let go of
            if (at == 0) lap ^= 1;
            at = at == 0 ? S::STAGES - 1 : at - 1;
            ok = bar_wait(shared_addr(&bars.empty[at]), lap);
        }
    }
    return ok;
}

// All threads of the CTA, each role in its own code.
__device__ __forceinline__ void sync_roles() {
    tmem_fence_before();
    asm volatile("bar.sync 0;" ::: "memory");
    tmem_fence_after();
}

// A role's part of all of the CTA's pieces; true where a wait ran out.
template <typename T, bool E4M3, int D, bool SHARED, int ROLE>
__device__ __forceinline__ bool attend_pieces(const AttnArgs &a, const AttnPlan &pl, const CUtensorMap &k_map,
                                              const CUtensorMap &v_map, TileBars &bars, uint32_t smem) {
    using S = TileShape<E4M3, D>;
    bool failed = false;
    for (int piece = 0; !SHARED || bars.piece[piece].b >= 0; piece ^= 1) {
        if (!SHARED || !failed) {
            const bool ok = attend_piece<T, E4M3, D, SHARED, ROLE>(a, pl, k_map, v_map, bars, piece, smem);
            if (!ok) bars.failed = 1;
        } else if (ROLE == kSoftmax && threadIdx.x == 0) {
            bars.piece[piece ^ 1] = next_piece(a, pl, bars.walk);
        }
        sync_roles();
        failed = bars.failed != 0;
        if (ROLE == kSoftmax && failed) {                                  // rows of NaN
            const TilePiece &pc = bars.piece[piece];
            const Request r = request_of(a, pc.b);
            const int32_t row = pc.row0 + static_cast<int32_t>(threadIdx.x);
            if (row < r.q_rows * a.G) {
                const int64_t token = r.q0 + row / a.G;
                const int32_t h = pc.hk * a.G + row % a.G;
                T *op = static_cast<T *>(a.out.p) + token * a.out.token_stride + h * a.out.head_stride;
                if (pc.part >= 0) {
                    *reinterpret_cast<float2 *>(a.part_ml + (pc.part + static_cast<int64_t>(threadIdx.x)) * 2) = make_float2(NAN, NAN);
                } else {
                    for (int c = 0; c < D; ++c) op[c] = static_cast<T>(NAN);
                    if (a.lse) a.lse[token * a.Hq + h] = NAN;
                }
            }
        }
        if (!SHARED) break;
        if (ROLE == kSoftmax && threadIdx.x == 0 && !failed) init_bars<S::STAGES, E4M3 ? S::LOADERS * 32 : 1>(bars, true);
        sync_roles();
    }
    return failed;
}

template <typename T, bool E4M3, int D, bool SHARED>
__global__ void __launch_bounds__(TileShape<E4M3, D>::THREADS, 1)
k_attend_tile(AttnArgs a, AttnPlan pl, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    using S = TileShape<E4M3, D>;
    extern __shared__ uint8_t raw_smem[];
    __shared__ TileBars bars;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t smem = (shared_addr(raw_smem) + 1023) & ~1023u;
    if (SHARED) {
        find_share<S::THREADS>(a, pl, bars);
    } else {
        // x: row tiles (the longest first) by key heads; y: chunks; z: requests.
        TilePiece pc = {static_cast<int32_t>(blockIdx.z), static_cast<int32_t>(blockIdx.x) % a.Hk,
                        (pl.tiles - 1 - static_cast<int32_t>(blockIdx.x) / a.Hk) * kPairRows, 0, INT32_MAX, -1};
        const Request r = request_of(a, pc.b);
        if (pc.row0 >= r.q_rows * a.G) return;
        if (pl.n_chunks > 1) {
            int32_t base;
            const int n = chunks_of(a, r, pl, &base), chunk = blockIdx.y;
            if (chunk >= n) return;
            pc.p0 = base / kBlock + chunk * (pl.chunk / kBlock);
            pc.p1 = pc.p0 + pl.chunk / kBlock;
            if (n > 1) pc.part = static_cast<int32_t>(part_row(a, pl, pc.b, pc.hk, chunk, pc.row0));
        }
        if (threadIdx.x == 0) bars.piece[0] = pc;
    }
    if (threadIdx.x == 0) {
        init_bars<S::STAGES, E4M3 ? S::LOADERS * 32 : 1>(bars, false);
        bars.failed = 0;
    }
    if (warp == 8) tmem_alloc<512>(shared_addr(&bars.tmem));
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (SHARED) {
        if (warp == 11 && lane == 0) bars.piece[0] = next_piece(a, pl, bars.walk);
        __syncthreads();
    }
    // Each role has its own registers, so its own loop.
    bool failed = false;
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::SOFTMAX_REGS));
        failed = attend_pieces<T, E4M3, D, SHARED, kSoftmax>(a, pl, k_map, v_map, bars, smem);
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::PRODUCT_REGS));
        failed = attend_pieces<T, E4M3, D, SHARED, kProducts>(a, pl, k_map, v_map, bars, smem);
    } else if constexpr (E4M3) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::LOADER_REGS));
        failed = attend_pieces<T, E4M3, D, SHARED, kLoads>(a, pl, k_map, v_map, bars, smem);
    }
    if (warp == 8) tmem_free<512>(bars.tmem);
    if (failed && threadIdx.x == 0) atomicAdd(&g_attention_timeouts, 1ull);
    grid_dep_allow();
}

// The driver's tensor-map encoder, found through the runtime.
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// A 16-bit cache as a tensor (element, slot, head, page) in boxes of 64 elements
// by the slots of a page that a block takes; for V the head's 64-element columns
// are an axis of their own, all of them in a box.  (K's columns have to lie a
// whole block apart, as one product takes all of its rows.)  Half as many boxes
// for V count with pages of 16 slots: six ragged chunks 304 us before, 260
// after.
bool cache_map(const AttnArgs &a, const void *cache, bool columns, CUtensorMap *map) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return false;
    const cuuint64_t slots = static_cast<cuuint64_t>(a.pg.page_size), heads = static_cast<cuuint64_t>(a.Hk),
                     pages = static_cast<cuuint64_t>(a.pg.n_pages);
    // the stride of an axis of one entry is never used
    const auto stride = [&](int64_t s, int64_t n) { return static_cast<cuuint64_t>(n > 1 ? s : a.D) * 2; };
    const cuuint64_t slot_s = stride(a.pg.slot_stride, a.pg.page_size), head_s = stride(a.pg.head_stride, a.Hk),
                     page_s = stride(a.pg.page_stride, a.pg.n_pages);
    const cuuint32_t high = static_cast<cuuint32_t>(a.pg.page_size < kBlock ? a.pg.page_size : kBlock);
    const cuuint32_t wide = static_cast<cuuint32_t>(a.D / 64);
    const cuuint64_t dims4[4] = {static_cast<cuuint64_t>(a.D), slots, heads, pages}, dims5[5] = {64, slots, wide, heads, pages};
    const cuuint64_t strides4[3] = {slot_s, head_s, page_s}, strides5[4] = {slot_s, 128, head_s, page_s};
    const cuuint32_t box4[4] = {64, high, 1, 1}, box5[5] = {64, high, wide, 1, 1}, ones[5] = {1, 1, 1, 1, 1};
    return encode(map, a.dtype == BEVPOOL_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                  columns ? 5 : 4, const_cast<void *>(cache), columns ? dims5 : dims4, columns ? strides5 : strides4,
                  columns ? box5 : box4, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t attention_timeouts(int64_t *count) {
    unsigned long long n = 0;
    cudaError_t e = cudaDeviceSynchronize();               // a copy alone leaves out streams that do not wait for the default one
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&n, g_attention_timeouts, sizeof(n));
    if (e == cudaSuccess) *count = static_cast<int64_t>(n);
    return e;
}

cudaError_t launch_attend_tile(const AttnArgs &a, const AttnPlan &pl) {
    CUtensorMap k_map = {}, v_map = {};
    if (!a.cache_e4m3 && (!cache_map(a, a.k_cache, false, &k_map) || !cache_map(a, a.v_cache, true, &v_map))) return cudaErrorInvalidValue;
    auto launch = [&](auto t, auto e4m3, auto d, auto shared, dim3 grid) {
        constexpr bool E = decltype(e4m3)::value, SHARED = decltype(shared)::value;
        constexpr int D = decltype(d)::value;
        using S = TileShape<E, D>;
        const cudaError_t e = allow_smem<&k_attend_tile<decltype(t), E, D, SHARED>>(S::SMEM);
        if (e != cudaSuccess) return e;
        k_attend_tile<decltype(t), E, D, SHARED><<<grid, S::THREADS, S::SMEM, a.stream>>>(a, pl, k_map, v_map);
        count_launch();
        return cudaGetLastError();
    };
    auto run = [&](auto t, auto e4m3, auto d) {
        if (pl.share) return launch(t, e4m3, d, std::true_type{}, dim3(static_cast<unsigned>(pl.share)));
        return launch(t, e4m3, d, std::false_type{},
                      dim3(static_cast<unsigned>(pl.tiles * a.Hk), static_cast<unsigned>(pl.n_chunks),
                           static_cast<unsigned>(a.pg.n_seqs)));
    };
    auto by_d = [&](auto t, auto e4m3) {
        return a.D == 64 ? run(t, e4m3, std::integral_constant<int, 64>{})
                         : run(t, e4m3, std::integral_constant<int, 128>{});
    };
    auto by_e = [&](auto t) { return a.cache_e4m3 ? by_d(t, std::true_type{}) : by_d(t, std::false_type{}); };
    return a.dtype == BEVPOOL_F16 ? by_e(__half{}) : by_e(__nv_bfloat16{});
}

}  // namespace bevpool
