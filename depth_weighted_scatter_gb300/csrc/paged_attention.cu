// paged_attention.cu -- attention of new tokens over the paged cache: how a
// call is laid out, and its launches.
#include <algorithm>
#include <cmath>

#include "paged_attention.cuh"

namespace bevpool {

namespace {

// CTAs that a few-rows call's chunks make of its longest requests.  An SM holds
// two, so a multiple w of 304: each wave costs its start, about 4 us, while w
// waves leave about 1 / (2 w) of the time t of the read to ragged lengths, so w
// is near sqrt(t / 8 us); a lone request is not ragged.  Measured with w = 1 /
// 2 / 4 / 8: one request of 40000 keys (8 key heads of 128, bf16) - / 41 / 49 /
// 55 us, 64 of up to 8192 - / 248 / 240 / 236 us.
int64_t few_ctas(int64_t keys, int64_t pairs, int32_t n_seqs, int32_t D) {
    if (n_seqs == 1) return 152 * 2;
    const double t = static_cast<double>(keys) * static_cast<double>(pairs) * D * 4 / 6.7e6;      // us, 16-bit cache
    const int64_t w = static_cast<int64_t>(std::sqrt(t / 8) + 0.5);
    return 152 * 2 * (w < 1 ? 1 : w > 6 ? 6 : w);
}

constexpr int32_t kSms = 152;

// What the plan of the few-rows kernel cuts keys by, and of the tiled one.
constexpr int32_t kFewAlign = 64, kTileAlign = 128;

// Most chunks that a tiled call is cut into.
constexpr int64_t kTileChunks = 32;

// Keys of a CTA's share of a tiled call, at least.
constexpr int64_t kLeastShare = 6 * 128;

// Keys from the first that a request's rows see, rounded down to align, to the last.
int64_t keys_of(int32_t max_q_len, int32_t max_kv_len, int32_t window, int32_t align) {
    int64_t keys = max_kv_len;
    if (window > 0 && static_cast<int64_t>(window) + max_q_len + align < keys)
        keys = static_cast<int64_t>(window) + max_q_len + align;
    return keys < 1 ? 1 : keys;
}

// Few CTAs (less than the GPU's SMs) leave SMs idle, so the keys are cut then:
// the cost of n chunks is its waves of CTAs times the keys of one plus what a
// CTA costs besides, in keys (its start, and its partial results).  Four waves
// are even enough uncut.
//
// Waves that are not full, or a last one as long as the others, can cost more
// than that, so the pairs' blocks may be shared out evenly among one CTA an SM
// instead (2 x 2500 rows of 8 heads of 64 over 12500 keys, 160 pairs: 158 us in
// three chunks, 131 shared): each CTA then has pieces of two pairs and a pair's
// share of whole ones.  Not where the pairs of a key head would read its keys at
// times so far apart that they have left L2 meanwhile: shared, keys * pairs a
// head / 152 of them lie between, over all heads; chunks walk together (six
// chunks of up to 500 tokens over 226 MB of cache, 71 MB apart: 1.2 GB from DRAM
// and 300 us shared, 258 us as one chunk).  A pair starts at 700 keys, a CTA at
// 1500 and the join besides: 2 x 1000 tokens of 8 heads of 64 over 8000 keys are
// 62.5 us in two chunks, 51.2 shared; 64 tokens over 20000 keys 18.7 in 32, 24.8
// shared, as a share is not less than kLeastShare.  Not for a causal prompt either:
// its tiles are not alike, and with the longest first no wave is left half full
// (4096 tokens: 144 us shared, 118 not; 5000 that all see each other, 8 heads of
// 64: 83 shared, 108 not).
int64_t tile_chunks(int64_t tiles, int64_t heads, int64_t keys, int64_t D, bool alike, bool *share) {
    *share = false;
    if (tiles >= 4 * kSms) return 1;
    int64_t best = 1, least = div_up(tiles, kSms) * (keys + 512);
    for (int64_t n = 2; n <= kTileChunks && n * 512 <= keys; ++n) {
        const int64_t cost = div_up(tiles * n, kSms) * (div_up(keys, n) + 1200);
        if (cost < least) {
            least = cost;
            best = n;
        }
    }
    constexpr int64_t kApart = 48 << 20;
    const int64_t cache = heads * keys * D * 4;                            // of 16 bits, at most
    if (alike && (tiles <= heads || cache / kSms * heads <= kApart))
        *share = std::max(tiles * (keys + 700) / kSms, kLeastShare) + 1500 < least;
    return *share ? 1 : best;
}

}  // namespace

AttnPlan attention_plan(const AttnSizes &z) {
    AttnPlan pl = {};
    const int32_t q_len = z.max_q_len < z.T ? z.max_q_len : z.T;
    pl.rows = q_len * (z.Hq / z.Hk);
    pl.few = pl.rows <= 16;
    pl.align = pl.few ? kFewAlign : kTileAlign;
    const int64_t keys = keys_of(q_len, z.max_kv_len, z.window, pl.align), pairs = static_cast<int64_t>(z.n_seqs) * z.Hk;
    int64_t n = 1;
    if (pl.few) {
        if (pairs > 0) n = (few_ctas(keys, pairs, z.n_seqs, z.D) + pairs / 2) / pairs;
    } else {
        bool share;
        pl.tiles = static_cast<int32_t>(div_up(pl.rows, kPairRows));
        n = tile_chunks(pl.tiles * pairs, pairs, keys, z.D, !z.causal || 2 * static_cast<int64_t>(q_len) <= keys, &share);
        if (share) pl.share = kSms;
    }
    int64_t chunk = div_up(div_up(keys, n < 1 ? 1 : n), pl.align) * pl.align;
    if (chunk > keys) chunk = div_up(keys, pl.align) * pl.align;
    pl.chunk = static_cast<int32_t>(chunk);
    pl.n_chunks = static_cast<int32_t>(div_up(keys, chunk));
    if (pl.n_chunks > 1) pl.parts = static_cast<int64_t>(z.n_seqs) * z.Hk * pl.n_chunks * pl.rows;
    if (pl.share) pl.parts = static_cast<int64_t>(pl.share) * 2 * kPairRows;
    return pl;
}

size_t attention_workspace_bytes(AttnSizes z) {
    size_t most = 0;
    for (z.causal = 0; z.causal < 2; ++z.causal) {
        const AttnPlan pl = attention_plan(z);
        const size_t cuts = pl.share ? static_cast<size_t>(pl.tiles) * z.Hk * z.n_seqs : 0;
        most = std::max(most, static_cast<size_t>(pl.parts) * (z.D + 2) * sizeof(float) + cuts * sizeof(int2));
    }
    return most;
}

cudaError_t launch_paged_attention(const AttnArgs &args, void *workspace) {
    AttnArgs a = args;
    const AttnPlan pl = attention_plan({a.pg.n_seqs, a.T, a.Hq, a.Hk, a.D, a.max_q_len, a.max_kv_len, a.window, a.causal});
    a.part_o = static_cast<float *>(workspace);
    a.part_ml = a.part_o + pl.parts * a.D;
    a.cut = reinterpret_cast<int2 *>(a.part_ml + pl.parts * 2);
    const cudaError_t e = pl.few ? launch_attend_few(a, pl) : launch_attend_tile(a, pl);
    if (e != cudaSuccess || pl.parts == 0) return e;
    return launch_attend_join(a, pl);
}

}  // namespace bevpool
