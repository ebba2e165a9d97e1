// paged_attention.cu -- attention of new tokens over the paged cache: how a
// call is laid out, and its launches.
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

// Keys from the first that a request's rows see, rounded down to kFewAlign, to the last.
int64_t keys_of(int32_t max_q_len, int32_t max_kv_len, int32_t window) {
    int64_t keys = max_kv_len;
    if (window > 0 && static_cast<int64_t>(window) + max_q_len + kFewAlign < keys)
        keys = static_cast<int64_t>(window) + max_q_len + kFewAlign;
    return keys < 1 ? 1 : keys;
}

// Whether a call's tile pairs are shared out among one CTA an SM, each with the
// same number of blocks, rather than a CTA each: where there are few of them a
// wave that is not full, or a long one in the last, costs more than the pieces
// that are cut (2 x 2500 rows of 8 heads of 64 over 12500 keys, 160 pairs: 158 us
// with chunks of equal length, 130 shared).  Not where all keys are few, and not
// where the pairs of a key head would read its keys at times so far apart that
// they have left L2 meanwhile: shared, they are keys * pairs a head / 152 apart,
// over all heads; a CTA each, they walk together (six chunks of up to 500 tokens
// over 226 MB of cache, 71 MB apart: 1.2 GB from DRAM and 300 us shared, 260 us
// not).  With SMs to spare that counts for less.
int32_t tile_share(int64_t tiles, int64_t heads, int64_t keys, int64_t D) {
    constexpr int64_t kApart = 48 << 20;
    if (tiles >= 4 * kSms || keys < 1024) return 0;
    const int64_t cache = heads * keys * D * 4;                            // of 16 bits, at most
    const bool near = tiles <= heads || cache / kSms * heads <= kApart;
    return near || tiles <= kSms * 3 / 4 ? kSms : 0;
}

}  // namespace

AttnPlan attention_plan(const AttnSizes &z) {
    AttnPlan pl = {};
    const int32_t q_len = z.max_q_len < z.T ? z.max_q_len : z.T;
    pl.rows = q_len * (z.Hq / z.Hk);
    pl.few = pl.rows <= 16;
    const int64_t keys = keys_of(q_len, z.max_kv_len, z.window), pairs = static_cast<int64_t>(z.n_seqs) * z.Hk;
    pl.n_chunks = 1;
    if (pl.few) {
        const int64_t n = pairs > 0 ? (few_ctas(keys, pairs, z.n_seqs, z.D) + pairs / 2) / pairs : 1;
        int64_t chunk = div_up(div_up(keys, n < 1 ? 1 : n), kFewAlign) * kFewAlign;
        if (chunk > keys) chunk = div_up(keys, kFewAlign) * kFewAlign;
        pl.chunk = static_cast<int32_t>(chunk);
        pl.n_chunks = static_cast<int32_t>(div_up(keys, chunk));
    } else {
        pl.tiles = static_cast<int32_t>(div_up(pl.rows, kPairRows));
        pl.share = tile_share(pl.tiles * pairs, pairs, keys, z.D);
    }
    if (pl.n_chunks > 1) pl.parts = static_cast<int64_t>(z.n_seqs) * z.Hk * pl.n_chunks * pl.rows;
    if (pl.share) pl.parts = static_cast<int64_t>(pl.share) * 2 * kPairRows;
    return pl;
}

size_t attention_workspace_bytes(const AttnSizes &z) {
    const AttnPlan pl = attention_plan(z);
    return static_cast<size_t>(pl.parts) * (z.D + 2) * sizeof(float) + static_cast<size_t>(pl.share) * sizeof(int2);
}

cudaError_t launch_paged_attention(const AttnArgs &args, void *workspace) {
    AttnArgs a = args;
    const AttnPlan pl = attention_plan({a.pg.n_seqs, a.T, a.Hq, a.Hk, a.D, a.max_q_len, a.max_kv_len, a.window});
    a.part_o = static_cast<float *>(workspace);
    a.part_ml = a.part_o + pl.parts * a.D;
    a.cut = reinterpret_cast<int2 *>(a.part_ml + pl.parts * 2);
    const cudaError_t e = pl.few ? launch_attend_few(a, pl) : launch_attend_tile(a, pl);
    if (e != cudaSuccess || pl.parts == 0) return e;
    return launch_attend_join(a, pl);
}

}  // namespace bevpool
