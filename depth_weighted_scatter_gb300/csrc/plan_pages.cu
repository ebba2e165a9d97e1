// plan_pages.cu -- a batch's pages and places from its lengths: pages given
// back and handed out, the new block tables, cu_q, positions and slots.
//
// One launch.  Every CTA works out the three sums over the requests (new tokens,
// pages wanted, pages given back) for itself, from L2 into shared memory, and then
// its part of the outputs; nothing is exchanged between CTAs, so nothing waits.
// (A sum by one CTA and a second kernel would be two launches of about the same
// length; a call is bound by its launch.)  The free pages are a stack whose top is
// handed out first; pages given back lie on top of it in the requests' order, so
// that a page taken from there is found by a search of the sums.
//
// Measured on a GB300, a call: 64 single tokens over up to 8192, 8.3 to 8.7 us (launch
// and call: its nine outputs are one allocation, 17 us with nine); 46000 tokens of four
// frames, 9.1 to 10.2; 4000 requests of up to 7 tokens over up to 2000, 14.3: the sums
// and then four lookups that wait for each other.  Two CTAs an SM: 19.8, as each works
// the sums out.
#include "plan_pages.cuh"

namespace bevpool {

namespace {

constexpr int kPlanThreads = 512, kPlanWarps = kPlanThreads / 32;
constexpr int kSegment = 256;                              // columns of a table that a warp takes at a time

struct Sums {                                              // of one request, or of those before it
    int64_t q, want, drop;
};

// What request b keeps and gets.
struct Change {
    int32_t q, old, pages, drop, kept, had, has;
    bool ends;
};

__device__ __forceinline__ int32_t pages_for(uint32_t tokens, int shift) {
    return static_cast<int32_t>((tokens >> shift) + ((tokens & ((1u << shift) - 1)) != 0 ? 1 : 0));
}

__device__ __forceinline__ Change change_of(const PlanArgs &a, int b) {
    Change c;
    c.q = max(a.q_len[b], 0);
    c.old = max(a.kv_len[b], 0);
    const int32_t d = a.drop ? a.drop[b] : 0;
    c.pages = pages_for(static_cast<uint32_t>(c.old), a.page_shift);
    c.ends = d < 0;
    c.drop = c.ends ? c.pages : min(d, c.pages);
    c.kept = static_cast<int32_t>(max(static_cast<int64_t>(c.old) - (static_cast<int64_t>(c.drop) << a.page_shift), static_cast<int64_t>(0)));
    c.had = c.pages - c.drop;
    c.has = pages_for(static_cast<uint32_t>(c.kept) + static_cast<uint32_t>(c.q), a.page_shift);
    return c;
}

// The position of the first token kept (an ended request starts anew).
__device__ __forceinline__ int32_t first_of(const PlanArgs &a, int b, const Change &c) {
    return c.ends ? 0 : static_cast<int32_t>(static_cast<uint32_t>(a.first[b]) + static_cast<uint32_t>(c.old - c.kept));
}

// The last of the n + 1 ascending sums that is not above x, at most n - 1.
__device__ __forceinline__ int find(const int32_t *sums, int n, int32_t x) {
    int lo = 0, hi = n;                                    // sums[lo] <= x < sums[hi], as far as is known
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads, 1)
k_plan_pages(PlanArgs a) {
    extern __shared__ int32_t smem[];                      // sums before each request, and all: cu, wants, drops
    __shared__ Sums warp_sums[kPlanWarps];
    __shared__ int misfit[kPlanWarps];
    const int B = a.n_seqs, W = a.table_pages, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t *cu = smem, *wants = cu + B + 1, *drops = wants + B + 1;

    // What each request adds, read in order; then the sums, a run of requests a thread.
    bool bad = false;
#pragma unroll 4
    for (int b = threadIdx.x; b < B; b += kPlanThreads) {
        const Change c = change_of(a, b);
        bad = bad || c.has > W || c.pages > W || c.q > a.n_tokens;
        cu[b] = c.q;
        wants[b] = c.has - c.had;
        drops[b] = c.drop;
    }
    __syncthreads();
    const int per = (B + kPlanThreads - 1) / kPlanThreads | 1;             // odd: lanes' runs start in different banks
    const int b0 = min(static_cast<int>(threadIdx.x) * per, B), b1 = min(b0 + per, B);
    Sums s = {0, 0, 0};
    for (int b = b0; b < b1; ++b) s.q += cu[b], s.want += wants[b], s.drop += drops[b];
    const Sums mine = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t q = __shfl_up_sync(0xffffffffu, s.q, o), w = __shfl_up_sync(0xffffffffu, s.want, o),
                      d = __shfl_up_sync(0xffffffffu, s.drop, o);
        if (lane >= o) s.q += q, s.want += w, s.drop += d;
    }
    if (lane == 31) warp_sums[warp] = s;
    const bool any_bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) misfit[warp] = any_bad;
    __syncthreads();
    Sums at = {s.q - mine.q, s.want - mine.want, s.drop - mine.drop}, all = {0, 0, 0};
    bool fits = true;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
        const Sums x = warp_sums[w];
        if (w < warp) at.q += x.q, at.want += x.want, at.drop += x.drop;
        all.q += x.q, all.want += x.want, all.drop += x.drop;
        fits = fits && !misfit[w];
    }
    const int32_t n_free = max(*a.n_free, 0);
    const int64_t top = n_free + all.drop;
    fits = fits && all.q <= a.n_tokens && top <= a.n_pool;
    const bool ok = fits && all.want <= top;
    if (ok) {                                              // the sums fit 32 bits then
        for (int b = b0; b < b1; ++b) {
            const int32_t q = cu[b], w = wants[b], d = drops[b];
            cu[b] = static_cast<int32_t>(at.q);
            wants[b] = static_cast<int32_t>(at.want);
            drops[b] = static_cast<int32_t>(at.drop);
            at.q += q, at.want += w, at.drop += d;
        }
        if (threadIdx.x == 0) {
            cu[B] = static_cast<int32_t>(all.q);
            wants[B] = static_cast<int32_t>(all.want);
            drops[B] = static_cast<int32_t>(all.drop);
        }
    }
    __syncthreads();

    // Page i from the bottom of the stack.
    const auto stacked = [&](int32_t i) {
        if (i < n_free) return a.free_pages[i];
        const int32_t x = i - n_free;
        const int b = find(drops, B, x);
        return a.block_table[static_cast<int64_t>(b) * W + x - drops[b]];
    };
    // Page `col` of request b after the change.
    const auto page_at = [&](int b, const Change &c, int32_t col) {
        if (col < c.had) return a.block_table[static_cast<int64_t>(b) * W + col + c.drop];
        return stacked(static_cast<int32_t>(top) - 1 - (wants[b] + col - c.had));
    };

    const int64_t thread = static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x, threads = static_cast<int64_t>(gridDim.x) * kPlanThreads;
    // tokens
    for (int64_t t = thread; t < a.n_tokens; t += threads) {
        int32_t position = 0;
        int64_t slot = -1;
        if (ok && t < cu[B]) {
            const int b = find(cu, B, static_cast<int32_t>(t));
            const Change c = change_of(a, b);
            const int32_t place = c.kept + static_cast<int32_t>(t) - cu[b];
            position = static_cast<int32_t>(static_cast<uint32_t>(first_of(a, b, c)) + static_cast<uint32_t>(place));
            slot = (static_cast<int64_t>(page_at(b, c, place >> a.page_shift)) << a.page_shift) + (place & ((1 << a.page_shift) - 1));
        }
        a.positions[t] = position;
        a.slots[t] = slot;
    }
    // tables, a segment of a row a warp
    const int segments = (W + kSegment - 1) / kSegment;
    const int64_t units = static_cast<int64_t>(B) * segments;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kPlanWarps + warp; u < units; u += static_cast<int64_t>(gridDim.x) * kPlanWarps) {
        const int b = static_cast<int>(u / segments), col0 = static_cast<int>(u % segments) * kSegment;
        const Change c = change_of(a, b);
        const int64_t row = static_cast<int64_t>(b) * W;
#pragma unroll 4
        for (int col = col0 + lane; col < min(col0 + kSegment, W); col += 32)
            a.block_table_out[row + col] = !ok ? a.block_table[row + col] : col < c.has ? page_at(b, c, col) : -1;
    }
    // the stack
    const int32_t left = ok ? static_cast<int32_t>(top - all.want) : min(n_free, a.n_pool);
#pragma unroll 4
    for (int64_t i = thread; i < a.n_pool; i += threads)
        a.free_out[i] = i < left ? (ok ? stacked(static_cast<int32_t>(i)) : a.free_pages[i]) : -1;
    // requests
    for (int64_t i = thread; i <= B; i += threads) {
        const int b = static_cast<int>(i);
        a.cu_q[b] = ok ? cu[b] : 0;
        if (b == B) break;
        const Change c = change_of(a, b);
        a.kv_len_out[b] = ok ? c.kept + c.q : c.old;
        a.first_out[b] = ok ? first_of(a, b, c) : a.first[b];
    }
    if (thread == 0) {
        *a.n_free_out = ok ? left : n_free;
        const int64_t lack = all.want - top;
        *a.missing = !fits ? -1 : lack <= 0 ? 0 : static_cast<int32_t>(lack < INT32_MAX ? lack : INT32_MAX);
    }
}

}  // namespace

cudaError_t launch_plan_pages(const PlanArgs &a) {
    const int smem = 3 * (a.n_seqs + 1) * static_cast<int>(sizeof(int32_t));
    const cudaError_t e = allow_smem<&k_plan_pages>(3 * (kMaxPlanSeqs + 1) * static_cast<int>(sizeof(int32_t)));
    if (e != cudaSuccess) return e;
    const int64_t work = a.n_tokens + static_cast<int64_t>(a.n_seqs) * (a.table_pages + 1) + a.n_pool;
    int64_t grid = div_up(work, kPlanThreads);
    if (grid > 152) grid = 152;
    k_plan_pages<<<static_cast<unsigned>(grid < 1 ? 1 : grid), kPlanThreads, smem, a.stream>>>(a);
    count_launch();
    return cudaGetLastError();
}

}  // namespace bevpool
