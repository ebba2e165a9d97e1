// plan_pages.cuh -- arguments of the page plan.
#pragma once

#include "bevpool_internal.cuh"

namespace bevpool {

constexpr int32_t kMaxPlanSeqs = 16384;    // three sums a request fit the shared memory of a CTA

struct PlanArgs {
    const int32_t *q_len, *kv_len, *first, *drop;          // drop null: none
    const int32_t *block_table, *free_pages, *n_free;
    int32_t n_seqs, table_pages, n_pool, n_tokens, page_shift;
    int32_t *cu_q, *positions;
    int64_t *slots;
    int32_t *kv_len_out, *first_out, *block_table_out, *free_out, *n_free_out, *missing;
    cudaStream_t stream;
};
cudaError_t launch_plan_pages(const PlanArgs &a);

}  // namespace bevpool
