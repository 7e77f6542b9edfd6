// paging.h -- arguments and launchers of the page plan and of the move of
// accepted tokens (page_plan.cu, kv_accept.cu).
#pragma once

#include "attn.h"

namespace moe {

struct PagePlanArgs {
    int32_t *ring;      // [cap] free page numbers, `count` of them from `head` on
    int cap;
    const int32_t *state;  // head, count
    int32_t *state_out;
    int32_t *table;
    int table_stride, page_shift;
    const int32_t *seq_lens, *new_lens, *dropped, *kept, *offsets;
    int window, sinks, B, rows;
    int32_t *seq_lens_out, *kept_out, *cu_q, *cu_k, *positions, *slots;
    uint8_t *workspace;
};
size_t page_plan_workspace(int B);
cudaError_t launch_page_plan(const PagePlanArgs &a, cudaStream_t s);

struct AcceptArgs {
    KvView kv;
    int cache_type, D;
    const int32_t *page_table;
    int table_stride;
    const int32_t *base, *accept;
    int B, P;
    Ctrl *ctrl;
};
cudaError_t launch_kv_accept(const AcceptArgs &a, cudaStream_t s);

}  // namespace moe
