// attn_serve_api.cu -- the C ABI around the paged cache (moe_attn_serve.h):
// argument validation and launches.
#include "attn_check.h"
#include "moe_attn_serve.h"
#include "paging.h"

using namespace moe;

static_assert(MOE_TREE_TOKENS == kTreeTokens, "drafted tokens of a sequence");

extern "C" {

size_t moe_page_plan_workspace_size(int B) { return B < 0 || B > 65535 ? 0 : page_plan_workspace(B); }

moe_status_t moe_page_plan(int32_t *ring, int ring_size, const int32_t *state, int32_t *state_out,
                           int32_t *page_table, int table_stride, int page_size,
                           const int32_t *seq_lens, const int32_t *new_lens, const int32_t *dropped, const int32_t *kept,
                           const int32_t *offsets, int window, int sinks, int B, int rows,
                           int32_t *seq_lens_out, int32_t *kept_out, int32_t *cu_q, int32_t *cu_k,
                           int32_t *positions, int32_t *slots, void *workspace, size_t ws_bytes,
                           moe_stream_t stream) {
    const size_t need = moe_page_plan_workspace_size(B);
    if (need == 0 || !ring || ring_size < 1 || ring_size >= 1 << 30 || !state || !state_out || table_stride < 1 ||
        (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128 && page_size != 256) ||
        window < 0 || sinks < 0 || rows < 0 || rows >= INT_MAX - 256 || !cu_q || !workspace ||
        (rows > 0 && (!positions || !slots)) || (B > 0 && (!page_table || !seq_lens || !new_lens || !seq_lens_out)) ||
        (B > 0 && window > 0 && (!kept || !kept_out)))
        return MOE_ERR_INVALID_ARG;
    const void *words[] = {ring,    state,  state_out, page_table, seq_lens,  new_lens, dropped,
                           kept,    offsets, cu_q,     cu_k,       seq_lens_out, kept_out, positions, slots};
    for (const void *p : words)
        if (!aligned(p, 4)) return MOE_ERR_MISALIGNED;
    if (!aligned(workspace, 256)) return MOE_ERR_MISALIGNED;
    if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
    const moe_status_t st = check_device();
    if (st != MOE_OK) return st;
    const PagePlanArgs a = {ring,     ring_size, state,  state_out, page_table, table_stride, log2_of(page_size),
                            seq_lens, new_lens,  dropped, kept,     offsets,    window,       sinks, B,
                            rows,     seq_lens_out, kept_out, cu_q, cu_k,       positions,    slots,
                            static_cast<uint8_t *>(workspace)};
    return launched(launch_page_plan(a, stream_of(stream)));
}

moe_status_t moe_attn_decode_window(const uint16_t *q, int64_t q_stride, const moe_kv_cache_t *cache,
                                    const int32_t *page_table, int table_stride, const int32_t *seq_lens, int window,
                                    int sinks, float scale, uint16_t *out, int64_t out_stride, float *lse, int B,
                                    int Hq, void *workspace, size_t ws_bytes, moe_stream_t stream) {
    if (window < 1 || sinks < 0) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_decode(q, q_stride, cache, page_table, table_stride, seq_lens, scale, out,
                                         out_stride, lse, B, Hq, workspace, ws_bytes);
    if (st != MOE_OK) return st;
    if (B == 0) return launched(cudaMemsetAsync(workspace, 0, sizeof(Ctrl), stream_of(stream)));
    DecodeAttnArgs a = {q,        q_stride, view_of(cache), cache->type, cache->D, page_table,
                        table_stride, seq_lens, scale, out, out_stride, lse, B, Hq,
                        static_cast<uint8_t *>(workspace), test_no_copies(), window, sinks, 0, nullptr, nullptr, 0};
    return launched(launch_attn_decode_window(a, stream_of(stream)));
}

moe_status_t moe_attn_prefill_window(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                                     const uint16_t *v, int64_t v_stride, const int32_t *cu_q, const int32_t *cu_k,
                                     int B, int Tq, int Tk, int Hq, int Hkv, int D, int window, int sinks, float scale,
                                     uint16_t *out, int64_t out_stride, float *lse, void *workspace, size_t ws_bytes,
                                     moe_stream_t stream) {
    if (window < 1 || sinks < 0) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_prefill(q, q_stride, k, k_stride, v, v_stride, cu_q, cu_k, B, Tq, Tk, Hq, Hkv, D,
                                          scale, out, out_stride, lse, workspace, ws_bytes);
    if (st != MOE_OK) return st;
    if (Tq == 0 || B == 0) return launched(cudaMemsetAsync(workspace, 0, sizeof(Ctrl), stream_of(stream)));
    const PrefillArgs a = {q,  k,  v,  q_stride, k_stride, v_stride, cu_q, cu_k, B,   Tq,
                           Tk, Hq, Hkv, D,       1,        scale,    out,  out_stride, lse,
                           static_cast<uint8_t *>(workspace), test_no_copies(), window, sinks};
    return launched(launch_attn_prefill_window(a, stream_of(stream)));
}

size_t moe_attn_tree_workspace_size(int B, int T, int Hq, int Hkv, int D) {
    if (B < 0 || B > 65535 || !head_sizes_ok(Hq, Hkv, D) || T < 0 || (int64_t)T * Hq >= INT_MAX) return 0;
    return tree_workspace(B, T, Hq, Hkv, D);
}

moe_status_t moe_attn_tree(const uint16_t *q, int64_t q_stride, const moe_kv_cache_t *cache,
                           const int32_t *page_table, int table_stride, const int32_t *seq_lens, const int32_t *cu_q,
                           const uint64_t *tree, float scale, uint16_t *out, int64_t out_stride, float *lse, int B,
                           int T, int Hq, void *workspace, size_t ws_bytes, moe_stream_t stream) {
    moe_status_t st = check_cache(cache);
    if (st != MOE_OK) return st;
    const size_t need = moe_attn_tree_workspace_size(B, T, Hq, cache->Hkv, cache->D);
    if (need == 0 || !(scale > 0.f) || !std::isfinite(scale) || table_stride < 1 || !workspace ||
        (B > 0 && (!page_table || !seq_lens || !cu_q)) || (B > 0 && T > 0 && (!q || !tree || !out)))
        return MOE_ERR_INVALID_ARG;
    const int64_t width = (int64_t)Hq * cache->D;
    if (!stride_ok(q_stride, width) || !stride_ok(out_stride, width)) return MOE_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(page_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(cu_q, 4) || !aligned(tree, 8) || !aligned(lse, 4) || !aligned(workspace, 256))
        return MOE_ERR_MISALIGNED;
    if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if ((st = check_device()) != MOE_OK) return st;
    if (B == 0 || T == 0) return launched(cudaMemsetAsync(workspace, 0, sizeof(Ctrl), stream_of(stream)));
    const DecodeAttnArgs a = {q,        q_stride, view_of(cache), cache->type, cache->D, page_table,
                              table_stride, seq_lens, scale, out, out_stride, lse, B, Hq,
                              static_cast<uint8_t *>(workspace), test_no_copies(), 0, 0, 0, cu_q, tree, T};
    return launched(launch_attn_tree(a, stream_of(stream)));
}

moe_status_t moe_kv_accept(const moe_kv_cache_t *cache, const int32_t *page_table, int table_stride,
                           const int32_t *base, const int32_t *accept, int B, int P, void *workspace, size_t ws_bytes,
                           moe_stream_t stream) {
    moe_status_t st = check_cache(cache);
    if (st != MOE_OK) return st;
    if (B < 0 || B > 65535 || P < 0 || P > 64 || table_stride < 1 || !workspace ||
        (B > 0 && P > 0 && (!page_table || !base || !accept)))
        return MOE_ERR_INVALID_ARG;
    if (!aligned(page_table, 4) || !aligned(base, 4) || !aligned(accept, 4) || !aligned(workspace, 256))
        return MOE_ERR_MISALIGNED;
    if (ws_bytes < MOE_ATTN_STATUS_BYTES) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if ((st = check_device()) != MOE_OK) return st;
    if (B == 0 || P == 0) return launched(cudaMemsetAsync(workspace, 0, sizeof(Ctrl), stream_of(stream)));
    const AcceptArgs a = {view_of(cache), cache->type, cache->D, page_table, table_stride,
                          base,           accept,      B,        P,          static_cast<Ctrl *>(workspace)};
    return launched(launch_kv_accept(a, stream_of(stream)));
}

}  // extern "C"
