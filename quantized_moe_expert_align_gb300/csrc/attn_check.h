// attn_check.h -- checks of arguments shared by the entry points of the
// attention half (attn_api.cu, attn_serve_api.cu).
#pragma once

#include <climits>
#include <cmath>
#include <cstdlib>

#include "attn.h"

namespace moe {
namespace {

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int log2_of(int v) {
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}

inline bool head_sizes_ok(int Hq, int Hkv, int D) {
    return (D == 64 || D == 128) && Hkv >= 1 && Hq >= Hkv && Hq <= 1024 && Hq % Hkv == 0;
}

inline bool cache_sizes_ok(int type, int num_pages, int page_size, int Hkv, int D) {
    return (type == MOE_KV_BF16 || type == MOE_KV_FP8) && num_pages >= 1 &&
           (page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128 ||
            page_size == 256) &&
           Hkv >= 1 && Hkv <= 1024 && (D == 64 || D == 128) &&
           (int64_t)num_pages * page_size * Hkv * 2 < INT_MAX;
}

// A cache descriptor that the kernels may use.
inline moe_status_t check_cache(const moe_kv_cache_t *c) {
    if (!c || !cache_sizes_ok(c->type, c->num_pages, c->page_size, c->Hkv, c->D) || !c->data)
        return MOE_ERR_INVALID_ARG;
    if ((c->type == MOE_KV_FP8) != (c->scales != nullptr)) return MOE_ERR_INVALID_ARG;
    if (!aligned(c->data, 16) || !aligned(c->scales, 16)) return MOE_ERR_MISALIGNED;
    return MOE_OK;
}

inline KvView view_of(const moe_kv_cache_t *c) {
    return {static_cast<const uint8_t *>(c->data), c->scales, c->num_pages, log2_of(c->page_size),
            c->Hkv};
}

// A stride between tokens of rows of `width` elements: no overlap, 16-byte steps.
inline bool stride_ok(int64_t stride, int64_t width) {
    return stride >= width && stride % 8 == 0 && stride < ((int64_t)1 << 31);
}

inline moe_status_t launched(cudaError_t e) {
    if (e == cudaSuccess) return MOE_OK;
    cudaGetLastError();
    return MOE_ERR_CUDA;
}

// Failure-path test switch, read once per process.
inline int test_no_copies() {
    static const int v = [] {
        const char *e = std::getenv("MOE_ATTN_TEST_NO_COPIES");
        return e && std::atoi(e) != 0 ? 1 : 0;
    }();
    return v;
}

inline cudaStream_t stream_of(moe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }


// The arguments of attention of single tokens.
inline moe_status_t check_decode(const uint16_t *q, int64_t q_stride, const moe_kv_cache_t *cache,
                                 const int32_t *page_table, int table_stride, const int32_t *seq_lens, float scale,
                                 const uint16_t *out, int64_t out_stride, const float *lse, int B, int Hq,
                                 const void *workspace, size_t ws_bytes) {
    moe_status_t st = check_cache(cache);
    if (st != MOE_OK) return st;
    const size_t need = moe_attn_decode_workspace_size(B, Hq, cache->Hkv, cache->D);
    if (need == 0 || !(scale > 0.f) || !std::isfinite(scale) || table_stride < 1 || !workspace ||
        (B > 0 && (!q || !page_table || !seq_lens || !out)))
        return MOE_ERR_INVALID_ARG;
    const int64_t width = (int64_t)Hq * cache->D;
    if (!stride_ok(q_stride, width) || !stride_ok(out_stride, width)) return MOE_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(page_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(lse, 4) || !aligned(workspace, 256))
        return MOE_ERR_MISALIGNED;
    if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
    return check_device();
}

// The arguments of attention over packed prompts.
inline moe_status_t check_prefill(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                                  const uint16_t *v, int64_t v_stride, const int32_t *cu_q, const int32_t *cu_k, int B,
                                  int Tq, int Tk, int Hq, int Hkv, int D, float scale, const uint16_t *out,
                                  int64_t out_stride, const float *lse, const void *workspace, size_t ws_bytes) {
    const size_t need = moe_attn_prefill_workspace_size(B, Tq, Hq, Hkv, D);
    if (need == 0 || Tk < 0 || Tk >= INT_MAX - 256 || !(scale > 0.f) || !std::isfinite(scale) || !workspace ||
        (B > 0 && (!cu_q || !cu_k)) || (Tq > 0 && B > 0 && (!q || !out)) ||
        (Tq > 0 && Tk > 0 && B > 0 && (!k || !v)))
        return MOE_ERR_INVALID_ARG;
    if (!stride_ok(q_stride, (int64_t)Hq * D) || !stride_ok(out_stride, (int64_t)Hq * D) ||
        !stride_ok(k_stride, (int64_t)Hkv * D) || !stride_ok(v_stride, (int64_t)Hkv * D))
        return MOE_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(cu_q, 4) ||
        !aligned(cu_k, 4) || !aligned(lse, 4) || !aligned(workspace, 256))
        return MOE_ERR_MISALIGNED;
    if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
    return check_device();
}

}  // namespace
}  // namespace moe
