// attn_api.cu -- the C ABI of the attention half: argument validation and
// launches.
#include <climits>
#include <cmath>
#include <cstdlib>

#include "attn.h"

using namespace moe;

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int log2_of(int v) {
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}

bool head_sizes_ok(int Hq, int Hkv, int D) {
    return (D == 64 || D == 128) && Hkv >= 1 && Hq >= Hkv && Hq <= 1024 && Hq % Hkv == 0;
}

bool cache_sizes_ok(int type, int num_pages, int page_size, int Hkv, int D) {
    return (type == MOE_KV_BF16 || type == MOE_KV_FP8) && num_pages >= 1 &&
           (page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128 ||
            page_size == 256) &&
           Hkv >= 1 && Hkv <= 1024 && (D == 64 || D == 128) &&
           (int64_t)num_pages * page_size * Hkv * 2 < INT_MAX;
}

// A cache descriptor that the kernels may use.
moe_status_t check_cache(const moe_kv_cache_t *c) {
    if (!c || !cache_sizes_ok(c->type, c->num_pages, c->page_size, c->Hkv, c->D) || !c->data)
        return MOE_ERR_INVALID_ARG;
    if ((c->type == MOE_KV_FP8) != (c->scales != nullptr)) return MOE_ERR_INVALID_ARG;
    if (!aligned(c->data, 16) || !aligned(c->scales, 16)) return MOE_ERR_MISALIGNED;
    return MOE_OK;
}

KvView view_of(const moe_kv_cache_t *c) {
    return {static_cast<const uint8_t *>(c->data), c->scales, c->num_pages, log2_of(c->page_size),
            c->Hkv};
}

// A stride between tokens of rows of `width` elements: no overlap, 16-byte steps.
bool stride_ok(int64_t stride, int64_t width) {
    return stride >= width && stride % 8 == 0 && stride < ((int64_t)1 << 31);
}

moe_status_t launched(cudaError_t e) {
    if (e == cudaSuccess) return MOE_OK;
    cudaGetLastError();
    return MOE_ERR_CUDA;
}

// Failure-path test switch, read once per process.
int test_no_copies() {
    static const int v = [] {
        const char *e = std::getenv("MOE_ATTN_TEST_NO_COPIES");
        return e && std::atoi(e) != 0 ? 1 : 0;
    }();
    return v;
}

cudaStream_t stream_of(moe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

extern "C" {

moe_status_t moe_kv_cache_size(int type, int num_pages, int page_size, int Hkv, int D,
                               size_t *data_bytes, size_t *scale_bytes) {
    if (data_bytes) *data_bytes = 0;
    if (scale_bytes) *scale_bytes = 0;
    if (!data_bytes || !scale_bytes || !cache_sizes_ok(type, num_pages, page_size, Hkv, D))
        return MOE_ERR_INVALID_ARG;
    const size_t rows = (size_t)num_pages * page_size * Hkv * 2;
    *data_bytes = rows * D * (type == MOE_KV_FP8 ? 1 : 2);
    *scale_bytes = type == MOE_KV_FP8 ? rows * 4 : 0;
    return MOE_OK;
}

moe_status_t moe_qk_rope_append(const uint16_t *q, int64_t q_stride, const uint16_t *k,
                                int64_t k_stride, const uint16_t *v, int64_t v_stride,
                                const uint16_t *q_norm, const uint16_t *k_norm, float eps,
                                const float *cos_sin, int max_pos, int rot, int interleaved,
                                const int32_t *positions, const int32_t *slots, uint16_t *q_out,
                                int64_t q_out_stride, uint16_t *k_out, int64_t k_out_stride,
                                const moe_kv_cache_t *cache, int T, int Hq, int Hkv, int D,
                                void *workspace, size_t ws_bytes, moe_stream_t stream) {
    if (!head_sizes_ok(Hq, Hkv, D) || T < 0 || (int64_t)T * (Hq + 2 * Hkv) >= INT_MAX ||
        rot < 0 || rot > D || rot % 16 || !(eps >= 0.f) || !std::isfinite(eps) || !workspace)
        return MOE_ERR_INVALID_ARG;
    if (rot > 0 && (max_pos < 1 || !cos_sin)) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!q || !k || !v || !q_out || (rot > 0 && !positions) || (cache && !slots)))
        return MOE_ERR_INVALID_ARG;
    if (!stride_ok(q_stride, (int64_t)Hq * D) || !stride_ok(q_out_stride, (int64_t)Hq * D) ||
        !stride_ok(k_stride, (int64_t)Hkv * D) || !stride_ok(v_stride, (int64_t)Hkv * D) ||
        (k_out && !stride_ok(k_out_stride, (int64_t)Hkv * D)))
        return MOE_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_norm, 16) ||
        !aligned(k_norm, 16) || !aligned(cos_sin, 16) || !aligned(positions, 4) ||
        !aligned(slots, 4) || !aligned(q_out, 16) || !aligned(k_out, 16) ||
        !aligned(workspace, 256))
        return MOE_ERR_MISALIGNED;
    if (cache) {
        const moe_status_t st = check_cache(cache);
        if (st != MOE_OK) return st;
        if (cache->Hkv != Hkv || cache->D != D) return MOE_ERR_INVALID_ARG;
    }
    if (ws_bytes < MOE_ATTN_STATUS_BYTES) return MOE_ERR_WORKSPACE_TOO_SMALL;
    const moe_status_t st = check_device();
    if (st != MOE_OK) return st;
    AppendArgs a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_norm = q_norm;
    a.k_norm = k_norm;
    a.eps = eps;
    a.cos_sin = cos_sin;
    a.max_pos = max_pos;
    a.rot = rot;
    a.interleaved = interleaved != 0;
    a.positions = positions;
    a.slots = slots;
    a.q_out = q_out;
    a.k_out = k_out;
    a.q_out_stride = q_out_stride;
    a.k_out_stride = k_out_stride;
    if (cache) {
        a.data = static_cast<uint8_t *>(cache->data);
        a.scales = cache->scales;
        a.cache_type = cache->type;
        a.num_pages = cache->num_pages;
        a.page_shift = log2_of(cache->page_size);
    }
    a.T = T;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = D;
    a.ctrl = static_cast<Ctrl *>(workspace);
    return launched(launch_append(a, stream_of(stream)));
}

moe_status_t moe_kv_gather(const moe_kv_cache_t *cache, const int32_t *page_table,
                           int table_stride, const int32_t *cu_k, int B, int Tk, uint16_t *k_out,
                           int64_t k_out_stride, uint16_t *v_out, int64_t v_out_stride,
                           void *workspace, size_t ws_bytes, moe_stream_t stream) {
    moe_status_t st = check_cache(cache);
    if (st != MOE_OK) return st;
    if (B < 0 || B > 65535 || Tk < 0 || Tk >= INT_MAX - 256 || table_stride < 0 || !cu_k ||
        !workspace || (Tk > 0 && (B == 0 || !page_table || table_stride == 0 || !k_out || !v_out)))
        return MOE_ERR_INVALID_ARG;
    const int64_t width = (int64_t)cache->Hkv * cache->D;
    if (!stride_ok(k_out_stride, width) || !stride_ok(v_out_stride, width))
        return MOE_ERR_INVALID_ARG;
    if (!aligned(page_table, 4) || !aligned(cu_k, 4) || !aligned(k_out, 16) ||
        !aligned(v_out, 16) || !aligned(workspace, 256))
        return MOE_ERR_MISALIGNED;
    if (ws_bytes < MOE_ATTN_STATUS_BYTES) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if ((st = check_device()) != MOE_OK) return st;
    const GatherKvArgs a = {view_of(cache), cache->type, cache->D,     page_table, table_stride,
                            cu_k,           B,           Tk,           k_out,      v_out,
                            k_out_stride,   v_out_stride, static_cast<Ctrl *>(workspace)};
    return launched(launch_kv_gather(a, stream_of(stream)));
}

size_t moe_attn_decode_workspace_size(int B, int Hq, int Hkv, int D) {
    if (B < 0 || B > 65535 || !head_sizes_ok(Hq, Hkv, D)) return 0;
    return decode_attn_workspace(B, Hq, Hkv, D);
}

moe_status_t moe_attn_decode(const uint16_t *q, int64_t q_stride, const moe_kv_cache_t *cache,
                             const int32_t *page_table, int table_stride, const int32_t *seq_lens,
                             float scale, uint16_t *out, int64_t out_stride, float *lse, int B,
                             int Hq, void *workspace, size_t ws_bytes, moe_stream_t stream) {
    moe_status_t st = check_cache(cache);
    if (st != MOE_OK) return st;
    const size_t need = moe_attn_decode_workspace_size(B, Hq, cache->Hkv, cache->D);
    if (need == 0 || !(scale > 0.f) || !std::isfinite(scale) || table_stride < 1 || !workspace ||
        (B > 0 && (!q || !page_table || !seq_lens || !out)))
        return MOE_ERR_INVALID_ARG;
    const int64_t width = (int64_t)Hq * cache->D;
    if (!stride_ok(q_stride, width) || !stride_ok(out_stride, width)) return MOE_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(page_table, 4) ||
        !aligned(seq_lens, 4) || !aligned(lse, 4) || !aligned(workspace, 256))
        return MOE_ERR_MISALIGNED;
    if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if ((st = check_device()) != MOE_OK) return st;
    if (B == 0) return launched(cudaMemsetAsync(workspace, 0, sizeof(Ctrl), stream_of(stream)));
    const DecodeAttnArgs a = {q,        q_stride, view_of(cache), cache->type, cache->D, page_table,
                              table_stride, seq_lens, scale, out, out_stride, lse, B, Hq,
                              static_cast<uint8_t *>(workspace), test_no_copies()};
    return launched(launch_attn_decode(a, stream_of(stream)));
}

size_t moe_attn_prefill_workspace_size(int B, int Tq, int Hq, int Hkv, int D) {
    if (B < 0 || B > 65535 || !head_sizes_ok(Hq, Hkv, D) || Tq < 0 || (int64_t)Tq * Hq >= INT_MAX)
        return 0;
    return prefill_workspace(B, Tq, Hq, Hkv, D);
}

moe_status_t moe_attn_prefill(const uint16_t *q, int64_t q_stride, const uint16_t *k,
                              int64_t k_stride, const uint16_t *v, int64_t v_stride,
                              const int32_t *cu_q, const int32_t *cu_k, int B, int Tq, int Tk,
                              int Hq, int Hkv, int D, int causal, float scale, uint16_t *out,
                              int64_t out_stride, float *lse, void *workspace, size_t ws_bytes,
                              moe_stream_t stream) {
    const size_t need = moe_attn_prefill_workspace_size(B, Tq, Hq, Hkv, D);
    if (need == 0 || Tk < 0 || Tk >= INT_MAX - 256 || !(scale > 0.f) || !std::isfinite(scale) || !workspace ||
        (B > 0 && (!cu_q || !cu_k)) || (Tq > 0 && B > 0 && (!q || !out)) ||
        (Tq > 0 && Tk > 0 && B > 0 && (!k || !v)))
        return MOE_ERR_INVALID_ARG;
    if (!stride_ok(q_stride, (int64_t)Hq * D) || !stride_ok(out_stride, (int64_t)Hq * D) ||
        !stride_ok(k_stride, (int64_t)Hkv * D) || !stride_ok(v_stride, (int64_t)Hkv * D))
        return MOE_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
        !aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(lse, 4) || !aligned(workspace, 256))
        return MOE_ERR_MISALIGNED;
    if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
    const moe_status_t st = check_device();
    if (st != MOE_OK) return st;
    if (Tq == 0 || B == 0)
        return launched(cudaMemsetAsync(workspace, 0, sizeof(Ctrl), stream_of(stream)));
    const PrefillArgs a = {q,  k,  v,  q_stride, k_stride, v_stride, cu_q,  cu_k, B,   Tq,
                           Tk, Hq, Hkv, D,       causal != 0, scale, out, out_stride, lse,
                           static_cast<uint8_t *>(workspace), test_no_copies()};
    return launched(launch_attn_prefill(a, stream_of(stream)));
}

}  // extern "C"
