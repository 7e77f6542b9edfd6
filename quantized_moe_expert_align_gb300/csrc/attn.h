// attn.h -- arguments and launchers of the attention half of a decoder layer
// (rope_append.cu, attn_decode.cu, attn_prefill.cu).
#pragma once

#include <atomic>

#include <cuda.h>

#include "moe_attn.h"
#include "moe_internal.h"

namespace moe {

// Raises a kernel's dynamic shared memory limit, once per device (ordinals
// of 64 and more: at every call).
struct SmemOnce {
    std::atomic<uint64_t> done{0};
    cudaError_t set(const void *fn, size_t bytes) {
        int dev = 0;
        cudaError_t err = cudaGetDevice(&dev);
        if (err != cudaSuccess) return err;
        const uint64_t bit = dev < 64 ? 1ull << dev : 0;
        if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
        err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
        return err;
    }
};

// MOE_OK if the current device is an sm_103 GPU (api.cu).
moe_status_t check_device();

// Tiled tensor map of `rank` <= 5 dimensions (innermost first; strides in
// bytes, of dimensions 1 and up; unit element strides, out-of-range reads 0).
bool encode_tensor_map(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *ptr,
                       const uint64_t *dims, const uint64_t *strides, const uint32_t *box,
                       CUtensorMapSwizzle swizzle);

// A paged cache as the kernels see it.
struct KvView {
    const uint8_t *data;
    const float *scales;
    int num_pages, page_shift, Hkv;  // page_size = 1 << page_shift
};

struct AppendArgs {
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const uint16_t *q_norm, *k_norm;
    float eps;
    const float *cos_sin;
    int max_pos, rot, interleaved;
    const int32_t *positions, *slots;
    uint16_t *q_out, *k_out;
    int64_t q_out_stride, k_out_stride;
    uint8_t *data;   // cache; null: nothing is cached
    float *scales;
    int cache_type, num_pages, page_shift;
    int T, Hq, Hkv, D;
    Ctrl *ctrl;
};
cudaError_t launch_append(const AppendArgs &a, cudaStream_t s);

struct GatherKvArgs {
    KvView kv;
    int cache_type, D;
    const int32_t *page_table;
    int table_stride;
    const int32_t *cu_k;
    int B, Tk;
    uint16_t *k_out, *v_out;
    int64_t k_out_stride, v_out_stride;
    Ctrl *ctrl;
};
cudaError_t launch_kv_gather(const GatherKvArgs &a, cudaStream_t s);

struct DecodeAttnArgs {
    const uint16_t *q;
    int64_t q_stride;
    KvView kv;
    int cache_type, D;
    const int32_t *page_table;
    int table_stride;
    const int32_t *seq_lens;
    float scale;
    uint16_t *out;
    int64_t out_stride;
    float *lse;
    int B, Hq;
    uint8_t *workspace;
    int test_no_copies;  // failure-path test: the kernel issues no copies
};
size_t decode_attn_workspace(int B, int Hq, int Hkv, int D);
cudaError_t launch_attn_decode(const DecodeAttnArgs &a, cudaStream_t s);

struct PrefillArgs {
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const int32_t *cu_q, *cu_k;
    int B, Tq, Tk, Hq, Hkv, D, causal;
    float scale;
    uint16_t *out;
    int64_t out_stride;
    float *lse;
    uint8_t *workspace;
    int test_no_copies;  // failure-path test: the kernel issues no copies
};
size_t prefill_workspace(int B, int Tq, int Hq, int Hkv, int D);
cudaError_t launch_attn_prefill(const PrefillArgs &a, cudaStream_t s);

}  // namespace moe
