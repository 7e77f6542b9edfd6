// attn_simple.cu -- attention, one warp per (query row, query head): the
// keys of the row in ascending order with a running maximum and sum.
#include <cmath>

#include "attn.h"
#include "device_common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;

// E = D / 32 values a lane; load(j, kv, x) brings this lane's values of key /
// value row j.
template <int E, class Load>
__device__ __forceinline__ void attend(const float (&q)[E], int n, const Load &load, float (&o)[E],
                                       float &lse) {
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = 0.f;
    for (int j = 0; j < n; ++j) {
        float k[E], v[E];
        load(j, 0, k);
        load(j, 1, v);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
        for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        const float mn = fmaxf(m, s);
        const float base = mn == -INFINITY ? 0.f : mn;
        const float alpha = expf(m - base), p = expf(s - base);
        l = l * alpha + p;
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = o[i] * alpha + p * v[i];
        m = mn;
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] *= inv;
    lse = l == 0.f ? -INFINITY : m + logf(l);
}

template <int D>
__global__ void prefill_simple(PrefillArgs a) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    Ctrl *ctrl = reinterpret_cast<Ctrl *>(a.workspace);
    auto seq_ok = [&](int b) {
        const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
        return q0 >= 0 && q1 >= q0 && q1 <= a.Tq && k0 >= 0 && k1 >= k0 && k1 <= a.Tk;
    };
    if (blockIdx.x == 0) {
        if (threadIdx.x >= 32) return;
        int bad = 0x7fffffff;
        for (int b = lane; b < a.B; b += 32)
            if (!seq_ok(b) && b < bad) bad = b;
        bad = __reduce_min_sync(0xffffffffu, bad);
        if (lane == 0) {
            ctrl->status = bad == 0x7fffffff ? MOE_OK : MOE_ERR_DEVICE_BAD_INDEX;
            ctrl->detail = bad == 0x7fffffff ? 0 : bad;
        }
        return;
    }
    const int64_t row = (int64_t)(blockIdx.x - 1) * kWarps + (threadIdx.x >> 5);
    if (row >= (int64_t)a.Tq * a.Hq) return;
    const int t = (int)(row / a.Hq), h = (int)(row % a.Hq), hk = h / (a.Hq / a.Hkv);
    int b = 0;
    while (b < a.B && !(seq_ok(b) && a.cu_q[b] <= t && t < a.cu_q[b + 1])) ++b;
    if (b == a.B) return;
    const int nq = a.cu_q[b + 1] - a.cu_q[b], k0 = a.cu_k[b], nk = a.cu_k[b + 1] - k0;
    int n = nk;
    if (a.causal) n = min(nk, max(0, t - a.cu_q[b] + nk - nq + 1));
    float q[E], o[E], lse;
    for (int i = 0; i < E; ++i)
        q[i] = bf16_bits_to_float(a.q[t * a.q_stride + h * D + lane * E + i]) * a.scale;
    attend<E>(q, n, [&](int j, int kv, float (&x)[E]) {
        const uint16_t *r = kv ? a.v + (k0 + j) * a.v_stride : a.k + (k0 + j) * a.k_stride;
        for (int i = 0; i < E; ++i) x[i] = bf16_bits_to_float(r[hk * D + lane * E + i]);
    }, o, lse);
    for (int i = 0; i < E; ++i)
        a.out[t * a.out_stride + h * D + lane * E + i] = __bfloat16_as_ushort(__float2bfloat16_rn(o[i]));
    if (a.lse && lane == 0) a.lse[row] = lse;
}

}  // namespace

size_t prefill_workspace(int, int, int, int, int) { return sizeof(Ctrl); }

cudaError_t launch_attn_prefill(const PrefillArgs &a, cudaStream_t s) {
    const int grid = (int)(((int64_t)a.Tq * a.Hq + kWarps - 1) / kWarps) + 1;
    a.D == 128 ? prefill_simple<128><<<grid, kWarps * 32, 0, s>>>(a)
               : prefill_simple<64><<<grid, kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
