// rope_append.cu -- the two HBM-bound row kernels around the attention:
//   append: per-head RMS norm and rotation of q and k and the cache write of
//           k and v, one pass over the projection's rows;
//   gather: cached tokens of sequences back as packed bf16 rows.
#include "attn.h"
#include "device_common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}
// 4 floats -> 4 e4m3 codes (nearest-even, beyond 448: 448; NaN: NaN)
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}
// 4 e4m3 codes -> 4 floats, exactly
__device__ __forceinline__ void from_e4m3x4(uint32_t w, float (&f)[4]) {
    uint32_t a, b;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"((uint16_t)w));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"((uint16_t)(w >> 16)));
    const float2 x = __half22float2(*reinterpret_cast<__half2 *>(&a));
    const float2 y = __half22float2(*reinterpret_cast<__half2 *>(&b));
    f[0] = x.x;
    f[1] = x.y;
    f[2] = y.x;
    f[3] = y.y;
}

// Smallest index over a block (INT_MAX: none), in thread 0.
__device__ __forceinline__ int block_min(int v) {
    __shared__ int part[kThreads / 32];
    v = __reduce_min_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int i = 1; i < kThreads / 32; ++i) v = min(v, part[i]);
    return v;
}
constexpr int kNone = 0x7fffffff;
__device__ __forceinline__ void write_status(Ctrl *ctrl, int first_bad) {
    ctrl->status = first_bad == kNone ? MOE_OK : MOE_ERR_DEVICE_BAD_INDEX;
    ctrl->detail = first_bad == kNone ? 0 : first_bad;
}

__device__ __forceinline__ bool token_ok(const AppendArgs &a, int t, int &slot) {
    slot = (a.data && a.slots) ? __ldg(a.slots + t) : -1;
    const bool pos_ok = a.rot == 0 || (unsigned)__ldg(a.positions + t) < (unsigned)a.max_pos;
    return pos_ok && slot >= -1 && slot < (a.num_pages << a.page_shift);
}

// Block 0 looks every token over and writes the status word; block
// 1 + t * gridDim.y... handles one part of token t's heads: groups of D/8
// lanes take one head each (8 values a lane), so the norm and the cache
// scale are shuffles within a group, and a half-layout pair's partner is
// another lane of the group.
template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendArgs a) {
    constexpr int L = D / 8;               // lanes per head
    constexpr int NG = kThreads / L;       // groups per block
    if (blockIdx.x == 0) {
        if (blockIdx.y) return;
        int bad = kNone, slot;
        for (int t = threadIdx.x; t < a.T; t += kThreads)
            if (bad == kNone && !token_ok(a, t, slot)) bad = t;
        bad = block_min(bad);
        if (threadIdx.x == 0) write_status(a.ctrl, bad);
        return;
    }
    const int t = blockIdx.x - 1;
    const int lane = threadIdx.x % L;
    const int d0 = lane * 8;
    int slot;
    if (!token_ok(a, t, slot)) return;
    // this lane's cosines and signed sines: out = x c + partner s
    float c[8], s[8];
    const bool turned = d0 < a.rot;
    const int half = a.rot / 2;
    int partner = threadIdx.x & 31;
    if (turned) {
        const float *row = a.cos_sin + (size_t)__ldg(a.positions + t) * a.rot;
        if (a.interleaved) {
            const float4 cc = __ldg(reinterpret_cast<const float4 *>(row + d0 / 2));
            const float4 ss = __ldg(reinterpret_cast<const float4 *>(row + half + d0 / 2));
            const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = cv[i / 2];
                s[i] = (i & 1) ? sv[i / 2] : -sv[i / 2];
            }
        } else {
            const bool first = d0 < half;
            const int i0 = first ? d0 : d0 - half;
            partner += first ? half / 8 : -(half / 8);
            const float sign = first ? -1.f : 1.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float4 cc = __ldg(reinterpret_cast<const float4 *>(row + i0) + j);
                const float4 ss = __ldg(reinterpret_cast<const float4 *>(row + half + i0) + j);
                c[4 * j] = cc.x, c[4 * j + 1] = cc.y, c[4 * j + 2] = cc.z, c[4 * j + 3] = cc.w;
                s[4 * j] = sign * ss.x, s[4 * j + 1] = sign * ss.y;
                s[4 * j + 2] = sign * ss.z, s[4 * j + 3] = sign * ss.w;
            }
        }
    }
    const int rows = a.Hq + 2 * a.Hkv;
    // (every lane of a warp runs every pass: the shuffles need them all)
    for (int r0 = blockIdx.y * NG; r0 < rows; r0 += gridDim.y * NG) {
        const int r = r0 + threadIdx.x / L;
        const bool live = r < rows;
        const int kind = r < a.Hq ? 0 : (r < a.Hq + a.Hkv ? 1 : 2);
        const int h = kind == 0 ? r : (kind == 1 ? r - a.Hq : r - a.Hq - a.Hkv);
        const uint16_t *src = kind == 0 ? a.q + t * a.q_stride
                                        : (kind == 1 ? a.k + t * a.k_stride : a.v + t * a.v_stride);
        uint4 in = make_uint4(0, 0, 0, 0);
        if (live) in = *reinterpret_cast<const uint4 *>(src + h * D + d0);
        float x[8];
        unpack8(in, x);
        const uint16_t *w = kind == 0 ? a.q_norm : (kind == 1 ? a.k_norm : nullptr);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (w) {
            const float r_ = rsqrtf(ss * (1.0f / D) + a.eps);
            float wf[8];
            unpack8(__ldg(reinterpret_cast<const uint4 *>(w + d0)), wf);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * r_ * wf[i];
        }
        float p[8];
        if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = x[i ^ 1];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = __shfl_sync(0xffffffffu, x[i], partner);
        }
        if (turned && kind < 2) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], c[i], p[i] * s[i]);
        }
        float amax = 0.f, scale = 0.f;
        if (FP8) {
            float nan = 0.f;  // NaN if any value is infinite or NaN
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                amax = fmaxf(amax, fabsf(x[i]));
                nan = fmaf(x[i], 0.f, nan);
            }
#pragma unroll
            for (int o = L / 2; o; o >>= 1) {
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                nan += __shfl_xor_sync(0xffffffffu, nan, o);
            }
            amax += nan;
        }
        if (!live) continue;
        if (kind == 0) {
            *reinterpret_cast<uint4 *>(a.q_out + t * a.q_out_stride + h * D + d0) = pack8(x);
            continue;
        }
        if (kind == 1 && a.k_out)
            *reinterpret_cast<uint4 *>(a.k_out + t * a.k_out_stride + h * D + d0) = pack8(x);
        if (slot < 0) continue;
        const size_t page = (size_t)(slot >> a.page_shift);
        const size_t row = (((page * a.Hkv + h) * 2 + (kind - 1)) << a.page_shift) +
                           (slot & ((1 << a.page_shift) - 1));
        if (FP8) {
            scale = amax / 448.0f;
            const float inv = amax > 0.f ? 448.0f / amax : (amax == 0.f ? 0.f : amax);
            const uint2 o = make_uint2(e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                                       e4m3x4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
            *reinterpret_cast<uint2 *>(a.data + row * D + d0) = o;
            if (lane == 0) a.scales[row] = scale;
        } else {
            *reinterpret_cast<uint4 *>(a.data + (row * D + d0) * 2) = pack8(x);
        }
    }
}

// Sequence of packed row t: the last b with cu[b] <= t (cu[0] <= t assumed;
// a non-monotone cu gives some b in [0, B), which the caller checks).
__device__ __forceinline__ int find_seq(const int32_t *cu, int B, int t) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(cu + mid) <= t) lo = mid; else hi = mid;
    }
    return lo;
}

constexpr int kGatherTokens = 16;

// Block 0 looks the tables over; every other block reads kGatherTokens
// tokens, all heads, K and V.  A thread moves 8 values at a time.
template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) gather_kernel(GatherKvArgs a) {
    constexpr int L = D / 8;
    constexpr int NG = kThreads / L;
    const int page_mask = (1 << a.kv.page_shift) - 1;
    if (blockIdx.x == 0) {
        int bad = kNone;
        for (int b = threadIdx.x; b < a.B; b += kThreads) {
            const int64_t n = (int64_t)__ldg(a.cu_k + b + 1) - __ldg(a.cu_k + b);
            if ((n < 0 || n > ((int64_t)a.table_stride << a.kv.page_shift)) && b < bad) bad = b;
        }
        // the pages in use, one warp per sequence
        for (int b = threadIdx.x >> 5; b < a.B; b += kThreads / 32) {
            const int64_t n = (int64_t)__ldg(a.cu_k + b + 1) - __ldg(a.cu_k + b);
            const int64_t pages = min((n + page_mask) >> a.kv.page_shift, (int64_t)a.table_stride);
            for (int64_t i = threadIdx.x & 31; i < pages; i += 32)
                if ((unsigned)__ldg(a.page_table + (size_t)b * a.table_stride + i) >=
                        (unsigned)a.kv.num_pages && b < bad)
                    bad = b;
        }
        if (threadIdx.x == 0 && bad == kNone && (__ldg(a.cu_k) != 0 || __ldg(a.cu_k + a.B) != a.Tk))
            bad = a.B;
        bad = block_min(bad);
        if (threadIdx.x == 0) write_status(a.ctrl, bad);
        return;
    }
    // row of head 0's K in the cache for each of this block's tokens, -1: none
    __shared__ int64_t base[kGatherTokens];
    const int t0 = (blockIdx.x - 1) * kGatherTokens;
    const int nt = min(kGatherTokens, a.Tk - t0);
    if (threadIdx.x < nt) {
        const int t = t0 + threadIdx.x;
        const int b = find_seq(a.cu_k, a.B, t);
        const int64_t i = (int64_t)t - __ldg(a.cu_k + b);
        int64_t at = -1;
        if (i >= 0 && t < __ldg(a.cu_k + b + 1) && (i >> a.kv.page_shift) < a.table_stride) {
            const int pg = __ldg(a.page_table + (size_t)b * a.table_stride + (i >> a.kv.page_shift));
            if ((unsigned)pg < (unsigned)a.kv.num_pages)
                at = (((int64_t)pg * a.kv.Hkv * 2) << a.kv.page_shift) + (i & page_mask);
        }
        base[threadIdx.x] = at;
    }
    __syncthreads();
    const int lane = threadIdx.x % L;
    const int n = nt * a.kv.Hkv * 2;
#pragma unroll 4
    for (int w = threadIdx.x / L; w < n; w += NG) {
        const int i = w % nt, hk = w / nt;  // hk = h * 2 + (0 K, 1 V)
        const int64_t b = base[i];
        uint4 o = make_uint4(0, 0, 0, 0);
        if (b >= 0) {
            const size_t row = (size_t)b + ((size_t)hk << a.kv.page_shift);
            if (FP8) {
                const uint2 u = __ldg(reinterpret_cast<const uint2 *>(a.kv.data + row * D) + lane);
                const float sc = __ldg(a.kv.scales + row);
                float x[4], y[4];
                from_e4m3x4(u.x, x);
                from_e4m3x4(u.y, y);
                o = make_uint4(pack2(x[0] * sc, x[1] * sc), pack2(x[2] * sc, x[3] * sc),
                               pack2(y[0] * sc, y[1] * sc), pack2(y[2] * sc, y[3] * sc));
            } else {
                o = __ldg(reinterpret_cast<const uint4 *>(a.kv.data + row * D * 2) + lane);
            }
        }
        const int t = t0 + i, h = hk >> 1;
        uint16_t *dst = (hk & 1) ? a.v_out + t * a.v_out_stride : a.k_out + t * a.k_out_stride;
        *(reinterpret_cast<uint4 *>(dst + h * D) + lane) = o;
    }
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, cudaStream_t s) {
    const int L = a.D / 8, groups = kThreads / L;
    const int passes = (a.Hq + 2 * a.Hkv + groups - 1) / groups;
    // few tokens: one pass of heads per block; many: one block per token
    const int parts = a.T >= 1024 ? 1 : passes;
    const dim3 grid(a.T + 1, parts);
    const bool fp8 = a.cache_type == MOE_KV_FP8 && a.data;
    if (a.D == 128)
        fp8 ? append_kernel<128, true><<<grid, kThreads, 0, s>>>(a)
            : append_kernel<128, false><<<grid, kThreads, 0, s>>>(a);
    else
        fp8 ? append_kernel<64, true><<<grid, kThreads, 0, s>>>(a)
            : append_kernel<64, false><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_kv_gather(const GatherKvArgs &a, cudaStream_t s) {
    const int grid = (a.Tk + kGatherTokens - 1) / kGatherTokens + 1;
    const bool fp8 = a.cache_type == MOE_KV_FP8;
    if (a.D == 128)
        fp8 ? gather_kernel<128, true><<<grid, kThreads, 0, s>>>(a)
            : gather_kernel<128, false><<<grid, kThreads, 0, s>>>(a);
    else
        fp8 ? gather_kernel<64, true><<<grid, kThreads, 0, s>>>(a)
            : gather_kernel<64, false><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
