// rope_append.cu -- the two HBM-bound row kernels around the attention:
//   append: per-head RMS norm and rotation of q and k and the cache write of
//           k and v, one pass over the projection's rows;
//   gather: cached tokens of sequences back as packed bf16 rows.
// Both move every byte once and do little else, so HBM bounds them; measured on
// one GB300 (copy rate 6.79 TB/s): append of 16384 tokens, 64 + 8 + 8 heads of
// 128, fp8 cache and k_out, 681 MB in 118 us (5.8 TB/s), gather of 8 contexts up
// to 32768 tokens, fp8, 605 MB in 94.5 us (6.4 TB/s).  A call of a few tokens
// takes 4.7 us on the GPU, less than the host needs to make it.
#include "attn.h"
#include "device_common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;        // gather
constexpr int kAppendThreads = 64;

__device__ __forceinline__ void unpack4(const uint2 &u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x << 16);
    x[1] = __uint_as_float(u.x & 0xFFFF0000u);
    x[2] = __uint_as_float(u.y << 16);
    x[3] = __uint_as_float(u.y & 0xFFFF0000u);
}
// Two interleaved pieces of 4 -> the first and the second sides of their
// pairs, and back.
__device__ __forceinline__ void sides(float (&x)[4], float (&y)[4]) {
    const float a[4] = {x[0], x[2], y[0], y[2]}, b[4] = {x[1], x[3], y[1], y[3]};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = a[i], y[i] = b[i];
}
__device__ __forceinline__ void pieces(float (&x)[4], float (&y)[4]) {
    const float a[4] = {x[0], y[0], x[1], y[1]}, b[4] = {x[2], y[2], x[3], y[3]};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = a[i], y[i] = b[i];
}
// x y and x y + z on pairs of fp32
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, r;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 r, x, y;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, r;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 r, x, y, z;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
    return r;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
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
    __shared__ int part[32];
    v = __reduce_min_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int i = 1; i < blockDim.x / 32; ++i) v = min(v, part[i]);
    return v;
}
constexpr int kNone = 0x7fffffff;
__device__ __forceinline__ void write_status(Ctrl *ctrl, int first_bad) {
    ctrl->status = first_bad == kNone ? MOE_OK : MOE_ERR_DEVICE_BAD_INDEX;
    ctrl->detail = first_bad == kNone ? 0 : first_bad;
}

// (slot is -1 without a cache, the position 0 without a rotation)
__device__ __forceinline__ bool token_ok(const AppendArgs &a, int pos, int slot) {
    return (a.rot == 0 || (unsigned)pos < (unsigned)a.max_pos) && slot >= -1 &&
           slot < (a.num_pages << a.page_shift);
}

// Block (0, 0) looks every token over and writes the status word; blocks
// (1 + t, y) share the heads of token t.  A group of D/8 lanes takes one head
// (a row), 8 values a lane in two pieces of 4 that hold both sides of its
// pairs: pieces rot/2 apart in the half layout, neighbours otherwise.  The
// rotation then needs no other lane; the norm and the cache scale are
// shuffles within the group.
//
// HBM bounds the work, but with 4 values in and 2 to 4 bytes out per value
// the instructions come close: norm weights, cosines and sines of a lane's
// four pairs are folded into 16 factors once per token, each kind of row has
// its own loop, and the arithmetic is on pairs of fp32.
enum Kind { kQuery, kKey, kValue };

// A lane's place in a row.
struct Place {
    int lane, dA, dB;
    bool turned;      // its values are rotated
    uint32_t group;   // the lanes of its group
};

// a' = rms (a ac - b bs), b' = rms (b bc + a as) of a lane's pairs, two at a time
struct Turn {
    float2 ac[2], as[2], bc[2], bs[2];
};

// The weights of a lane's pairs, one from each side, by pairs of pairs.
__device__ __forceinline__ Turn fold(const uint16_t *w, const Place &p, bool interleaved, float4 c, float4 s) {
    float x[4] = {1.f, 1.f, 1.f, 1.f}, y[4] = {1.f, 1.f, 1.f, 1.f};
    if (w) {
        unpack4(__ldg(reinterpret_cast<const uint2 *>(w + p.dA)), x);
        unpack4(__ldg(reinterpret_cast<const uint2 *>(w + p.dB)), y);
    }
    if (interleaved) sides(x, y);
    Turn t;
    t.ac[0] = make_float2(x[0] * c.x, x[1] * c.y);
    t.ac[1] = make_float2(x[2] * c.z, x[3] * c.w);
    t.as[0] = make_float2(x[0] * s.x, x[1] * s.y);
    t.as[1] = make_float2(x[2] * s.z, x[3] * s.w);
    t.bc[0] = make_float2(y[0] * c.x, y[1] * c.y);
    t.bc[1] = make_float2(y[2] * c.z, y[3] * c.w);
    t.bs[0] = make_float2(-y[0] * s.x, -y[1] * s.y);
    t.bs[1] = make_float2(-y[2] * s.z, -y[3] * s.w);
    return t;
}

// Rows r, r + step, ... < n of one kind, the next two on the way at any time.
// PART: some values of a row are not rotated (16384 tokens of 64 + 8 + 8 rows:
// 118.7 us, 117.2 where all are).
template <int D, bool FP8, bool PART, int KIND>
__device__ __forceinline__ void walk(const AppendArgs &a, const Place &p, const Turn &f, bool norm,
                                     const uint16_t *src, uint16_t *dst, int &r, int n, int step, int slot,
                                     const uint2 (&ahead)[2][2]) {
    constexpr int L = D / 8;
    uint2 in[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        if (KIND == kQuery) {
            in[u][0] = ahead[u][0];
            in[u][1] = ahead[u][1];
        } else if (r + u * step < n) {
            in[u][0] = *reinterpret_cast<const uint2 *>(src + (r + u * step) * D + p.dA);
            in[u][1] = *reinterpret_cast<const uint2 *>(src + (r + u * step) * D + p.dB);
        }
    }
    const size_t page = (size_t)(max(slot, 0) >> a.page_shift);
    const size_t row0 = ((page * a.Hkv * 2 + (KIND == kValue)) << a.page_shift) +
                        (slot & ((1 << a.page_shift) - 1));
    const bool cached = KIND != kQuery && slot >= 0;
    while (r < n) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (r >= n) return;
            float x[4], y[4];
            unpack4(in[u][0], x);
            unpack4(in[u][1], y);
            if (r + 2 * step < n) {
                in[u][0] = *reinterpret_cast<const uint2 *>(src + (r + 2 * step) * D + p.dA);
                in[u][1] = *reinterpret_cast<const uint2 *>(src + (r + 2 * step) * D + p.dB);
            }
            if (KIND != kValue) {
                float2 rms = make_float2(1.f, 1.f);
                if (norm) {
                    float2 q = mul2(make_float2(x[0], x[1]), make_float2(x[0], x[1]));
                    q = fma2(make_float2(x[2], x[3]), make_float2(x[2], x[3]), q);
                    q = fma2(make_float2(y[0], y[1]), make_float2(y[0], y[1]), q);
                    q = fma2(make_float2(y[2], y[3]), make_float2(y[2], y[3]), q);
                    float ss = q.x + q.y;
#pragma unroll
                    for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(p.group, ss, o);
                    rms.x = rms.y = rsqrtf(ss * (1.0f / D) + a.eps);
                }
                if (a.interleaved) sides(x, y);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2 A = mul2(make_float2(x[2 * k], x[2 * k + 1]), rms);
                    const float2 B = mul2(make_float2(y[2 * k], y[2 * k + 1]), rms);
                    float2 A2 = mul2(B, f.bs[k]), B2 = mul2(A, f.as[k]);
                    // (a value without a rotation must not meet its partner,
                    // not even times 0: that may be an infinity or NaN)
                    if (PART && !p.turned) A2 = B2 = make_float2(0.f, 0.f);
                    A2 = fma2(A, f.ac[k], A2);
                    B2 = fma2(B, f.bc[k], B2);
                    x[2 * k] = A2.x;
                    x[2 * k + 1] = A2.y;
                    y[2 * k] = B2.x;
                    y[2 * k + 1] = B2.y;
                }
                if (a.interleaved) pieces(x, y);
            }
            const uint2 oA = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
            const uint2 oB = make_uint2(pack2(y[0], y[1]), pack2(y[2], y[3]));
            if (KIND != kValue && dst) {
                *reinterpret_cast<uint2 *>(dst + r * D + p.dA) = oA;
                *reinterpret_cast<uint2 *>(dst + r * D + p.dB) = oB;
            }
            if (cached) {
                const size_t row = row0 + ((size_t)(r * 2) << a.page_shift);
                if (FP8) {
                    // the largest magnitude by its bits: above every number
                    // stand infinity and then NaN
                    uint32_t top = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
                        top = max(top, __float_as_uint(y[i]) & 0x7FFFFFFFu);
                    }
#pragma unroll
                    for (int o = L / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(p.group, top, o));
                    // (below 2^-119 the factor 448 / amax would overflow)
                    constexpr uint32_t kLeast = (127 - 119) << 23;
                    const float amax = __uint_as_float(
                        top >= 0x7F800000u ? 0x7FFFFFFFu : (top == 0 ? 0 : max(top, kLeast)));
                    const float inv = top == 0 ? 0.f : 448.0f / amax;
                    *reinterpret_cast<uint32_t *>(a.data + row * D + p.dA) =
                        e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
                    *reinterpret_cast<uint32_t *>(a.data + row * D + p.dB) =
                        e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
                    if (p.lane == 0) a.scales[row] = amax / 448.0f;
                } else {
                    uint16_t *to = reinterpret_cast<uint16_t *>(a.data) + row * D;
                    *reinterpret_cast<uint2 *>(to + p.dA) = oA;
                    *reinterpret_cast<uint2 *>(to + p.dB) = oB;
                }
            }
            r += step;
        }
    }
}

template <int D, bool FP8, bool PART>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(AppendArgs a) {
    constexpr int L = D / 8;               // lanes per head
    constexpr int NG = kAppendThreads / L; // groups per block
    if (blockIdx.x == 0) {
        if (blockIdx.y) return;
        // 16 tokens a thread at a time: what a block of its own can be late with
        // is latency (15015 tokens of 7 rows: 47 us one after another)
        constexpr int kAtOnce = 16;
        int bad = kNone;
        for (int64_t t0 = threadIdx.x; t0 < a.T; t0 += kAtOnce * kAppendThreads) {
            int slot[kAtOnce], pos[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const int64_t t = t0 + i * kAppendThreads;
                slot[i] = t < a.T && a.data ? __ldg(a.slots + t) : -1;
                pos[i] = t < a.T && a.rot ? __ldg(a.positions + t) : 0;
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                if (!token_ok(a, pos[i], slot[i])) bad = min(bad, (int)t0 + i * kAppendThreads);
        }
        bad = block_min(bad);
        if (threadIdx.x == 0) write_status(a.ctrl, bad);
        return;
    }
    const int t = blockIdx.x - 1;
    Place p;
    p.lane = threadIdx.x % L;
    p.group = (L == 32 ? 0xffffffffu : (1u << (L & 31)) - 1) << ((threadIdx.x & 31) / L * L);
    const int half = a.rot / 2;
    p.turned = p.lane * 8 < a.rot;
    const bool apart = p.turned && !a.interleaved;
    p.dA = apart ? p.lane * 4 : p.lane * 8;
    p.dB = apart ? half + p.lane * 4 : p.lane * 8 + 4;
    // The token's rows in order, q, k and v: this group takes r, r + step, ...
    // The first loads go out before anything that depends on the position.
    const int step = gridDim.y * NG;
    int r = blockIdx.y * NG + threadIdx.x / L;
    const uint16_t *q = a.q + t * a.q_stride;
    uint2 ahead[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
        if (r + u * step < a.Hq) {
            ahead[u][0] = *reinterpret_cast<const uint2 *>(q + (r + u * step) * D + p.dA);
            ahead[u][1] = *reinterpret_cast<const uint2 *>(q + (r + u * step) * D + p.dB);
        }
    const int slot = a.data ? __ldg(a.slots + t) : -1;
    const int pos = a.rot ? __ldg(a.positions + t) : 0;
    if (!token_ok(a, pos, slot)) return;
    // this lane's four pairs are the pairs 4 lane .. 4 lane + 3
    float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.turned) {
        const float *row = a.cos_sin + (size_t)pos * a.rot + p.lane * 4;
        c = __ldg(reinterpret_cast<const float4 *>(row));
        s = __ldg(reinterpret_cast<const float4 *>(row + half));
    }
    if (r < a.Hq)
        walk<D, FP8, PART, kQuery>(a, p, fold(a.q_norm, p, a.interleaved, c, s), a.q_norm != nullptr, q,
                                   a.q_out + t * a.q_out_stride, r, a.Hq, step, slot, ahead);
    r -= a.Hq;
    if (r < a.Hkv)
        walk<D, FP8, PART, kKey>(a, p, fold(a.k_norm, p, a.interleaved, c, s), a.k_norm != nullptr,
                                 a.k + t * a.k_stride, a.k_out ? a.k_out + t * a.k_out_stride : nullptr, r,
                                 a.Hkv, step, slot, ahead);
    r -= a.Hkv;
    if (r < a.Hkv && slot >= 0)
        walk<D, FP8, PART, kValue>(a, p, Turn{}, false, a.v + t * a.v_stride, nullptr, r, a.Hkv, step, slot,
                                   ahead);
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
// tokens, all heads, K and V.  A thread moves 8 values at a time: half as many
// bytes in (fp8) as out, whole 16-byte stores to neighbouring addresses.  Four
// rows in flight per thread instead of one: 115 -> 94.5 us at 605 MB.
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
    const int n = kGatherTokens * a.kv.Hkv * 2;
    // kWay rows' loads are in flight before the first is written
    constexpr int kWay = 4;
    for (int w0 = threadIdx.x / L; w0 < n; w0 += NG * kWay) {
        uint4 u[kWay];
        float sc[kWay];
#pragma unroll
        for (int k = 0; k < kWay; ++k) {
            const int w = w0 + k * NG;
            const int i = w % kGatherTokens, hk = w / kGatherTokens;  // hk = h * 2 + (0 K, 1 V)
            const int64_t b = w < n && i < nt ? base[i] : -1;
            u[k] = make_uint4(0, 0, 0, 0);
            sc[k] = 0.f;
            if (b >= 0) {
                const size_t row = (size_t)b + ((size_t)hk << a.kv.page_shift);
                if (FP8) {
                    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(a.kv.data + row * D) + lane);
                    u[k].x = v.x;
                    u[k].y = v.y;
                    sc[k] = __ldg(a.kv.scales + row);
                } else {
                    u[k] = __ldg(reinterpret_cast<const uint4 *>(a.kv.data + row * D * 2) + lane);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kWay; ++k) {
            const int w = w0 + k * NG;
            const int i = w % kGatherTokens, hk = w / kGatherTokens;
            if (w >= n || i >= nt) continue;
            uint4 o = u[k];
            if (FP8) {
                float x[4], y[4];
                from_e4m3x4(u[k].x, x);
                from_e4m3x4(u[k].y, y);
                o = make_uint4(pack2(x[0] * sc[k], x[1] * sc[k]), pack2(x[2] * sc[k], x[3] * sc[k]),
                               pack2(y[0] * sc[k], y[1] * sc[k]), pack2(y[2] * sc[k], y[3] * sc[k]));
            }
            const int t = t0 + i, h = hk >> 1;
            uint16_t *dst = (hk & 1) ? a.v_out + t * a.v_out_stride : a.k_out + t * a.k_out_stride;
            *(reinterpret_cast<uint4 *>(dst + h * D) + lane) = o;
        }
    }
}

}  // namespace

template <int D, bool FP8>
static void append(const AppendArgs &a, cudaStream_t s) {
    // Few tokens: one row per group, so that the heads of a token spread over
    // blocks (latency counts).  Many: a block takes a whole token, so that its
    // position's cosines and the weights are fetched once.  In between as many
    // blocks as make 16 an SM (1023 tokens of 80 rows: 18.5 us with a row per
    // group, 15.9 with a block per token, 13.9).
    constexpr int kGroups = kAppendThreads / (D / 8), kEnough = 16 * 152;
    const int passes = (a.Hq + 2 * a.Hkv + kGroups - 1) / kGroups;
    const int shares = kEnough / (a.T > 0 ? a.T : 1) + 1;
    const dim3 grid(a.T + 1, passes < shares ? passes : shares);
    if (a.rot == D)
        append_kernel<D, FP8, false><<<grid, kAppendThreads, 0, s>>>(a);
    else
        append_kernel<D, FP8, true><<<grid, kAppendThreads, 0, s>>>(a);
}

cudaError_t launch_append(const AppendArgs &a, cudaStream_t s) {
    const bool fp8 = a.cache_type == MOE_KV_FP8 && a.data;
    if (a.D == 128)
        fp8 ? append<128, true>(a, s) : append<128, false>(a, s);
    else
        fp8 ? append<64, true>(a, s) : append<64, false>(a, s);
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
