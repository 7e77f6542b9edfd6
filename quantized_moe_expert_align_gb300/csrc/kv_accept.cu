// kv_accept.cu -- the accepted tokens of a verified tree move to their places.
//
// Token accept[i] of a tree, cached at base + accept[i], becomes token base + i.
// accept rises, so that accept[i] >= i: in the order of i no row is written that
// is still to be read, and a thread that moves one 16-byte column of a sequence's
// rows, a few at a time, needs no others.  What it moves is read and written
// once; a batch moves a few megabytes, so latency bounds it: all table entries are
// looked up together, and up to kWay rows of a column are in flight.  One block looks
// all paths over for the status word, a thread an element.
// Measured: 256 paths of up to 8 tokens, 8 heads of 128, bf16, 7.6 us on the GPU (31 with
// a warp a path in the look over).  That look bounds very large calls: 2048 paths of 64
// take 0.33 ms, 65535 of them 13.6.
#include <type_traits>

#include "device_common.cuh"
#include "paging.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMost = 64;  // accepted tokens of a sequence
constexpr int kWay = 8;
constexpr int kLook = 2048;  // paths that are looked over together

// Whether the path of sequence b may be moved: by one warp, all lanes agree.
// n: its tokens; lane's tokens i = lane and lane + 32: from and to (slots).
__device__ __forceinline__ bool look(const AcceptArgs &a, int b, int &n, int (&from)[2], int (&to)[2]) {
    const int lane = threadIdx.x & 31;
    const int base = __ldg(a.base + b);
    const int64_t room = min((int64_t)a.table_stride << a.kv.page_shift, (int64_t)1 << 30);
    const int mask = (1 << a.kv.page_shift) - 1;
    int acc[2];
    n = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int i = lane + 32 * k;
        acc[k] = i < a.P ? __ldg(a.accept + (size_t)b * a.P + i) : -1;
        const uint32_t end = __ballot_sync(0xffffffffu, acc[k] == -1);
        if (n == 32 * k) n += end ? __ffs(end) - 1 : 32;
    }
    bool bad = base < 0;
    const int32_t *row = a.page_table + (size_t)b * a.table_stride;
    int last = -1;  // the token before this lane's first
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int i = lane + 32 * k;
        int prev = __shfl_up_sync(0xffffffffu, acc[k], 1);
        if (lane == 0) prev = last;
        last = __shfl_sync(0xffffffffu, acc[k], 31);
        from[k] = to[k] = -1;
        if (i >= n) continue;
        bad = bad || acc[k] <= prev || (int64_t)base + acc[k] >= room;
        if (bad) continue;
        const int src = base + acc[k], dst = base + i;  // (dst <= src)
        if (src == dst) continue;
        const int ps = __ldg(row + (src >> a.kv.page_shift)), pd = __ldg(row + (dst >> a.kv.page_shift));
        bad = (unsigned)ps >= (unsigned)a.kv.num_pages || (unsigned)pd >= (unsigned)a.kv.num_pages;
        from[k] = (int)((uint32_t)ps << a.kv.page_shift) + (src & mask);
        to[k] = (int)((uint32_t)pd << a.kv.page_shift) + (dst & mask);
    }
    return !__any_sync(0xffffffffu, bad);
}

// The first sequence whose path may not be moved, into the status word: by one
// block, a thread an element.
__device__ void look_over(const AcceptArgs &a) {
    __shared__ int length[kLook], first_bad;
    const int tid = threadIdx.x;
    const int64_t room = min((int64_t)a.table_stride << a.kv.page_shift, (int64_t)1 << 30);
    if (tid == 0) first_bad = 0x7fffffff;
    for (int b0 = 0; b0 < a.B; b0 += kLook) {
        const int nb = min(kLook, a.B - b0), n = nb * a.P;
        const int32_t *path = a.accept + (size_t)b0 * a.P;
        __syncthreads();
        for (int b = tid; b < nb; b += kThreads) length[b] = a.P;
        __syncthreads();
#pragma unroll 8
        for (int e = tid; e < n; e += kThreads)
            if (__ldg(path + e) == -1) atomicMin(&length[e / a.P], e % a.P);
        __syncthreads();
#pragma unroll 4
        for (int e = tid; e < n; e += kThreads) {
            const int b = e / a.P, i = e % a.P;
            if (i >= length[b]) continue;
            const int acc = __ldg(path + e), prev = i ? __ldg(path + e - 1) : -1, base = __ldg(a.base + b0 + b);
            bool bad = base < 0 || acc <= prev || (int64_t)base + acc >= room;
            if (!bad && acc != i) {
                const int32_t *row = a.page_table + (size_t)(b0 + b) * a.table_stride;
                bad = (unsigned)__ldg(row + ((base + acc) >> a.kv.page_shift)) >= (unsigned)a.kv.num_pages ||
                      (unsigned)__ldg(row + ((base + i) >> a.kv.page_shift)) >= (unsigned)a.kv.num_pages;
            }
            if (bad) atomicMin(&first_bad, b0 + b);
        }
        // (a path without tokens has a base all the same)
        for (int b = tid; b < nb; b += kThreads)
            if (__ldg(a.base + b0 + b) < 0) atomicMin(&first_bad, b0 + b);
    }
    __syncthreads();
    if (tid == 0) {
        a.ctrl->status = first_bad == 0x7fffffff ? MOE_OK : MOE_ERR_DEVICE_BAD_INDEX;
        a.ctrl->detail = first_bad == 0x7fffffff ? 0 : first_bad;
    }
}

// Block 0 looks every path over and writes the status word; block (1 + b, y)
// moves kThreads columns of sequence b.
__global__ void __launch_bounds__(kThreads) accept_kernel(const AcceptArgs a, const int pieces) {
    __shared__ int from[kMost], to[kMost], n_shared;
    const int tid = threadIdx.x, warp = tid >> 5;
    if (blockIdx.x == 0) {
        if (blockIdx.y == 0) look_over(a);
        return;
    }
    int n, f[2], t[2];
    if (warp == 0) {
        const bool ok = look(a, blockIdx.x - 1, n, f, t);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            from[tid + 32 * k] = f[k];
            to[tid + 32 * k] = t[k];
        }
        if (tid == 0) n_shared = ok ? n : 0;
    }
    __syncthreads();
    n = n_shared;
    // a column: 16 bytes of K or V of one head, or (after those) its scale
    const int rows = a.kv.Hkv * 2, c = blockIdx.y * kThreads + tid;
    const int page_mask = (1 << a.kv.page_shift) - 1;
    auto row_of = [&](int slot, int hk) {
        return (((size_t)(slot >> a.kv.page_shift) * rows + hk) << a.kv.page_shift) + (slot & page_mask);
    };
    auto move = [&](auto *p, size_t width, int hk) {
        for (int i0 = 0; i0 < n; i0 += kWay) {
            std::remove_reference_t<decltype(*p)> v[kWay];
#pragma unroll
            for (int k = 0; k < kWay; ++k)
                if (i0 + k < n && from[i0 + k] >= 0) v[k] = p[row_of(from[i0 + k], hk) * width];
#pragma unroll
            for (int k = 0; k < kWay; ++k)
                if (i0 + k < n && from[i0 + k] >= 0) p[row_of(to[i0 + k], hk) * width] = v[k];
        }
    };
    if (c < rows * pieces)
        move(reinterpret_cast<uint4 *>(const_cast<uint8_t *>(a.kv.data)) + c % pieces, pieces, c / pieces);
    else if (a.kv.scales && c < rows * pieces + rows)
        move(const_cast<float *>(a.kv.scales), 1, c - rows * pieces);
}

}  // namespace

cudaError_t launch_kv_accept(const AcceptArgs &a, cudaStream_t s) {
    const int pieces = a.D * (a.cache_type == MOE_KV_FP8 ? 1 : 2) / 16;
    const int columns = a.kv.Hkv * 2 * (pieces + (a.kv.scales ? 1 : 0));
    accept_kernel<<<dim3(a.B + 1, (columns + kThreads - 1) / kThreads), kThreads, 0, s>>>(a, pieces);
    return cudaGetLastError();
}

}  // namespace moe
