// page_plan.cu -- page tables, slots and positions of one step from the
// requests' lengths, and the pages that go back.
//
// A sequence of L0 cached tokens whose pages are there for d more (dropped ones)
// and that gets n new ones needs pages ceil((L0 + d) / P) to ceil((L0 + n) / P) - 1,
// or has some to give back; which free pages these are, and where its rows,
// and the pages that it gives back, stand among everybody's, are prefix sums over
// the sequences.  Free pages are a ring: taken from its head, given back behind
// its tail, so that no place that is read is written by the same call.  All the
// rest is a few integers a row: latency bounds small calls, bytes large ones.
//
// One block makes the sums; if the step is valid and the pages suffice, rows and
// pages follow from its records.
//  kOwnBlock: small steps are finished by the same block.
//  kEveryBlock: larger ones by a whole grid, every block of which makes the sums for
//    itself: a sequence's numbers are read by all, so none of them may be written
//    in place.
//  kTwoKernels: in place, or too many sequences for that, by a second kernel.
// Measured (in a captured graph): 90 sequences of a token each with windows 7.5 us, in
// place 7.0; 256 prompts of 902 thousand rows, 7.3 MB, 9.4 us by every block, and 12.5 to
// 15 by two kernels, as where the pool's state moves on in place (the Python layer's
// default).
#include <climits>

#include "device_common.cuh"
#include "paging.h"

namespace moe {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kRowsPerWarp = 256;
// Rows and sequences up to which the plan's own block finishes the step.
constexpr int kSmallRows = 4096, kSmallSeqs = kPlanThreads;
enum Mode { kOwnBlock, kEveryBlock, kTwoKernels };

// What the rest of the step needs to know of a sequence.
struct __align__(16) Rec {
    int32_t len, grow;    // cached tokens before, new tokens (-1: it has finished)
    int32_t row, take;    // first row; pages taken by the sequences before
    int32_t give, held;   // pages given back by the sequences before; pages in its table
    // Pages that go back: finished, [0, end) and [from, held); else [from, end), which
    // are behind the window, and those past the new length.
    int32_t from, end;
};
struct PlanState {
    int32_t ok, head, count, rows;
};
struct PlanLayout {
    size_t state, rec, total;
};
__host__ __device__ inline PlanLayout plan_layout(int B) {
    PlanLayout l;
    l.state = 256;
    l.rec = 512;
    l.total = l.rec + (size_t)(B > 0 ? B : 1) * sizeof(Rec);
    return l;
}

__device__ __forceinline__ int pages_for(int tokens, int shift) {
    return (int)(((int64_t)tokens + (1 << shift) - 1) >> shift);
}
// The place of the ring that `at` < 3 cap means.
__device__ __forceinline__ int ring_at(int64_t at, int cap) {
    if (at >= 2 * (int64_t)cap) at -= 2 * (int64_t)cap;
    return (int)(at >= cap ? at - cap : at);
}

// Four sums over a block's threads: the totals of the threads before this one,
// and of all.
struct Sums {
    int64_t v[4];
};
// Only the first `used` threads have any; one warp adds up the warps' sums.
__device__ __forceinline__ void warp_scan(Sums &x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x.v[i], o);
            if (lane >= o) x.v[i] += y;
        }
}
__device__ __forceinline__ void block_scan(const Sums &mine, int used, Sums &before, Sums &all, Sums *shared) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Sums x = mine;
    if (warp * 32 < used) {
        warp_scan(x);
        if (lane == 31) shared[warp] = x;
    }
    __syncthreads();
    if (warp == 0) {  // (32 warps)
        Sums w = lane * 32 < used ? shared[lane] : Sums{{0, 0, 0, 0}};
        warp_scan(w);
        shared[lane] = w;
    }
    __syncthreads();
    all = shared[31];
#pragma unroll
    for (int i = 0; i < 4; ++i) before.v[i] = (warp ? shared[warp - 1].v[i] : 0) + x.v[i] - mine.v[i];
    __syncthreads();
}

// The pages of one sequence that a group of `step` threads takes and gives back.
__device__ __forceinline__ void move_pages(const PagePlanArgs &a, int b, const Rec &r, const PlanState &st, int first,
                                           int step) {
    int32_t *row = a.table + (size_t)b * a.table_stride;
    const int p1 = r.grow >= 0 ? pages_for(r.len + r.grow, a.page_shift) : 0;
#pragma unroll 4
    for (int i = first; i < p1 - r.held; i += step)
        row[r.held + i] = a.ring[ring_at((int64_t)st.head + r.take + i, a.cap)];
    const int a0 = r.grow < 0 ? 0 : r.from, an = r.end - a0, b0 = r.grow < 0 ? r.from : min(p1, r.held);
#pragma unroll 4
    for (int i = first; i < an + r.held - b0; i += step)
        a.ring[ring_at((int64_t)st.head + st.count + r.give + i, a.cap)] = row[i < an ? a0 + i : b0 + i - an];
}

// Position and slot of row t, of sequence b.
__device__ __forceinline__ int2 look_up(const PagePlanArgs &a, const Rec &r, const PlanState &st, int b, int t) {
    int pos = 0, slot = -1;
    if (t < st.rows) {
        const int j = r.len + t - r.row, p = j >> a.page_shift;
        const int pg = p < r.held ? a.table[(size_t)b * a.table_stride + p]
                              : a.ring[ring_at((int64_t)st.head + r.take + p - r.held, a.cap)];
        slot = (int)(((uint32_t)pg << a.page_shift) + (j & ((1 << a.page_shift) - 1)));
        if (pg < 0) slot = -1;
        pos = a.offsets ? (int)((uint32_t)r.len + (uint32_t)a.offsets[t]) : j;
    }
    return make_int2(pos, slot);
}
// The sequence of row t: the last one whose first row is at most t (one warp,
// all lanes; 32 places are looked at together).
__device__ __forceinline__ int find_sequence(const int32_t *cu, int B, int t) {
    int lo = 0, n = B;  // it is in [lo, lo + n)
    const int lane = threadIdx.x & 31;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lo + lane * step;
        const bool le = lane * step < n && *(volatile const int32_t *)(cu + at) <= t;
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);
        n = min(step, n - k * step);
        lo += k * step;
    }
    return lo;
}
// The same by one thread, among the sequences from b on.
__device__ __forceinline__ int find_from(const int32_t *cu, int B, int b, int t) {
    int n = B - b;
    while (n > 1) {
        const int half = n / 2;
        if (cu[b + half] <= t) {
            b += half;
            n -= half;
        } else {
            n = half;
        }
    }
    return b;
}
// Rows [t0, t0 + kRowsPerWarp) by one warp; the loads of all of a lane's rows are
// in flight together.
__device__ __forceinline__ void put_rows(const PagePlanArgs &a, const Rec *recs, const int32_t *cu, const PlanState &st,
                                         int t0) {
    const int lane = threadIdx.x & 31, b0 = t0 < st.rows ? find_sequence(cu, a.B, t0) : 0;
    const Rec r0 = recs[b0];
    constexpr int kEach = kRowsPerWarp / 32;
    int2 v[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int t = min(t0 + 32 * i + lane, a.rows - 1);
        const bool later = t < st.rows && t >= r0.row + max(r0.grow, 0);  // a later sequence's
        const int b = later ? find_from(cu, a.B, b0, t) : b0;
        v[i] = look_up(a, later ? recs[b] : r0, st, b, t);
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int t = t0 + 32 * i + lane;
        if (t < a.rows) {
            a.positions[t] = v[i].x;
            a.slots[t] = v[i].y;
        }
    }
}

// All rows and all pages, by the warps of a grid.
__device__ __forceinline__ void fill(const PagePlanArgs &a, const Rec *recs, const int32_t *cu, const PlanState &st) {
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x / 32);
    const int64_t me = (int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
    const int64_t row_items = ((int64_t)a.rows + kRowsPerWarp - 1) / kRowsPerWarp;
    for (int64_t w = me; w < row_items + a.B; w += warps) {
        if (w < row_items) {
            put_rows(a, recs, cu, st, (int)(w * kRowsPerWarp));
        } else if (st.ok) {
            const int b = (int)(w - row_items);
            move_pages(a, b, recs[b], st, threadIdx.x & 31, 32);
        }
    }
}

__global__ void __launch_bounds__(kPlanThreads) plan_step(const PagePlanArgs a, const Mode mode) {
    __shared__ Sums shared[kPlanThreads / 32];
    __shared__ int first_bad, cu_shared[kSmallSeqs];
    __shared__ Rec recs_shared[kSmallSeqs];
    pdl_trigger();
    const int tid = threadIdx.x;
    const PlanLayout L = plan_layout(a.B);
    Rec *recs = mode == kTwoKernels ? reinterpret_cast<Rec *>(a.workspace + L.rec) : recs_shared;
    const bool tells = blockIdx.x == 0;  // writes what is not a row's or a page's
    if (tid == 0) first_bad = INT_MAX;
    const int head = a.state[0], count = a.state[1];
    const int64_t room = min((int64_t)a.table_stride << a.page_shift, (int64_t)1 << 30);
    const int first = a.window ? (int)(((int64_t)a.sinks + (1 << a.page_shift) - 1) >> a.page_shift) : 0;
    const bool ring_ok = head >= 0 && head < a.cap && count >= 0 && count <= a.cap;
    int len = 0, n = 0, kept = 0;  // (of the last pass's sequence)
    Sums base = {{0, 0, 0, 0}};  // of the sequences before this pass: rows, pages taken, given back, lengths
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        Rec r = {0, 0, 0, 0, 0, 0, 0, 0};
        Sums mine = {{0, 0, 0, 0}};
        bool bad = false;
        if (b < a.B) {
            len = a.seq_lens[b];
            n = a.new_lens[b];
            kept = a.window ? a.kept[b] : 0;
            const int dropped = a.dropped ? a.dropped[b] : 0;
            bad = len < 0 || len > room || dropped < 0 || (int64_t)len + dropped > room || n < -1 ||
                  (int64_t)len + max(n, 0) > room;
            const int held = bad ? 0 : pages_for(len + dropped, a.page_shift);
            // (pages [first, kept) went back behind a window and lie wholly below the length:
            // else it has lost tokens of one of them, whose places are somebody else's by now)
            bad = bad || kept < 0 || kept > max(first, len >> a.page_shift);
            if (!bad) {
                r.len = len;
                r.grow = n;
                r.held = held;
                const int p1 = pages_for(len + max(n, 0), a.page_shift);
                if (n < 0) {
                    r.end = a.window ? min(first, held) : held;
                    r.from = a.window ? max(max(kept, first), r.end) : held;
                    if (r.from > held) r.from = held;
                } else if (a.window) {
                    // behind the window: none of these does a later token see
                    const int behind = (int)(max((int64_t)len + 1 - a.window, (int64_t)0) >> a.page_shift);
                    r.from = max(kept, first);
                    r.end = max(r.from, behind);
                }
                mine.v[0] = max(n, 0);
                mine.v[1] = n < 0 ? 0 : max(p1 - held, 0);
                mine.v[2] = n < 0 ? r.end + held - r.from : r.end - r.from + max(held - p1, 0);
                mine.v[3] = n < 0 ? 0 : len + n;
            }
        }
        Sums before, all;
        block_scan(mine, a.B - b0, before, all, shared);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            before.v[i] += base.v[i];
            base.v[i] += all.v[i];
        }
        if (b < a.B) {
            bad = bad || before.v[0] + mine.v[0] > a.rows || before.v[1] + mine.v[1] > count ||
                  before.v[3] + mine.v[3] > INT_MAX;
            r.row = (int)before.v[0];
            r.take = (int)before.v[1];
            r.give = (int)before.v[2];
            recs[b] = r;
            if (tells) a.cu_q[b] = r.row;
            if (mode != kTwoKernels) cu_shared[b] = r.row;
            if (tells && a.cu_k) a.cu_k[b] = (int)before.v[3];
            if (bad) atomicMin(&first_bad, b);
        }
    }
    // (more pages given back than the ring has places for: one is given twice)
    if (tid == 0 && (!ring_ok || base.v[2] > a.cap - count)) atomicMin(&first_bad, a.B);
    __syncthreads();
    const bool ok = first_bad == INT_MAX;
    for (int b = tid; b < a.B && tells; b += kPlanThreads) {
        if (a.B > kPlanThreads) {
            len = a.seq_lens[b];
            n = a.new_lens[b];
            kept = a.window ? a.kept[b] : 0;
        }
        const int behind = a.window ? (int)(max((int64_t)len + 1 - a.window, (int64_t)0) >> a.page_shift) : 0;
        a.seq_lens_out[b] = !ok ? len : (n < 0 ? 0 : len + n);
        if (a.window) a.kept_out[b] = !ok ? kept : (n < 0 ? 0 : max(kept, behind));
        if (!ok) {
            a.cu_q[b] = 0;
            if (a.cu_k) a.cu_k[b] = 0;
        }
    }
    const PlanState st = {ok, ok ? head : 0, ok ? count : 0, ok ? (int)base.v[0] : 0};
    if (tid == 0 && tells) {
        a.cu_q[a.B] = st.rows;
        if (a.cu_k) a.cu_k[a.B] = ok ? (int)base.v[3] : 0;
        a.state_out[0] = ok ? ring_at(head + base.v[1], a.cap) : head;
        a.state_out[1] = ok ? (int)(count - base.v[1] + base.v[2]) : count;
        Ctrl *ctrl = reinterpret_cast<Ctrl *>(a.workspace);
        ctrl->status = ok ? MOE_OK : MOE_ERR_DEVICE_BAD_INDEX;
        ctrl->detail = ok ? 0 : first_bad;
        *reinterpret_cast<PlanState *>(a.workspace + L.state) = st;
    }
    if (mode == kTwoKernels) return;
    __syncthreads();
    if (mode == kEveryBlock) {
        fill(a, recs, cu_shared, st);
        return;
    }
    const int warp = tid >> 5, lane = tid & 31;
    if (ok) {
        // a thread its sequence; those with more pages than a few, a warp together
        for (int b0 = warp * 32; b0 < a.B; b0 += kPlanThreads) {
            Rec r = {0, 0, 0, 0, 0, 0, 0, 0};
            if (b0 + lane < a.B) r = recs[b0 + lane];
            const int most = r.grow < 0 ? r.end + r.held - r.from
                                        : max(r.grow >> a.page_shift, r.held - (r.len >> a.page_shift) + r.end - r.from);
            const uint32_t big = __ballot_sync(0xffffffffu, most > 2);
            if (b0 + lane < a.B && most <= 2) move_pages(a, b0 + lane, r, st, 0, 1);
            for (uint32_t m = big; m; m &= m - 1) {
                const int b = b0 + __ffs(m) - 1;
                move_pages(a, b, recs[b], st, lane, 32);
            }
        }
    }
    for (int t = tid; t < a.rows; t += kPlanThreads)
    {
        const int b = t < st.rows ? find_from(cu_shared, a.B, 0, t) : 0;
        const int2 v = look_up(a, recs[b], st, b, t);
        a.positions[t] = v.x;
        a.slots[t] = v.y;
    }
}

__global__ void __launch_bounds__(kFillThreads) fill_step(const PagePlanArgs a) {
    const PlanLayout L = plan_layout(a.B);
    const Rec *recs = reinterpret_cast<const Rec *>(a.workspace + L.rec);
    pdl_wait();
    const PlanState st = *reinterpret_cast<const PlanState *>(a.workspace + L.state);
    fill(a, recs, a.cu_q, st);
}

}  // namespace

size_t page_plan_workspace(int B) { return align_up(plan_layout(B).total, 256); }

cudaError_t launch_page_plan(const PagePlanArgs &a, cudaStream_t s) {
    const bool in_place =
        a.state == a.state_out || a.seq_lens == a.seq_lens_out || (a.window && a.kept == a.kept_out);
    const Mode mode = a.B > kSmallSeqs         ? kTwoKernels
                      : a.rows <= kSmallRows ? kOwnBlock
                      : in_place             ? kTwoKernels
                                             : kEveryBlock;
    const int64_t warps = ((int64_t)a.rows + kRowsPerWarp - 1) / kRowsPerWarp + a.B;
    const int64_t full = (warps * 32 + kPlanThreads - 1) / kPlanThreads;
    plan_step<<<mode == kEveryBlock ? (unsigned)(full < 152 ? full : 152) : 1, kPlanThreads, 0, s>>>(a, mode);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess || mode != kTwoKernels) return err;
    const int64_t blocks = (warps * 32 + kFillThreads - 1) / kFillThreads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks < 152 * 8 ? blocks : 152 * 8));
    cfg.blockDim = dim3(kFillThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fill_step, a);
}

}  // namespace moe
