// attn_decode.cuh -- attention of few query rows over the paged cache: single
// tokens (attn_decode.cu), single tokens through a sliding window
// (attn_decode_window.cu), small trees of drafted tokens (attn_tree_small.cu).
//
// For head h of sequence b:  o = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),
// s_j = scale log2(e) q . k_j, m the largest s_j.  Every cached byte is read
// once and used for the G query heads that share it (2 G multiply-adds a
// value), so HBM bounds the kernel by far; the work per byte is kept small:
//  * the products are computed transposed, S^T = K Q^T and O^T = V^T P^T, on
//    16 x 8 x 16 matrix instructions whose 16-row side is the keys (then the
//    values' columns) and whose 8-column side is the query heads, so up to 8
//    heads waste nothing and the cache is read from shared memory once;
//  * work is cut into units of 64 or 128 keys of one (sequence, key/value head);
//    the units of the whole batch, in order, are shared out evenly over two or
//    three blocks per SM whatever the lengths are.  A pair cut by a block's end is
//    joined by a second kernel, in key order, so results do not depend on
//    timing;
//  * one warp of a block copies (TMA, a ring of stages), four warps take 16 or
//    32 of a unit's keys each, with a running maximum and sum of their own,
//    joined once per (sequence, head).
// Rows of 128 bytes are swizzled by the copy (64-byte rows likewise), so the
// fragment loads are free of bank conflicts.
//
// Measured on one GB300 (copy rate 6.79 TB/s): 256 sequences up to 8192 keys,
// 64 heads over 8, fp8, 1.79 GB in 280 us (6.4 TB/s); 90 up to 8192, 32 over 4,
// bf16 pages of 16, 657 MB in 108 us (6.1 TB/s); one of 131072 keys, fp8, 277
// MB in 53 us, of which 41 are the bytes and the rest the set-up (lengths, page
// table, first copies) and the join; one of 517 keys 10.2 us.  More heads per
// byte, or fewer bytes per key, are bound by what the warps of an SM get done
// instead: 64 sequences up to 8192 keys, 64 heads of 128 over 4, fp8, 69 us (39
// for the bytes), bf16 94 (76); 64 of 64 over 8 55 (40) and 87 (75).  With 16
// heads of 128 over fp8 registers allow two blocks an SM (five warps each: 168
// registers), too few to hide a warp's chain of steps, and spill: 1.3% of the
// instructions are local loads and stores.  (The figures beside the choices
// below were taken before NaN codes were looked for, which adds 1 to 4% to fp8.)
#pragma once

#include <algorithm>

#include "attn_common.cuh"
#include "gemm_tc.h"

namespace moe {
namespace {

using namespace attn;

constexpr int kCWarps = 4;                 // consumer warps
constexpr int kThreads = (kCWarps + 1) * 32;
constexpr int kMaxGrid = 512;

// What a sequence's query rows see.
//  kPlain: one token, every key.
//  kWindow: one token, the last `window` keys and the first `sinks`.  The keys
//    between are left out of the numbering: the visible ones, each end rounded
//    to whole boxes (the rows of one copy), are keys 0, 1, ... of the kernel,
//    so that what is copied and shared out is what is seen.
//  kTree: up to 64 drafted tokens, the sequence's last keys: each sees every
//    key before them and those of them that its mask names.  The tokens' heads
//    are rows like the heads of one token: row r is head r % G of token r / G.
enum Mode { kPlain, kWindow, kTree };

// A (sequence, head tile) pair whose units the blocks first .. first + parts - 1
// share; parts 0: none.
struct Join {
    int32_t b, hv, parts, first;
};
// Records by pair where the blocks are several times as many as the pairs, by
// the block that a pair starts in otherwise.
__host__ __device__ inline bool join_by_pair(int64_t B, int HV, int blocks) { return B * HV * 8 <= blocks; }
struct Err {
    int32_t timeout, bad;  // role that gave up; first sequence with a bad page or length
};

struct DecodeLayout {
    size_t ctrl, err, join, ml, part, total;
};
// rows = most heads of a tile
__host__ __device__ inline DecodeLayout decode_layout(int rows, int D) {
    DecodeLayout l;
    l.ctrl = 0;
    l.err = 256;
    l.join = l.err + kMaxGrid * sizeof(Err);
    l.ml = l.join + kMaxGrid * sizeof(Join);
    l.part = l.ml + (size_t)kMaxGrid * 2 * rows * 8;
    l.total = l.part + (size_t)kMaxGrid * 2 * rows * D * 4;
    return l;
}

template <int D, bool FP8, int NT>
struct Cfg {
    static constexpr int kRows = 8 * NT;                   // query heads of a tile
    // A consumer warp takes kGroups times 16 keys of a unit: two where a unit's
    // fixed steps (waits, maxima, votes) cost more than its bytes (64 sequences
    // up to 8192 keys, fp8: 64 heads of 64 over 8 63.5 -> 54.4 us, 64 of 128
    // over 4 72.9 -> 66.3).
    static constexpr int kGroups = D == 64 || (FP8 && NT == 2) ? 2 : 1;
    static constexpr int kChunk = 16 * kCWarps * kGroups;
    // Several blocks on an SM hide each other's set-up, joins and latencies:
    // two, for fp8 three (half the bytes for the same steps: 256 sequences up
    // to 8192 keys 282 -> 277 us), except where a tile of 16 heads needs the
    // registers of two (64 sequences, 64 heads over 4, units of 64 keys:
    // 122 us with three, 74).
    static constexpr int kBlocks = FP8 && (NT == 1 || D == 64) ? 3 : 2;
    static constexpr int kSmemLimit = (kBlocks == 2 ? 113 : 75) * 1024;
    static constexpr int kEs = FP8 ? 1 : 2;
    static constexpr int kRowB = D * kEs < 128 ? D * kEs : 128;
    static constexpr int kHalves = D * kEs / kRowB;
    static constexpr int kData = kChunk * D * kEs * 2;     // K and V of a unit
    static constexpr int kScales = FP8 ? kChunk * 8 : 0;
    static constexpr int kQ = kRows * D * 2;
    static constexpr int kStage = kData + kQ + 1024 * ((kScales + 1023) / 1024);
    static constexpr int kExch = kCWarps * 8 * 68 * 4;     // [warp][8 heads][64 + 4] floats
    static constexpr int kMl = kCWarps * kRows * 8;
    static constexpr int kFixed = kExch + kMl + 1024 /* barriers, scan */ + 1024 /* alignment */;
    static constexpr int kFit = (kSmemLimit - kFixed) / kStage;
    static constexpr int kStages = kFit > 8 ? 8 : kFit;
    static constexpr size_t kSmem = kFixed + (size_t)kStages * kStage;
    static_assert(kStages >= 2, "two stages at least");
};

struct Shared {
    uint64_t full[8], empty[8];
    int abort, bad;
    int b0;            // the sequence of this block's first unit
    int64_t first;     // and that unit's index among the sequence's units
    int64_t warp_sum[kThreads / 32];
};
static_assert(sizeof(Shared) <= 1024, "shared block");

// Where a unit of the batch lies.
struct Walk {
    int b, hv, j, n, units;  // sequence, head tile, chunk, keys, chunks of the sequence
    // kWindow: keys from `lead` on stand `shift` further on; of the keys, the
    // first `sinks` and those from `from` on are seen
    int lead, shift, from, sinks;
    // kTree: first row and number of the drafted tokens, tiles of rows (per
    // key/value head, in all)
    int q0, nq, RT, HV;
};

__device__ __forceinline__ int keys_of(const DecodeAttnArgs &a, int b) {
    const int64_t most = min((int64_t)a.table_stride << a.kv.page_shift, (int64_t)1 << 30);
    const int n = __ldg(a.seq_lens + b);
    return n < 0 ? 0 : (n > most ? (int)most : n);
}
// kTree: whether the tokens of sequence b may be used; their first row and number
// (0 too where the other launch has them).
__device__ __forceinline__ bool tokens_of(const DecodeAttnArgs &a, int b, int &q0, int &nq) {
    q0 = __ldg(a.cu_q + b);
    const int q1 = __ldg(a.cu_q + b + 1);
    nq = q1 - q0;
    const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.T && nq <= kTreeTokens && nq <= __ldg(a.seq_lens + b);
    if (!ok || (a.few && nq > a.few)) nq = 0;
    return ok;
}
// Fills in what depends on the sequence w.b alone.
template <int MODE, int kRows, int kChunk>
__device__ __forceinline__ void set_sequence(const DecodeAttnArgs &a, Walk &w) {
    w.n = keys_of(a, w.b);
    if (MODE == kWindow) {
        const int box = 1 << a.box_shift;
        w.sinks = min(a.sinks, w.n);
        w.from = a.window < w.n ? w.n - a.window : 0;
        w.lead = (int)min((int64_t)(w.sinks + (int64_t)box - 1) & -(int64_t)box, (int64_t)1 << 30);
        w.shift = max(0, (w.from & -box) - w.lead);
        w.from -= w.shift;
        w.n -= w.shift;
    }
    if (MODE == kTree) {
        tokens_of(a, w.b, w.q0, w.nq);
        if (w.nq == 0) w.n = 0;
        w.RT = (w.nq * (a.Hq / a.kv.Hkv) + kRows - 1) / kRows;
        w.HV = w.RT * a.kv.Hkv;
    }
    w.units = (w.n + kChunk - 1) / kChunk;
}
template <int MODE, int kRows, int kChunk>
__device__ __forceinline__ void next_sequence(const DecodeAttnArgs &a, Walk &w) {
    do {
        if (++w.b >= a.B) {
            w.n = w.units = 1;
            return;
        }
        set_sequence<MODE, kRows, kChunk>(a, w);
    } while (w.n == 0);
}

// 4 e4m3 codes, two each of two neighbouring keys (key 0: d, d + 1; key 1: d,
// d + 1) -> the pairs (key 0, key 1) of column d and of column d + 1 as bf16: a
// code's exponent and mantissa bits moved to the bf16 places are its value times
// 2^-120.  Exact, but for the NaN code, which comes out as 480; `most` keeps the
// largest magnitudes' moved bits, by which has_nan() knows one.
__device__ __forceinline__ void e4m3_columns(uint32_t w, uint32_t &lo, uint32_t &hi, uint32_t &most) {
    const uint32_t up = 0x7B807B80u;  // bf16 2^120
    const uint32_t ml = (w << 4) & 0x07F007F0u, mh = (w >> 4) & 0x07F007F0u;
    most = __vimax3_u16x2(most, ml, mh);
    const uint32_t l = ml | ((w << 8) & 0x80008000u);
    const uint32_t h = mh | (w & 0x80008000u);
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(l), "r"(up));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(h), "r"(up));
}
__device__ __forceinline__ bool has_nan(uint32_t most) { return ((most + 0x00100010u) & 0x08000800u) != 0; }
// Which columns of such a word hold a NaN code: bit 0 d, bit 1 d + 1.  live: a
// mask of the keys that exist.
__device__ __forceinline__ uint32_t nan_columns(uint32_t w, uint32_t live) {
    const uint32_t n = ((w & live & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    return (n & 0x00800080u ? 1u : 0u) | (n & 0x80008000u ? 2u : 0u);
}
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
    return r;
}

template <int D, bool FP8, int NT, int MODE>
__global__ void __launch_bounds__(kThreads, (Cfg<D, FP8, NT>::kBlocks))
decode_kernel(const DecodeAttnArgs a, const int HV, const int RT, const __grid_constant__ CUtensorMap map) {
    using C = Cfg<D, FP8, NT>;
    constexpr int S = C::kStages, kChunk = C::kChunk, KG = C::kGroups;
    extern __shared__ uint8_t raw[];
    const uint32_t raw_u = smem_u32(raw);
    uint8_t *base = raw + ((1024 - (raw_u & 1023)) & 1023);
    const uint32_t stage0 = smem_u32(base);
    uint8_t *after = base + S * C::kStage;
    float *exch = reinterpret_cast<float *>(after);
    float2 *ml = reinterpret_cast<float2 *>(after + C::kExch);
    Shared *sm = reinterpret_cast<Shared *>(after + C::kExch + C::kMl);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const DecodeLayout L = decode_layout(C::kRows, D);

    // ---- this block's share: units [u0, u1) of the batch's W
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&sm->full[i], 1);
            mbar_init(&sm->empty[i], kCWarps);
        }
        fence_barrier_init();
        sm->abort = 0;
        sm->bad = 0x7fffffff;
        prefetch_tensormap(&map);
    }
    pdl_trigger();
    const int per = (a.B + kThreads - 1) / kThreads;
    const int s0 = min(a.B, tid * per), s1 = min(a.B, s0 + per);
    int64_t mine = 0;
    int bad = 0x7fffffff;
    // units of a sequence for one tile of rows; kTree: for all its tiles
    auto units_of = [&](int b) {
        if (MODE == kPlain) return (int64_t)((keys_of(a, b) + kChunk - 1) / kChunk);
        Walk w;
        w.b = b;
        set_sequence<MODE, C::kRows, kChunk>(a, w);
        return MODE == kTree ? (int64_t)w.units * w.HV : (int64_t)w.units;
    };
    const int per_unit = MODE == kTree ? 1 : HV;
    for (int b = s0; b < s1; ++b) {
        const int n = keys_of(a, b);
        if (n != __ldg(a.seq_lens + b) && b < bad) bad = b;
        if (MODE == kTree) {
            int q0, nq;
            if (!tokens_of(a, b, q0, nq) && b < bad) bad = b;
        }
        mine += MODE == kPlain ? (n + kChunk - 1) / kChunk : units_of(b);
    }
    int64_t scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) sm->warp_sum[warp] = scan;
    __syncthreads();
    int64_t before = scan - mine, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += sm->warp_sum[w];
        total += sm->warp_sum[w];
    }
    if (bad != 0x7fffffff && blockIdx.x == 0) atomicMin(&sm->bad, bad);
    const int64_t W = total * per_unit;
    const int G = (int)min((int64_t)gridDim.x, W);  // blocks that have a share
    const int g = blockIdx.x;
    const int64_t u0 = g < G ? (int64_t)g * W / G : 0, u1 = g < G ? (int64_t)(g + 1) * W / G : 0;
    if (u0 < u1 && u0 >= before * per_unit && u0 < (before + mine) * per_unit) {
        int64_t at = before * per_unit;
        int b = s0;
        for (;; ++b) {
            const int64_t units = units_of(b) * per_unit;
            if (u0 < at + units) break;
            at += units;
        }
        sm->b0 = b;
        sm->first = u0 - at;
    }
    __syncthreads();

    Join *const join = reinterpret_cast<Join *>(a.workspace + L.join);
    const bool by_pair = join_by_pair(a.B, HV, gridDim.x);
    if (!by_pair && tid == 0) join[g] = Join{0, 0, 0, 0};
    // sequences without keys: zeros
    if (MODE == kTree) {  // (there: no tokens)
        if (by_pair)
            for (int b = g; b < a.B; b += gridDim.x) {
                Walk w;
                w.b = b;
                set_sequence<MODE, C::kRows, kChunk>(a, w);
                for (int i = w.HV + tid; i < HV; i += kThreads) join[b * HV + i] = Join{0, 0, 0, 0};
            }
    } else
    for (int b = g; b < a.B; b += gridDim.x)
        if (keys_of(a, b) == 0) {
            for (int i = tid; i < a.Hq * D / 8; i += kThreads)
                reinterpret_cast<uint4 *>(a.out + b * a.out_stride)[i] = make_uint4(0, 0, 0, 0);
            if (a.lse)
                for (int i = tid; i < a.Hq; i += kThreads) a.lse[(size_t)b * a.Hq + i] = -INFINITY;
            if (by_pair)
                for (int i = tid; i < HV; i += kThreads) join[b * HV + i] = Join{0, 0, 0, 0};
        }

    const int heads = a.Hq / a.kv.Hkv;  // query heads of one key/value head
    Walk w0;
    if (u0 < u1) {
        w0.b = sm->b0;
        set_sequence<MODE, C::kRows, kChunk>(a, w0);
        w0.hv = (int)(sm->first / w0.units);
        w0.j = (int)(sm->first % w0.units);
    }
    const int page_shift = a.kv.page_shift;
    // rows of one copy
    const int box_shift = MODE == kWindow ? a.box_shift : min(page_shift, 6), R = 1 << box_shift;
    // head tiles of a sequence, and those of one key/value head
    auto tiles = [&](const Walk &w) { return MODE == kTree ? w.HV : HV; };
    auto per_head = [&](const Walk &w) { return MODE == kTree ? w.RT : RT; };
    auto rows_of = [&](const Walk &w) { return MODE == kTree ? w.nq * heads : heads; };
    // a key's place in its sequence
    auto place = [&](const Walk &w, int key) { return MODE == kWindow && key >= w.lead ? key + w.shift : key; };
    const int box_bytes = R * D * C::kEs * 2;

    if (warp == kCWarps) {
        // ---------------- producer: one box of pages per lane
        if (u0 < u1) {
            Walk w = w0;
            const int boxes = kChunk >> box_shift;
            auto page_of = [&](const Walk &x) {  // this lane's page of a unit
                const int key = x.j * kChunk + (lane << box_shift);
                int pg = 0;
                if (lane < boxes && key < x.n)
                    pg = __ldg(a.page_table + (size_t)x.b * a.table_stride + (place(x, key) >> page_shift));
                return pg;
            };
            int s = 0;
            uint32_t phase = 1;
            int64_t done = 0;
            int pg = page_of(w);
            bool fresh = true;  // the first unit of a pair (or of the block)
            for (int64_t u = u0; u < u1 && !a.test_no_copies; ++u) {
                const Walk x = w;
                const int my = pg;
                const bool with_q = fresh;
                fresh = false;
                if (++w.j == w.units) {
                    w.j = 0;
                    fresh = true;
                    if (++w.hv == tiles(w)) {
                        w.hv = 0;
                        if (u + 1 < u1) next_sequence<MODE, C::kRows, kChunk>(a, w);
                    }
                }
                if (u + 1 < u1) pg = page_of(w);
                if (!warp_wait_flag(&sm->empty[s], phase, &sm->abort, 1)) break;
                const int key = x.j * kChunk + (lane << box_shift);
                const bool live = lane < boxes && key < x.n;
                const int n_live = __popc(__ballot_sync(0xffffffffu, live));
                const int hk = x.hv / per_head(x), r0 = (x.hv % per_head(x)) * C::kRows;
                const uint32_t st = stage0 + s * C::kStage;
                const uint32_t q_bytes = with_q ? min(C::kRows, rows_of(x) - r0) * D * 2 : 0;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sm->full[s], n_live * (box_bytes + (FP8 ? R * 8 : 0)) + q_bytes);
                    if (with_q && MODE != kTree)
                        bulk_g2s(st + C::kData, a.q + x.b * a.q_stride + (size_t)(hk * heads + r0) * D,
                                 q_bytes, &sm->full[s]);
                }
                __syncwarp();
                if (MODE == kTree && with_q && lane * D * 2 < q_bytes) {  // a row a lane
                    const int r = r0 + lane;
                    bulk_g2s(st + C::kData + lane * D * 2,
                             a.q + (x.q0 + r / heads) * a.q_stride + (size_t)(hk * heads + r % heads) * D, D * 2,
                             &sm->full[s]);
                }
                if (live) {
                    int p = my;
                    if ((unsigned)p >= (unsigned)a.kv.num_pages) {
                        atomicMin(&sm->bad, x.b);
                        p = 0;
                    }
                    const int row = place(x, key) & ((1 << page_shift) - 1);
                    const int64_t ph = (int64_t)p * a.kv.Hkv + hk;
                    tma_load_5d(st + lane * box_bytes, &map, 0, row, 0, 0, (int)ph, &sm->full[s]);
                    if (FP8) {
                        const float *sc = a.kv.scales + ((ph * 2) << page_shift) + row;
                        const uint32_t to = st + C::kData + C::kQ + lane * R * 8;
                        if (page_shift == box_shift) {  // K's and V's are neighbours
                            bulk_g2s(to, sc, R * 8, &sm->full[s]);
                        } else {
                            bulk_g2s(to, sc, R * 4, &sm->full[s]);
                            bulk_g2s(to + R * 4, sc + ((size_t)1 << page_shift), R * 4, &sm->full[s]);
                        }
                    }
                }
                __syncwarp();
                ++done;
                if (++s == S) {
                    s = 0;
                    phase ^= 1;
                }
            }
            // every copy has landed before the block ends
            if (*(volatile int *)&sm->abort)
                for (int64_t i = done > S ? done - S : 0; i < done; ++i)
                    wait_own(&sm->full[i % S], (i / S) & 1);
        }
    } else if (u0 < u1) {
        // ---------------- consumers: keys [16 KG warp, 16 KG (warp + 1)) of each unit
        Walk w = w0;
        const int gq = lane >> 2, t = lane & 3;
        const uint32_t half_b = R * C::kRowB, kv_b = half_b * C::kHalves;
        // this warp's rows, then this lane's row and 16-byte column of the
        // fragment loads (K: row-major; V: transposed)
        uint32_t my_rows[KG];
#pragma unroll
        for (int k = 0; k < KG; ++k) {
            const int row = 16 * (warp * KG + k);
            my_rows[k] = (row >> box_shift) * box_bytes + (row & (R - 1)) * C::kRowB;
        }
        const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8;   // rows 0-7, 8-15, 0-7, 8-15
        const int lcol = lane >> 4;                            // columns 0, 0, 1, 1
        const int swz = C::kRowB == 128 ? (lrow & 7) : ((lrow >> 1) & 3);
        auto frag = [&](uint32_t rows, int col) {  // col: 16-byte column of the row
            const int c = col + lcol;
            return rows + (c / (C::kRowB / 16)) * half_b + lrow * C::kRowB +
                   (((c & (C::kRowB / 16 - 1)) ^ swz) << 4);
        };
        const float base_scale = a.scale * kLog2e;
        int s = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int64_t u = u0; u < u1;) {
            const int todo = (int)min((int64_t)(w.units - w.j), u1 - u);
            const bool starts = w.j == 0, ends = w.j + todo == w.units;
            const int hk = w.hv / per_head(w), r0 = (w.hv % per_head(w)) * C::kRows;
            const int rows = min(C::kRows, rows_of(w) - r0);
            // kWindow: whether a key is seen; two neighbours as masks of 16 bits
            auto seen = [&](int key) { return key < w.sinks || key >= w.from; };
            auto seen_pair = [&](int key) { return (seen(key) ? 0xFFFFu : 0u) | (seen(key + 1) ? 0xFFFF0000u : 0u); };
            float o[NT][D / 16][4], m[NT][2], l[NT][2], sc2[NT][2];
            uint32_t qf[NT][D / 16][2];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                m[i][0] = m[i][1] = -INFINITY;
                l[i][0] = l[i][1] = 0.f;
                sc2[i][0] = sc2[i][1] = base_scale;
#pragma unroll
                for (int d = 0; d < D / 16; ++d)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][d][e] = 0.f;
            }
            for (int c = 0; c < todo; ++c) {
                // (a warp that gave up goes on without waiting or computing:
                // the others may be at the barriers below)
                ok = ok && warp_wait_flag(&sm->full[s], phase, &sm->abort, 2);
                const uint32_t st = stage0 + s * C::kStage;
                if (c == 0 && ok) {
                    // Q^T fragments: head gq (of each group of 8), column pairs
                    const uint8_t *qs = base + s * C::kStage + C::kData;
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const bool live = 8 * i + gq < rows;
                        const uint8_t *row = qs + (8 * i + gq) * D * 2;
                        if (!FP8) {
#pragma unroll
                            for (int d = 0; d < D / 16; ++d) {
                                qf[i][d][0] = live ? *reinterpret_cast<const uint32_t *>(row + d * 32 + t * 4) : 0;
                                qf[i][d][1] = live ? *reinterpret_cast<const uint32_t *>(row + d * 32 + t * 4 + 16) : 0;
                            }
                        } else {
                            // to fp16, scaled by a power of two so that the
                            // head's largest value is in [1, 2): exact but
                            // for values 2^-14 of it and less (off by at
                            // most 2^-25 of it)
                            float x[D / 16][4], most = 0.f;
#pragma unroll
                            for (int d = 0; d < D / 16; ++d) {
                                const uint2 v = live ? *reinterpret_cast<const uint2 *>(row + d * 32 + t * 8)
                                                     : make_uint2(0, 0);
                                x[d][0] = __uint_as_float(v.x << 16);
                                x[d][1] = __uint_as_float(v.x & 0xFFFF0000u);
                                x[d][2] = __uint_as_float(v.y << 16);
                                x[d][3] = __uint_as_float(v.y & 0xFFFF0000u);
#pragma unroll
                                for (int e = 0; e < 4; ++e) most = fmaxf(most, fabsf(x[d][e]));
                            }
                            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
                            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
                            const int e2 = max((int)(__float_as_uint(most) >> 23) - 127, -126);
                            const float down = e2 >= 127 ? 0x1p-127f : __uint_as_float((127 - e2) << 23);
                            const float up = e2 <= -126 ? 0x1p-126f : __uint_as_float((127 + e2) << 23);
#pragma unroll
                            for (int d = 0; d < D / 16; ++d)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const __half2 h = __floats2half2_rn(x[d][2 * e] * down, x[d][2 * e + 1] * down);
                                    qf[i][d][e] = *reinterpret_cast<const uint32_t *>(&h);
                                }
                            // the score's columns are heads 2 t and 2 t + 1
                            sc2[i][0] = base_scale * __shfl_sync(0xffffffffu, up, 8 * t);
                            sc2[i][1] = base_scale * __shfl_sync(0xffffffffu, up, 8 * t + 4);
                        }
                    }
                }
                // keys of this warp's groups
                const int key0 = (w.j + c) * kChunk + 16 * KG * warp;
                const int left = w.n - key0;
                if (left > 0 && ok) {
                    // (two sums in turns: a chain of products into one is
                    // as long as the tensor pipe's latency times D / 16)
                    float sT[KG][NT][4], sU[KG][NT][4];
#pragma unroll
                    for (int k = 0; k < KG; ++k)
#pragma unroll
                        for (int i = 0; i < NT; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e) sT[k][i][e] = sU[k][i][e] = 0.f;
                    if (!FP8) {
#pragma unroll
                        for (int d = 0; d < D / 16; ++d)
#pragma unroll
                            for (int k = 0; k < KG; ++k) {
                                uint32_t k4[4];
                                ldsm4(k4, frag(st + my_rows[k], 2 * d));
#pragma unroll
                                for (int i = 0; i < NT; ++i)
                                    mma16816<true>(d & 1 ? sU[k][i] : sT[k][i], k4, qf[i][d][0], qf[i][d][1]);
                            }
                    } else {
#pragma unroll
                        for (int d = 0; d < D / 16; d += 2)
#pragma unroll
                            for (int k = 0; k < KG; ++k) {
                                uint32_t k4[4];
                                ldsm4(k4, frag(st + my_rows[k], d));
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const uint32_t lo = k4[2 * e], hi = k4[2 * e + 1];
                                    const uint32_t af[4] = {e4m3_pair(lo), e4m3_pair(hi), e4m3_pair(lo >> 16),
                                                            e4m3_pair(hi >> 16)};
#pragma unroll
                                    for (int i = 0; i < NT; ++i)
                                        mma16816<false>(e & 1 ? sU[k][i] : sT[k][i], af, qf[i][d + e][0],
                                                        qf[i][d + e][1]);
                                }
                            }
                    }
                    // this lane's keys gq and gq + 8 of a group
                    float ks[KG][2], vs[KG][2];
                    bool see[KG][2];
#pragma unroll
                    for (int k = 0; k < KG; ++k) {
                        if (FP8) {
                            const int row = 16 * (warp * KG + k);
                            const float *sc = reinterpret_cast<const float *>(base + s * C::kStage + C::kData + C::kQ) +
                                              (row >> box_shift) * R * 2 + (row & (R - 1));
                            ks[k][0] = sc[gq];
                            ks[k][1] = sc[gq + 8];
                            vs[k][0] = sc[R + gq];
                            vs[k][1] = sc[R + gq + 8];
                        }
                        see[k][0] = 16 * k + gq < left;
                        see[k][1] = 16 * k + gq + 8 < left;
                        if (MODE == kWindow) {
                            see[k][0] = see[k][0] && seen(key0 + 16 * k + gq);
                            see[k][1] = see[k][1] && seen(key0 + 16 * k + gq + 8);
                        }
                    }
                    // kTree: the drafted tokens among these keys
                    const int drafted = w.n - w.nq - key0;  // the first one, from this warp's first key on
                    const bool some_drafted = MODE == kTree && drafted < 16 * KG;
                    uint32_t pf[KG][NT][2], pl[KG][NT][2];  // the weights' upper and lower parts
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        float x[KG][4], t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
                        for (int k = 0; k < KG; ++k) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float v = (sT[k][i][e] + sU[k][i][e]) *
                                                (FP8 ? sc2[i][e & 1] * ks[k][e >> 1] : sc2[i][e & 1]);
                                x[k][e] = see[k][e >> 1] ? v : -INFINITY;
                            }
                            if (MODE == kTree && some_drafted) {
#pragma unroll
                                for (int h = 0; h < 2; ++h) {  // this column's row
                                    const int r = min(r0 + 8 * i + 2 * t + h, w.nq * heads - 1);
                                    const uint64_t mask = __ldg(a.tree + w.q0 + r / heads);
#pragma unroll
                                    for (int e = 0; e < 2; ++e) {
                                        const int d = 16 * k + gq + 8 * e - drafted;
                                        if (d >= 0 && !(mask >> (d & 63) & 1)) x[k][2 * e + h] = -INFINITY;
                                    }
                                }
                            }
                            t0 = fmaxf(t0, fmaxf(x[k][0], x[k][2]));
                            t1 = fmaxf(t1, fmaxf(x[k][1], x[k][3]));
                        }
#pragma unroll
                        for (int sh = 4; sh < 32; sh <<= 1) {
                            t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, sh));
                            t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, sh));
                        }
                        // (most units leave every maximum as it is)
                        if (__any_sync(0xffffffffu, t0 > m[i][0] || t1 > m[i][1])) {
                            const float n0 = fmaxf(m[i][0], t0), n1 = fmaxf(m[i][1], t1);
                            const float a0 = n0 == -INFINITY ? 1.f : ex2(m[i][0] - n0);
                            const float a1 = n1 == -INFINITY ? 1.f : ex2(m[i][1] - n1);
                            m[i][0] = n0;
                            m[i][1] = n1;
                            l[i][0] *= a0;
                            l[i][1] *= a1;
#pragma unroll
                            for (int d = 0; d < D / 16; ++d) {
                                o[i][d][0] *= a0;
                                o[i][d][1] *= a1;
                                o[i][d][2] *= a0;
                                o[i][d][3] *= a1;
                            }
                        }
                        const float z0 = m[i][0] == -INFINITY ? 0.f : m[i][0];
                        const float z1 = m[i][1] == -INFINITY ? 0.f : m[i][1];
#pragma unroll
                        for (int k = 0; k < KG; ++k) {
                            x[k][0] = ex2(x[k][0] - z0);
                            x[k][1] = ex2(x[k][1] - z1);
                            x[k][2] = ex2(x[k][2] - z0);
                            x[k][3] = ex2(x[k][3] - z1);
                            l[i][0] += x[k][0] + x[k][2];
                            l[i][1] += x[k][1] + x[k][3];
                            // Weights for the product with v, v's scale with
                            // them; the sum l keeps the unrounded.  For a bf16
                            // cache the sum of two bf16: one alone would add as
                            // much error as the result's own rounding, and the
                            // second product is free (109 us either way for 90
                            // sequences up to 8192 keys).  For fp8 one, which
                            // adds up to 2^-8 of sum p |v| (2.3e-3 instead of
                            // 1.7e-3 relative over random values): there the
                            // work is bound by its instructions, and the second
                            // costs 256 sequences up to 8192 keys 280 -> 287 us,
                            // 64 with 64 heads over 4 69 -> 77.  (As fp16 times a
                            // factor per head that follows the largest weight:
                            // 2^-11, but 289 to 304 and 76 to 84 us.)
                            if (FP8) {
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    x[k][e] = see[k][e >> 1] ? x[k][e] * vs[k][e >> 1] : 0.f;
                            }
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint32_t hi = pack_bf16(x[k][2 * e], x[k][2 * e + 1]);
                                const float r0 = x[k][2 * e] - __uint_as_float(hi << 16);
                                const float r1 = x[k][2 * e + 1] - __uint_as_float(hi & 0xFFFF0000u);
                                pf[k][i][e] = transpose8x8(hi);
                                if (!FP8) pl[k][i][e] = transpose8x8(pack_bf16(r0, r1));
                            }
                        }
                    }
                    uint32_t most = 0;
#pragma unroll
                    for (int k = 0; k < KG; ++k) {
                        const uint32_t vr = st + my_rows[k] + kv_b;
                        if (!FP8) {
                            // keys past the end hold anything: zero v there (0 x NaN)
                            const int rest = left - 16 * k;
                            uint32_t mask0 = 0xFFFFFFFFu, mask1 = 0xFFFFFFFFu;
                            const int k0 = key0 + 16 * k;
                            const bool cut = rest < 16 || (MODE == kWindow && k0 < w.from && k0 + 16 > w.sinks);
                            if (cut) {
                                mask0 = (2 * t < rest ? 0xFFFFu : 0u) | (2 * t + 1 < rest ? 0xFFFF0000u : 0u);
                                mask1 = (2 * t + 8 < rest ? 0xFFFFu : 0u) | (2 * t + 9 < rest ? 0xFFFF0000u : 0u);
                                if (MODE == kWindow) {
                                    mask0 &= seen_pair(k0 + 2 * t);
                                    mask1 &= seen_pair(k0 + 2 * t + 8);
                                }
                            }
                            // a row-block pair (d, d + 8) per 16 columns: the
                            // matrices arrive as (keys 0-7, 8-15) x (d 0-7, 8-15)
#pragma unroll
                            for (int d = 0; d < D / 16; ++d) {
                                uint32_t v4[4];
                                ldsm4_t(v4, frag(vr, 2 * d));
                                uint32_t af[4] = {v4[0], v4[2], v4[1], v4[3]};
                                if (cut) {
                                    af[0] &= mask0;
                                    af[1] &= mask0;
                                    af[2] &= mask1;
                                    af[3] &= mask1;
                                }
#pragma unroll
                                for (int i = 0; i < NT; ++i) {
                                    mma16816<true>(o[i][d], af, pf[k][i][0], pf[k][i][1]);
                                    mma16816<true>(o[i][d], af, pl[k][i][0], pl[k][i][1]);
                                }
                            }
                        } else {
#pragma unroll
                            for (int d = 0; d < D / 16; d += 2) {
                                uint32_t v4[4];
                                ldsm4_t(v4, frag(vr, d));
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    uint32_t af[4];
                                    e4m3_columns(v4[2 * e], af[0], af[1], most);
                                    e4m3_columns(v4[2 * e + 1], af[2], af[3], most);
#pragma unroll
                                    for (int i = 0; i < NT; ++i)
                                        mma16816<true>(o[i][d + e], af, pf[k][i][0], pf[k][i][1]);
                                }
                            }
                        }
                    }
                    // A NaN code of a key that exists makes its column's sums NaN.
                    // (The codes are looked over only where the unit has one,
                    // be it past the sequence's end.  What knowing that costs:
                    // 256 sequences up to 8192 keys 277.8 -> 280.1 us, 64 with
                    // 64 heads over 4 65.9 -> 68.7.)
                    if (FP8 && __any_sync(0xffffffffu, has_nan(most))) {
#pragma unroll
                        for (int k = 0; k < KG; ++k) {
                            const uint32_t vr = st + my_rows[k] + kv_b;
                            const int rest = left - 16 * k - 2 * t;  // this lane's keys 0, 1, 8, 9
                            uint32_t live0 = (rest > 0 ? 0xFFFFu : 0u) | (rest > 1 ? 0xFFFF0000u : 0u);
                            uint32_t live1 = (rest > 8 ? 0xFFFFu : 0u) | (rest > 9 ? 0xFFFF0000u : 0u);
                            if (MODE == kWindow) {
                                live0 &= seen_pair(key0 + 16 * k + 2 * t);
                                live1 &= seen_pair(key0 + 16 * k + 2 * t + 8);
                            }
#pragma unroll
                            for (int d = 0; d < D / 16; d += 2) {
                                uint32_t v4[4];
                                ldsm4_t(v4, frag(vr, d));
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    uint32_t c = nan_columns(v4[2 * e], live0) | nan_columns(v4[2 * e + 1], live1);
                                    c |= __shfl_xor_sync(0xffffffffu, c, 1);
                                    c |= __shfl_xor_sync(0xffffffffu, c, 2);
#pragma unroll
                                    for (int i = 0; i < NT; ++i)
#pragma unroll
                                        for (int x = 0; x < 4; ++x)
                                            if (c >> (x >> 1) & 1) o[i][d + e][x] = __uint_as_float(0x7FFFFFFFu);
                                }
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->empty[s]);
                if (++s == S) {
                    s = 0;
                    phase ^= 1;
                }
            }
            // ---- join the four warps
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int sh = 4; sh < 32; sh <<= 1) {
                    l[i][0] += __shfl_xor_sync(0xffffffffu, l[i][0], sh);
                    l[i][1] += __shfl_xor_sync(0xffffffffu, l[i][1], sh);
                }
            if (gq == 0) {
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    ml[warp * C::kRows + 8 * i + 2 * t] = make_float2(m[i][0], l[i][0]);
                    ml[warp * C::kRows + 8 * i + 2 * t + 1] = make_float2(m[i][1], l[i][1]);
                }
            }
            const int slot = starts ? 1 : 0;
            const int head = tid >> 4, q4 = (tid & 15) * 4;  // reader: 8 heads x 16 float4
#pragma unroll
            for (int i = 0; i < NT; ++i) {
#pragma unroll
                for (int p = 0; p < D / 64; ++p) {
                    // (the barrier also keeps this pass's writes behind the
                    // last one's reads)
                    asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
                    for (int dd = 0; dd < 4; ++dd) {
                        const float(&x)[4] = o[i][4 * p + dd];
                        const int c0 = dd * 16 + (FP8 ? 2 * gq : gq), c1 = c0 + (FP8 ? 1 : 8);
                        float *to = exch + (warp * 8 + 2 * t) * 68;
                        to[c0] = x[0];
                        to[68 + c0] = x[1];
                        to[c1] = x[2];
                        to[68 + c1] = x[3];
                    }
                    asm volatile("bar.sync 1, 128;" ::: "memory");
                    const int r = 8 * i + head;
                    if (r < rows) {
                        float2 v[kCWarps];
                        float top = -INFINITY;
#pragma unroll
                        for (int k = 0; k < kCWarps; ++k) {
                            v[k] = ml[k * C::kRows + r];
                            top = fmaxf(top, v[k].x);
                        }
                        const float z = top == -INFINITY ? 0.f : top;
                        float sum = 0.f;
                        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int k = 0; k < kCWarps; ++k) {
                            const float f = ex2(v[k].x - z);
                            const float4 y = *reinterpret_cast<const float4 *>(exch + (k * 8 + head) * 68 + q4);
                            sum += f * v[k].y;
                            acc.x += f * y.x;
                            acc.y += f * y.y;
                            acc.z += f * y.z;
                            acc.w += f * y.w;
                        }
                        if (starts && ends) {
                            // (kTree: a row that sees nothing gets zeros)
                            const float inv = MODE == kTree && sum == 0.f ? 0.f : 1.f / sum;
                            const int row = MODE == kTree ? w.q0 + (r0 + r) / heads : w.b;
                            const int hq = hk * heads + (MODE == kTree ? (r0 + r) % heads : r0 + r);
                            *reinterpret_cast<uint2 *>(a.out + row * a.out_stride + hq * D + 64 * p + q4) =
                                make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
                            if (a.lse && p == 0 && q4 == 0)
                                a.lse[(size_t)row * a.Hq + hq] = (top + __log2f(sum)) * kLn2;
                        } else {
                            const size_t row = ((size_t)g * 2 + slot) * C::kRows + r;
                            *reinterpret_cast<float4 *>(reinterpret_cast<float *>(a.workspace + L.part) +
                                                        row * D + 64 * p + q4) = acc;
                            if (p == 0 && q4 == 0)
                                reinterpret_cast<float2 *>(a.workspace + L.ml)[row] = make_float2(top, sum);
                        }
                    }
                }
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");  // ml is free again
            if (starts && tid == 0 && (by_pair || !ends)) {
                // the block that holds the pair's last unit
                const int64_t last = u + (w.units - 1);
                const int owner = (int)(((last + 1) * G - 1) / W);
                join[by_pair ? w.b * HV + w.hv : g] = Join{w.b, w.hv, ends ? 0 : owner - g + 1, g};
            }
            u += todo;
            w.j += todo;
            if (w.j == w.units) {
                w.j = 0;
                if (++w.hv == tiles(w)) {
                    w.hv = 0;
                    if (u < u1) next_sequence<MODE, C::kRows, kChunk>(a, w);
                }
            }
        }
    }
    __syncthreads();
    if (tid == 0)
        reinterpret_cast<Err *>(a.workspace + L.err)[g] = Err{sm->abort, sm->bad};
}

// Joins the parts of a pair: blockIdx.x is its record, blockIdx.y has ROWS of
// its rows; GROUPS groups of threads take every GROUPS-th part, then their sums
// are added in order.  Few pairs in many parts (one sequence of 131072 keys: 57
// parts) want many groups, many pairs in two or three parts few blocks.
template <int D, int ROWS, int GROUPS, int MODE>
__global__ void __launch_bounds__(ROWS *GROUPS *D / 4)
decode_join(const DecodeAttnArgs a, int RT, const int tile_rows, const int n_blocks) {
    constexpr int kCols = D / 4, kGroup = ROWS * kCols;
    __shared__ float4 part[GROUPS][kGroup];
    __shared__ float2 sums[GROUPS][ROWS];
    __shared__ int red[2];
    const DecodeLayout L = decode_layout(tile_rows, D);
    const int tid = threadIdx.x;
    pdl_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        // the call's status word, from every block's record
        const Err *err = reinterpret_cast<const Err *>(a.workspace + L.err);
        if (tid == 0) red[0] = 0, red[1] = 0x7fffffff;
        __syncthreads();
        for (int i = tid; i < n_blocks; i += blockDim.x) {
            if (err[i].timeout) atomicMax(&red[0], err[i].timeout);
            if (err[i].bad != 0x7fffffff) atomicMin(&red[1], err[i].bad);
        }
        __syncthreads();
        if (tid == 0) {
            Ctrl *ctrl = reinterpret_cast<Ctrl *>(a.workspace);
            ctrl->status = red[0] ? MOE_ERR_DEVICE_TIMEOUT
                                  : (red[1] != 0x7fffffff ? MOE_ERR_DEVICE_BAD_INDEX : MOE_OK);
            ctrl->detail = red[0] ? red[0] : (red[1] != 0x7fffffff ? red[1] : 0);
        }
    }
    const Join jn = reinterpret_cast<const Join *>(a.workspace + L.join)[blockIdx.x];
    if (jn.parts == 0) return;
    const int heads = a.Hq / a.kv.Hkv;
    int q0 = jn.b, rows = heads;
    if (MODE == kTree) {
        int nq;
        tokens_of(a, jn.b, q0, nq);
        rows = nq * heads;
        RT = (rows + tile_rows - 1) / tile_rows;
    }
    const int hk = jn.hv / RT, r0 = (jn.hv % RT) * tile_rows;
    const int grp = tid / kGroup, in = tid % kGroup, col = in % kCols;
    const int r = blockIdx.y * ROWS + in / kCols;
    const bool live = r < min(tile_rows, rows - r0);
    const float2 *ml = reinterpret_cast<const float2 *>(a.workspace + L.ml);
    const float *pt = reinterpret_cast<const float *>(a.workspace + L.part);
    // the first part is its block's last one, the others are first ones
    auto row_of = [&](int i) { return ((size_t)(jn.first + i) * 2 + (i == 0 ? 1 : 0)) * tile_rows + r; };
    float top = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live)
        for (int i = col; i < jn.parts; i += kCols) top = fmaxf(top, ml[row_of(i)].x);
#pragma unroll
    for (int o = kCols / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (live) {
        const float z = top == -INFINITY ? 0.f : top;
#pragma unroll 4
        for (int i = grp; i < jn.parts; i += GROUPS) {
            const float2 v = ml[row_of(i)];
            const float4 y = *reinterpret_cast<const float4 *>(pt + row_of(i) * D + col * 4);
            const float f = ex2(v.x - z);
            sum += f * v.y;
            acc.x += f * y.x;
            acc.y += f * y.y;
            acc.z += f * y.z;
            acc.w += f * y.w;
        }
    }
    part[grp][in] = acc;
    if (col == 0) sums[grp][in / kCols] = make_float2(sum, 0.f);
    __syncthreads();
    if (grp || !live) return;
    sum = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) {
        const float4 y = part[k][in];
        sum += sums[k][in / kCols].x;
        acc.x += y.x;
        acc.y += y.y;
        acc.z += y.z;
        acc.w += y.w;
    }
    const float inv = MODE == kTree && sum == 0.f ? 0.f : 1.f / sum;
    const int row = MODE == kTree ? q0 + (r0 + r) / heads : jn.b;
    const int hq = hk * heads + (MODE == kTree ? (r0 + r) % heads : r0 + r);
    *reinterpret_cast<uint2 *>(a.out + row * a.out_stride + hq * D + col * 4) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    if (a.lse && col == 0) a.lse[(size_t)row * a.Hq + hq] = (top + __log2f(sum)) * kLn2;
}

// Groups of 8 heads in a tile.  More than 16 heads are several tiles, which read
// the cache again, mostly from L2: one tile of 32 needs the registers of a
// whole SM (64 sequences up to 8192 keys, 64 heads over 2: 108 us for fp8 and
// 110 for bf16 instead of 74 and 87).
int tiles_of(int G) { return G <= 8 ? 1 : 2; }

template <int D, bool FP8, int NT, int MODE>
cudaError_t run(const DecodeAttnArgs &a, int sms, cudaStream_t s) {
    using C = Cfg<D, FP8, NT>;
    CUtensorMap map;
    const int page = 1 << a.kv.page_shift, R = MODE == kWindow ? 1 << a.box_shift : page < 64 ? page : 64;
    const size_t row_b = (size_t)D * C::kEs;
    const uint64_t dims[5] = {(uint64_t)C::kRowB / C::kEs, (uint64_t)page, (uint64_t)C::kHalves, 2,
                              (uint64_t)a.kv.num_pages * a.kv.Hkv};
    const uint64_t strides[4] = {row_b, (uint64_t)C::kRowB, page * row_b, 2 * page * row_b};
    const uint32_t box[5] = {(uint32_t)C::kRowB / C::kEs, (uint32_t)R, (uint32_t)C::kHalves, 2, 1};
    if (!encode_tensor_map(&map, FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
                    a.kv.data, dims, strides, box,
                    C::kRowB == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
        return cudaErrorInvalidValue;
    // rows of a key/value head (kTree: at most), tiles of them
    const int tokens = MODE != kTree ? 1 : a.few ? a.few : a.T < kTreeTokens ? a.T : kTreeTokens;
    const int G = a.Hq / a.kv.Hkv * tokens;
    const int RT = (G + C::kRows - 1) / C::kRows, HV = a.kv.Hkv * RT;
    // no more blocks than units could exist
    int64_t keys = (int64_t)a.table_stride * page;
    if (MODE == kWindow) keys = std::min(keys, (int64_t)a.window + a.sinks + 2 * R);
    const int64_t units = (int64_t)a.B * HV * ((keys + C::kChunk - 1) / C::kChunk);
    int grid = C::kBlocks * sms < kMaxGrid ? C::kBlocks * sms : kMaxGrid;
    if (units < grid) grid = (int)units;
    auto fn = decode_kernel<D, FP8, NT, MODE>;
    static SmemOnce once;
    cudaError_t err = once.set(reinterpret_cast<const void *>(fn), C::kSmem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    err = cudaLaunchKernelEx(&cfg, fn, a, HV, RT, map);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cj = {};
    const bool by_pair = join_by_pair(a.B, HV, grid);
    const int rows = by_pair ? 1 : 4, groups = by_pair ? 16 : 4;
    cj.gridDim = dim3(by_pair ? a.B * HV : grid, C::kRows / rows);
    cj.blockDim = dim3(rows * groups * D / 4);
    cj.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cj.attrs = at;
    cj.numAttrs = 1;
    return by_pair ? cudaLaunchKernelEx(&cj, decode_join<D, 1, 16, MODE>, a, RT, (int)C::kRows, grid)
                   : cudaLaunchKernelEx(&cj, decode_join<D, 4, 4, MODE>, a, RT, (int)C::kRows, grid);
}

template <int MODE, int D, bool FP8>
cudaError_t pick(const DecodeAttnArgs &a, int rows, int sms, cudaStream_t s) {
    return tiles_of(rows) == 1 ? run<D, FP8, 1, MODE>(a, sms, s) : run<D, FP8, 2, MODE>(a, sms, s);
}
// rows: of a key/value head, at most
template <int MODE>
cudaError_t launch(const DecodeAttnArgs &a, int rows, cudaStream_t s) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const int sms = tc_grid(dev);
    if (sms < 1) return cudaErrorInvalidDevice;
    const bool fp8 = a.cache_type == MOE_KV_FP8;
    if (a.D == 128) return fp8 ? pick<MODE, 128, true>(a, rows, sms, s) : pick<MODE, 128, false>(a, rows, sms, s);
    return fp8 ? pick<MODE, 64, true>(a, rows, sms, s) : pick<MODE, 64, false>(a, rows, sms, s);
}

}  // namespace
}  // namespace moe
