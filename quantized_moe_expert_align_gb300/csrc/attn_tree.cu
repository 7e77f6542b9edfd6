// attn_tree.cu -- attention of drafted tokens over the paged cache on the tensor
// cores.
//
// A row is one (drafted token, query head of the group) pair; row tiles have 128
// of them, key tiles 128 keys.  Every cached byte is used for up to 256 rows,
// 2 multiply-adds each a value: HBM bounds the few-token trees, the tensor pipe
// and the softmax (128 exponentials a key and row tile) the large ones.  The
// products are those of the prompts (attn_prefill.cuh): S_t = Q_t K_j^T and
// O_t += P_t V_j with P_t over S_t in tensor memory, two row tiles t in turns, one
// warp issuing each one's products, one thread a softmax row with a reference
// that is raised when the maximum exceeds it by 2^8.
//  * 129 to 256 rows: the two row tiles share every key tile ("shared").
//  * Up to 128 rows: both warpgroups have the same rows, each half of a key tile's
//    keys (a maximum of both is exchanged, the reference is one); the scores of the
//    next key tile are made under the softmax of this one, in the tensor memory that
//    the second row tile has no use for.
//  * More rows: blocks of 256, which read the keys again, mostly from L2.
// The key tiles of the whole batch, in order, are shared out evenly over one block
// per SM; a range cut by a block's end is joined by a second kernel, in key order.
//
// Measured, 32 sequences of 8192 keys, 32 heads of 128 over 4, 16 tokens: bf16 102 us
// (5.3 TB/s; the rest is start, joins and ends of ranges), fp8 85; 64 tokens
// (512 rows) over fp8 278 us (990 TFLOP/s).  64 sequences of 4096 keys, 64 heads over
// 8, 16 tokens: bf16 183 us (5.9 TB/s), fp8 160 (3.5 TB/s: not the bytes but the way
// from scores over weights to products, some 2200 cycles a key tile of which the
// exponentials are 512).  What all warps run in turn counts too: this code is large, and
// a register spilled in the softmax costs a fifth.
//
// A bf16 cache is copied page by page into the swizzled operand tiles.  An fp8
// cache is used as it is for the scores: a row of Q, times a power of two, is the
// sum of two rows of e4m3 numbers, both multiplied with the codes (exact, but that
// a value below 2^-9 of its row's largest is off by up to 2^-17 of it), which takes
// as long as one product of 16-bit numbers.  Its scales multiply the scores in
// fp32.  Four warps turn V into fp16, code times scale times a power of two that
// follows the largest scale met so far (2^-11 for the scale, 2^-11 for the value,
// and 2^-25 times that power of two where a value is smaller than 2^-14 of it; where
// it grows, the sums are scaled down like where a reference grows).  The weights are
// fp16 too (2^-11), 2^6-fold, so that those below 2^-20 of the reference's lose bits.
// (The scales of V in the weights, as fp32 products in the softmax, cost 5% when that
// was tried: one more value a key that every softmax thread loads from shared memory.)
#include <type_traits>

#include "attn_tc.cuh"
#include "gemm_tc.h"

namespace moe {
namespace {

using namespace attn;

constexpr int kTile = 128;       // rows of a row tile
constexpr int kM = 2;            // row tiles in turns
constexpr int kKeys = 128;       // keys of a key tile
constexpr int kConvKeys = 32;    // keys that a converting warp has of a key tile
constexpr float kSlack = 8.f;    // a row's maximum may exceed its reference by this
constexpr int kMaxGrid = 160;    // blocks at most
constexpr int kParts = 2;        // in which a key tile's weights come
constexpr int kScaleBufs = 8;    // key tiles whose scales are held
constexpr int kSharedBytes = 3 << 10;  // barriers and what the warps tell each other

// Rows of a sequence's key/value head up to which small tiles have them where a batch
// is in two launches; bytes up to which small tiles may read all of a batch.
constexpr int kFewRows = 16;
constexpr double kFewBytes = 256 << 20;

// Items of at least this many key tiles run shared row tiles half a round apart.
constexpr int kApart = 4;

// Warps: two softmax warpgroups; one warp per row tile issuing products, one
// copying, one clearing (bf16) or copying V's codes (fp8: one warp alone takes
// 3300 cycles a key tile to issue its copies, the bytes 1400); for fp8 a warpgroup
// that converts.
constexpr int kMmaWarp = 8, kLoadWarp = 10, kFixWarp = 11, kConvWarp = 12;

template <int D, bool FP8>
struct Cfg {
    static constexpr int kThreads = FP8 ? 512 : 384;
    // Up to 128 rows of heads of 128 over fp8 the softmax warps' chain of waits is what a
    // key tile takes, so these look ahead at the barriers (a wait takes some 200 cycles
    // though its phase be over), poll where the halves meet, and Q is in tensor memory:
    // 64 sequences of 4096 keys, 64 heads over 8, 189 -> 166 us for 16 tokens, 177 -> 159
    // for 8.  Elsewhere it costs: heads of 64 81 -> 84, bf16 8 x 1000 keys 19.8 -> 21.4.
    static constexpr bool kQuick = FP8 && D == 128;
    // The launch's registers a thread (128 or 168), shared out anew.
    static constexpr int kRoleRegs = FP8 ? 64 : 72, kSoftmaxRegs = FP8 ? 192 : 216;
    static_assert((kThreads - 256) * kRoleRegs + 256 * kSoftmaxRegs <= kThreads * (FP8 ? 128 : 168), "register split");
    static constexpr int kQB = kTile * D * 2, kKvB = kKeys * D * 2;  // a Q tile, an operand tile of K or V
    // Rings: operand tiles (bf16: K and V; fp8: V), tiles of K's and of V's codes.
    static constexpr int kOps = FP8 ? (D == 128 ? 2 : 4) : (D == 128 ? 5 : 8);
    static constexpr int kKs = FP8 ? (D == 128 ? 3 : 4) : 1, kKB = kKeys * D;
    // (the first row tile's roles cannot signal the second's twice before it has looked
    // once: that many key tiles fill the ring of K)
    static_assert(FP8 ? kKs <= kApart : kOps <= 2 * kApart, "see kApart");
    static constexpr int kRaw = FP8 ? (D == 128 ? 2 : 4) : 1;
    static constexpr size_t kOpAt = (size_t)kM * kQB, kKAt = kOpAt + (size_t)kOps * kKvB;
    static constexpr size_t kRawAt = kKAt + (FP8 ? (size_t)kKs * kKB : 0);
    static constexpr size_t kSharedAt = kRawAt + (FP8 ? (size_t)kRaw * kKB : 0);
    // fp8: of kScaleBufs key tiles the scales of K and of V, [2][kKeys]
    static constexpr size_t kScalesAt = kSharedAt + kSharedBytes;
    static constexpr size_t kSmem = kScalesAt + (FP8 ? kScaleBufs * 2 * kKeys * 4 : 0);
    static_assert(kSmem > 114 * 1024 && kSmem <= 227 * 1024, "one block per SM: all of tensor memory is its own");
};

// Some key tiles of one block of rows.
struct Item {
    int32_t q0, nq, nk;       // the sequence's first row, drafted tokens, keys
    int32_t tok0, hk, h0, heads;  // first token of the rows; key/value head; first query head and their number
    int32_t shared;           // two row tiles share the key tiles
    int32_t j0, tiles;        // key tiles
    int32_t slot;             // place for its sums, -1: all of the keys
    int32_t done, b;
};
// A range of keys in parts: its rows (as in Item), the blocks first .. first +
// parts - 1 that have them.
struct __align__(16) Join {
    int32_t parts, first, q0, nq;
    int32_t tok0, h0, heads, tiles;  // row tiles
};
struct Err {
    int32_t timeout, bad;
};
struct TreeLayout {
    size_t err, join, ml, sums, total;
};
__host__ __device__ inline TreeLayout tree_layout(int D) {
    TreeLayout l;
    l.err = 256;
    l.join = l.err + kMaxGrid * sizeof(Err);
    l.ml = l.join + kMaxGrid * sizeof(Join);
    const size_t rows = (size_t)2 * kMaxGrid * kM * kTile;
    l.sums = (l.ml + rows * 8 + 255) / 256 * 256;
    l.total = l.sums + rows * D * 4;
    return l;
}
// Place of a part's four columns c .. c + 3 of row r of row tile t.
__host__ __device__ inline size_t part_at(int slot, int t, int c, int r, int D) {
    return ((((size_t)slot * kM + t) * (D / 4) + c / 4) * kTile + r) * 4;
}
// Query heads and tokens of a row tile, for groups of G heads.
__host__ __device__ inline int tile_heads(int G) { return G < kTile ? G : kTile; }
__host__ __device__ inline int tile_tokens(int G) { return kTile / tile_heads(G); }

struct Shared {
    uint64_t q_full[kM], q_ready[kM], q_empty[kM], op_full[8], op_empty[8], raw_full[4], raw_empty[4];
    uint64_t k_full[4], k_empty[4], sc_ready[kScaleBufs], sc_empty[kScaleBufs], s_full[kM], p_ready[kM][kParts], o_done[kM], offset;
    // (a key tile in turn; items by number)
    uint64_t s_split[2], p_split[2], o_split[2], exchange, item_done[kM][4];
    union {  // bf16; fp8
        uint64_t tail[8], sc_full[kScaleBufs];
    };
    uint64_t item_full[2], item_empty[2], finished;
    uint32_t tmem;
    int abort, bad;
    int expo[kScaleBufs];   // exponents of the largest scale so far, per key tile
    int b0;                 // the sequence of this block's first key tile
    int64_t first;          // and that tile's index among the sequence's
    int64_t warp_sum[16];
    Item item[2];
    // up to 128 rows: the maxima of a key tile's halves, then the sums of the weights
    float halves[2][2][kTile];
};
static_assert(kScaleBufs == 8, "as many as of tail");
static_assert(sizeof(Shared) <= kSharedBytes, "shared block");

// What a sequence has to do.
struct Seq {
    int q0, nq, nk, tiles, RB, HV;  // blocks of rows per head tile, in all
};
// (REST: of more than a.few tokens)
template <bool REST>
__device__ __forceinline__ bool seq_of(const DecodeAttnArgs &a, int b, int tpt, int HT, Seq &s) {
    const int64_t room = min((int64_t)a.table_stride << a.kv.page_shift, (int64_t)1 << 30);
    s.q0 = __ldg(a.cu_q + b);
    const int q1 = __ldg(a.cu_q + b + 1);
    s.nk = __ldg(a.seq_lens + b);
    s.nq = q1 - s.q0;
    const bool ok = s.q0 >= 0 && q1 >= s.q0 && q1 <= a.T && s.nq <= kTreeTokens && s.nk >= 0 && s.nk <= room &&
                    s.nq <= s.nk;
    if (!ok || (REST && s.nq <= a.few)) s.nq = 0;
    s.tiles = s.nq ? (s.nk + kKeys - 1) / kKeys : 0;
    s.RB = (s.nq + kM * tpt - 1) / (kM * tpt);
    s.HV = a.kv.Hkv * HT * s.RB;
    return ok;
}

// 4 e4m3 codes of neighbouring columns -> two pairs of fp16
__device__ __forceinline__ uint2 e4m3_f16(uint32_t w) {
    uint2 r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r.x) : "h"((uint16_t)w));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r.y) : "h"((uint16_t)(w >> 16)));
    return r;
}
// Two numbers to e4m3 (the first in the low byte), and what that leaves of them.
__device__ __forceinline__ uint32_t take_e4m3(float2 &x) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(x.y), "f"(x.x));
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    x.x -= v.x;
    x.y -= v.y;
    return c;
}
// 2^e, -127 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(e > -127 ? (uint32_t)(e + 127) << 23 : 0x00400000u); }
// fp16 weights are 2^kShift-fold, at most 2^8 (the slack) times this.
constexpr int kShift = 6;
// Codes [key][d] as a K-major operand, rows of 64 bytes with 64-byte swizzling.
__device__ __forceinline__ uint64_t sdesc_k_sw64(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)1 << 16 | (uint64_t)(512u >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)4 << 61;
}
__device__ __forceinline__ void mma_e4m3_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// A in tensor memory, a row a lane and four codes a column.
__device__ __forceinline__ void mma_e4m3_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

template <int D, bool FP8, bool REST>
__global__ void __launch_bounds__((Cfg<D, FP8>::kThreads), 1)
tree_kernel(const DecodeAttnArgs a, const int HT, const __grid_constant__ CUtensorMap map_q,
            const __grid_constant__ CUtensorMap map_kv) {
    using C = Cfg<D, FP8>;
    constexpr int S = C::kOps, kHalves = D / 64, kThreads = C::kThreads;
    constexpr uint32_t kQHalf = kTile * 128, kKvHalf = kKeys * 128;  // 64 columns of a tile
    // (aligned for the swizzle; there is no room to align it by hand)
    extern __shared__ __align__(1024) uint8_t raw[];
    uint8_t *const base = raw;
    uint8_t *op_base = base + C::kOpAt, *k_base = base + C::kKAt, *raw_base = base + C::kRawAt;
    Shared *sm = reinterpret_cast<Shared *>(base + C::kSharedAt);
    float *scales = reinterpret_cast<float *>(base + C::kScalesAt);
    const uint32_t q_smem = smem_u32(base), op_smem = smem_u32(op_base);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int tid = threadIdx.x, g = blockIdx.x;
    const int G = a.Hq / a.kv.Hkv, Gt = tile_heads(G), tpt = tile_tokens(G);
    const TreeLayout L = tree_layout(D);

    if (warp == kMmaWarp) tmem_alloc(&sm->tmem, 512);
    if (tid == 0) {
        for (int t = 0; t < kM; ++t) {
            mbar_init(&sm->q_full[t], 1);
            mbar_init(&sm->q_ready[t], 4);
            mbar_init(&sm->q_empty[t], 1);
            mbar_init(&sm->s_full[t], 1);
            for (int h = 0; h < kParts; ++h) mbar_init(&sm->p_ready[t][h], 4);
            mbar_init(&sm->o_done[t], 1);
            mbar_init(&sm->s_split[t], 1);
            mbar_init(&sm->p_split[t], 8);
            mbar_init(&sm->o_split[t], 1);
            for (int i = 0; i < 4; ++i) mbar_init(&sm->item_done[t][i], 1);
            mbar_init(&sm->item_full[t], 1);
            mbar_init(&sm->item_empty[t], FP8 ? 15 : 11);  // the warps that take items
        }
        for (int i = 0; i < 8; ++i) {
            mbar_init(&sm->op_full[i], FP8 ? 4 : 1);
            mbar_init(&sm->op_empty[i], kM);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sm->raw_full[i], 1);
            mbar_init(&sm->raw_empty[i], 4);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sm->k_full[i], 1);
            mbar_init(&sm->k_empty[i], kM);
        }
        for (int i = 0; i < kScaleBufs; ++i) {
            mbar_init(&sm->sc_full[i], 1);
            mbar_init(&sm->sc_ready[i], 4);
            mbar_init(&sm->sc_empty[i], 8);
        }
        mbar_init(&sm->exchange, 8);
        mbar_init(&sm->offset, 4);
        mbar_init(&sm->finished, kM);
        fence_barrier_init();
        sm->abort = 0;
        sm->bad = 0x7fffffff;
        prefetch_tensormap(&map_q);
        prefetch_tensormap(&map_kv);
    }
    pdl_trigger();

    // ---- this block's share: key tiles [u0, u1) of the batch's W
    const int per = (a.B + kThreads - 1) / kThreads;
    const int s0 = min(a.B, tid * per), s1 = min(a.B, s0 + per);
    int64_t mine = 0;
    int bad = 0x7fffffff;
    for (int b = s0; b < s1; ++b) {
        Seq s;
        if (!seq_of<REST>(a, b, tpt, HT, s) && b < bad) bad = b;
        mine += (int64_t)s.tiles * s.HV;
    }
    int64_t scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) sm->warp_sum[warp] = scan;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int64_t before = scan - mine, W = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += sm->warp_sum[w];
        W += sm->warp_sum[w];
    }
    if (bad != 0x7fffffff && g == 0) atomicMin(&sm->bad, bad);
    const int NG = (int)min((int64_t)gridDim.x, W);  // blocks that have a share
    const int64_t u0 = g < NG ? (int64_t)g * W / NG : 0, u1 = g < NG ? (int64_t)(g + 1) * W / NG : 0;
    if (u0 < u1 && u0 >= before && u0 < before + mine) {
        int64_t at = before;
        int b = s0;
        for (;; ++b) {
            Seq s;
            seq_of<REST>(a, b, tpt, HT, s);
            const int64_t n = (int64_t)s.tiles * s.HV;
            if (u0 < at + n) break;
            at += n;
        }
        sm->b0 = b;
        sm->first = u0 - at;
    }
    // (its address is 0; anything else is reported like a wait that gave up, and so
    // is shared memory that does not start where it should)
    if (tid == 0 && (sm->tmem != 0 || (q_smem & 1023))) sm->abort = 20;
    __syncthreads();
    constexpr uint32_t s_col = 0, o_col = kM * kKeys;
    static_assert(kM * (kKeys + D) <= 512, "tensor memory");
    // kQuick: both terms of Q, where the second row tile's sums would be (its
    // codes are read once a product from there, not from shared memory, whose bandwidth
    // the products, copies and conversions share).
    constexpr uint32_t q_col = o_col + D;

    auto take = [&](uint32_t n, Item &it) {
        if (!warp_wait_flag(&sm->item_full[n & 1], (n >> 1) & 1, &sm->abort, 1)) return false;
        it = sm->item[n & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->item_empty[n & 1]);
        return it.done == 0;
    };
    auto run_apart = [&](const Item &it) { return it.shared && it.tiles >= kApart; };
    const int page_shift = a.kv.page_shift, page_mask = (1 << page_shift) - 1;
    const int box_shift = min(page_shift, 7), R = 1 << box_shift;  // rows of one copy
    const int chunks = kKeys >> box_shift;
    // a copying lane's page of a key tile: that of its rows, chunk lane % chunks
    auto page_of = [&](int b, int j, int nk) {
        const int key = j * kKeys + ((lane % chunks) << box_shift);
        return key < nk ? __ldg(a.page_table + (size_t)b * a.table_stride + (key >> page_shift)) : 0;
    };
    // (after a give-up) nothing of a copying warp's may still be in flight
    auto land = [&]() {
        if (*(volatile int *)&sm->abort) {
            const long long t0 = clock64();
            while (clock64() - t0 < (1ll << 24)) __nanosleep(1000);
        }
    };

    // Both tiles of Q for item number n, by the second copying (or the clearing)
    // warp: the first one goes on with the item's keys, whose stages are free
    // sooner than the last item's Q.
    auto load_q = [&](const Item &it, uint32_t n) {
        for (int t = 0; t < kM; ++t) {
            if (!warp_wait_flag(&sm->q_empty[t], (n & 1) ^ 1, &sm->abort, 4)) return false;
            if (lane == 0) {
                mbar_arrive_expect_tx(&sm->q_full[t], (uint32_t)(Gt * tpt) * D * 2);
                for (int h = 0; h < kHalves; ++h)
                    tma_load_4d(base + t * C::kQB + h * kQHalf, &map_q, 0, it.h0,
                                it.q0 + it.tok0 + (it.shared ? t * tpt : 0), h, &sm->q_full[t]);
            }
            __syncwarp();
        }
        return true;
    };

    if (warp >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRoleRegs));
        if (warp == kLoadWarp) {
            // ---------------- copies, and the items for everyone
            Join *const join = reinterpret_cast<Join *>(a.workspace + L.join);
            if (lane == 0) join[g].parts = 0;
            __syncwarp();
            Seq sq = {};
            int b = 0, hv = 0, j = 0;
            if (u0 < u1) {
                b = sm->b0;
                seq_of<REST>(a, b, tpt, HT, sq);
                hv = (int)(sm->first / sq.tiles);
                j = (int)(sm->first % sq.tiles);
            }
            int pg = u0 < u1 ? page_of(b, j, sq.nk) : 0;
            uint32_t n = 0, op = 0, kt = 0;
            bool ok = true;
            int64_t u = u0;
            for (;; ++n) {
                Item it;
                it.done = u >= u1;
                if (!it.done) {
                    const int left = (int)min((int64_t)(sq.tiles - j), u1 - u);
                    const bool starts = j == 0, ends = j + left == sq.tiles;
                    const int rest = hv % (HT * sq.RB), ht = rest / sq.RB, rb = rest % sq.RB;
                    it.q0 = sq.q0;
                    it.nq = sq.nq;
                    it.nk = sq.nk;
                    it.tok0 = rb * kM * tpt;
                    it.hk = hv / (HT * sq.RB);
                    it.h0 = it.hk * G + ht * Gt;
                    it.heads = min(Gt, G - ht * Gt);
                    it.shared = sq.nq - it.tok0 > tpt;
                    it.j0 = j;
                    it.tiles = left;
                    it.b = b;
                    it.slot = starts && ends ? -1 : 2 * g + (starts ? 1 : 0);
                    if (starts && !ends && lane == 0) {
                        // up to the block that holds the range's last tile
                        const int owner = (int)(((u + sq.tiles) * NG - 1) / W);
                        join[g] = Join{owner - g + 1, g, it.q0, it.nq, it.tok0, it.h0, it.heads, it.shared ? 2 : 1};
                    }
                }
                if (!warp_wait_flag(&sm->item_empty[n & 1], ((n >> 1) & 1) ^ 1, &sm->abort, 2)) break;
                if (lane == 0) {
                    sm->item[n & 1] = it;
                    mbar_arrive(&sm->item_full[n & 1]);
                }
                __syncwarp();
                if (it.done) break;
                const int b_now = b;
                const int64_t head = (int64_t)it.hk;
                // where the next item starts
                u += it.tiles;
                j += it.tiles;
                if (j == sq.tiles) {
                    j = 0;
                    if (++hv == sq.HV) {
                        hv = 0;
                        if (u < u1)
                            do {
                                ++b;
                                seq_of<REST>(a, b, tpt, HT, sq);
                            } while (sq.tiles == 0);
                    }
                }
                for (int i = 0; i < it.tiles && ok && !a.test_no_copies; ++i) {
                    const int key0 = (it.j0 + i) * kKeys;
                    const int key = key0 + ((lane % chunks) << box_shift);
                    const bool live = key < it.nk;
                    int p = pg;
                    if (live && (unsigned)p >= (unsigned)a.kv.num_pages) {
                        atomicMin(&sm->bad, b_now);
                        p = 0;
                    }
                    // (the next tile's page is fetched while this one's copies wait)
                    if (i + 1 < it.tiles)
                        pg = page_of(b_now, it.j0 + i + 1, it.nk);
                    else if (u < u1)
                        pg = page_of(b, j, sq.nk);
                    const int64_t ph = (int64_t)p * a.kv.Hkv + head;
                    const int n_live = min(kKeys, it.nk - key0);  // keys
                    if (!FP8) {
                        const int copied = min(kKeys, (n_live + R - 1) & -R);  // rows that are copied
                        for (int kv = 0; kv < 2; ++kv) {
                            const uint32_t s = op % S, par = (op / S) & 1;
                            ok = ok && warp_wait_flag(&sm->op_empty[s], par ^ 1, &sm->abort, 3);
                            if (!ok) break;
                            // values past the sequence's end are cleared before they are used
                            uint64_t *bar = kv && n_live < kKeys ? &sm->tail[s] : &sm->op_full[s];
                            if (lane == 0) mbar_arrive_expect_tx(bar, copied * D * 2);
                            __syncwarp();
                            if (live && lane < chunks * kHalves) {
                                const int h = lane / chunks;
                                tma_load_4d(op_base + s * C::kKvB + h * kKvHalf + ((lane % chunks) << box_shift) * 128,
                                            &map_kv, 0, key & page_mask, h, (int)(ph * 2 + kv), bar);
                            }
                            __syncwarp();
                            ++op;
                        }
                    } else {
                        // K's codes and both scales
                        const int copied = min(kKeys, (n_live + R - 1) & -R);
                        const uint32_t sb = kt % kScaleBufs, s = kt % C::kKs;
                        ok = warp_wait_flag(&sm->k_empty[s], ((kt / C::kKs) & 1) ^ 1, &sm->abort, 3);
                        ok = ok && warp_wait_flag(&sm->sc_empty[sb], ((kt / kScaleBufs) & 1) ^ 1, &sm->abort, 18);
                        if (!ok) break;
                        if (lane < 2)
                            mbar_arrive_expect_tx(lane ? &sm->sc_full[sb] : &sm->k_full[s], lane ? copied * 8 : copied * D);
                        __syncwarp();
                        const int c = lane % chunks, row = key & page_mask;
                        if (live && lane < chunks)
                            tma_load_3d(k_base + s * C::kKB + c * R * D, &map_kv, 0, row, (int)(ph * 2),
                                        &sm->k_full[s]);
                        if (live && lane < 2 * chunks) {  // scales of K, then of V
                            const int kv = lane >= chunks;
                            bulk_g2s(smem_u32(scales + (sb * 2 + kv) * kKeys + c * R),
                                     a.kv.scales + (((ph * 2 + kv) << page_shift) + row), R * 4, &sm->sc_full[sb]);
                        }
                        __syncwarp();
                        ++kt;
                    }
                }
                if (!ok) break;
            }
            land();
        } else if (warp < kLoadWarp) {
            // ---------------- products of row tile t
            auto products = [&](auto tile) {
                constexpr int t = decltype(tile)::value;
                const uint64_t qd = sdesc_k_sw128(q_smem) + ((t * C::kQB) >> 4), k_desc = sdesc_k_sw128(op_smem);
                const uint64_t v_desc = sdesc_mn_sw128(op_smem, kKvHalf);
                // (e4m3 operands, kind::f8f6f4, have the format number of fp16 ones)
                constexpr uint32_t kIdS = FP8 ? idesc_f16_m128(kKeys) : idesc_bf16(kKeys, false);
                constexpr uint32_t kIdO = FP8 ? idesc_f16_m128(D) | 1u << 16 : idesc_bf16(D, true);
                const uint64_t c_desc = D == 128 ? sdesc_k_sw128(smem_u32(k_base)) : sdesc_k_sw64(smem_u32(k_base));
                constexpr uint32_t s_t = s_col + t * kKeys, o_t = o_col + t * D;
                uint32_t off_ph = 0;
                uint32_t tile0 = 0, shared0 = 0;  // key tiles of the items before, and of those shared
                uint32_t split_ph = 0;            // parities of p_split
                bool before_shared = false;       // the item before
                Item it;
                bool ok = true;
                // Waits for K (part 0) or V (1) of key tile number i: its stage, which
                // comes back with the barrier that frees it.
                auto wait_tile = [&](uint32_t i, int part, uint64_t *&free) {
                    uint32_t s;
                    if (FP8 && part == 0) {
                        s = i % C::kKs;
                        ok = ok && warp_wait_flag(&sm->k_full[s], (i / C::kKs) & 1, &sm->abort, 5);
                        free = &sm->k_empty[s];
                    } else {
                        const uint32_t at = FP8 ? i : 2 * i + part;
                        s = at % S;
                        ok = ok && warp_wait_flag(&sm->op_full[s], (at / S) & 1, &sm->abort, 5);
                        free = &sm->op_empty[s];
                    }
                    tc_fence_after();
                    return s;
                };
                // Scores of key tile i of all into tensor memory from `to` on.
                auto scores = [&](uint32_t i, uint32_t to, uint64_t *full, bool last, auto q_in_tmem) {
                    uint64_t *k_free;
                    const uint32_t k = wait_tile(i, 0, k_free);
                    if (!ok) return;
                    if (elect_one()) {
                        if (FP8) {
                            // both terms of Q: tiles of their own, or (heads of 64) the
                            // two halves of a row
                            const uint64_t kd = c_desc + ((k * C::kKB) >> 4);
#pragma unroll
                            for (int x = 0; x < 2 * (D / 32); ++x) {
                                const uint32_t term = x / (D / 32), in = x % (D / 32) * 32;
                                if (C::kQuick && decltype(q_in_tmem)::value)
                                    mma_e4m3_ts(to, q_col + (term * D + in) / 4, kd + (in >> 4), kIdS, x > 0);
                                else
                                    mma_e4m3_ss(to, qd + ((term * (D == 128 ? kQHalf : 64u) + in) >> 4), kd + (in >> 4),
                                                kIdS, x > 0);
                            }
                        } else {
                            const uint64_t kd = k_desc + ((k * C::kKvB) >> 4);
#pragma unroll
                            for (int x = 0; x < D / 16; ++x) {
                                const uint32_t in = (x & 3) * 32;
                                mma_bf16_ss(to, qd + (((x >> 2) * kQHalf + in) >> 4),
                                            kd + (((x >> 2) * kKvHalf + in) >> 4), kIdS, x > 0);
                            }
                        }
                        tc_commit(full);
                        tc_commit(k_free);
                        if (last) tc_commit(&sm->q_empty[t]);
                    }
                    __syncwarp();
                };
                // Steps [i0, i1) of 16 keys of O_t += P V, P from `from` on; the last
                // ones of a key tile: its values are done with.
                constexpr int kSteps = kKeys / 16;
                auto product = [&](uint32_t v, uint32_t from, int i0, int i1, bool first, uint64_t *done, uint64_t *v_free) {
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t vd = v_desc + ((v * C::kKvB) >> 4);
#pragma unroll
                        for (int i = 0; i < kSteps; ++i)
                            if (i >= i0 && i < i1)
                                mma_f16_ts(o_t, from + i * 8, vd + ((i * 2048) >> 4), kIdO, i > 0 ? 1u : (first ? 0u : 1u));
                        if (i1 == kSteps) {
                            tc_commit(done);
                            tc_commit(v_free);
                        }
                    }
                    __syncwarp();
                };
                for (uint32_t n = 0; ok && take(n, it); ++n) {
                    const int tiles = __shfl_sync(0xffffffffu, it.tiles, 0);
                    const bool both = __shfl_sync(0xffffffffu, it.shared, 0) != 0;
                    ok = warp_wait_flag(FP8 ? &sm->q_ready[t] : &sm->q_full[t], n & 1, &sm->abort, 6);
                    if (C::kQuick && t == 0 && !both)  // (half of Q by each warpgroup)
                        ok = ok && warp_wait_flag(&sm->q_ready[1], n & 1, &sm->abort, 6);
                    // The second row tile's tensor memory changes hands: its last products
                    // are over (items by number: one role may be two ahead of the other).
                    if (n > 0 && both != before_shared)
                        ok = ok && warp_wait_flag(&sm->item_done[1 - t][(n - 1) & 3], ((n - 1) >> 2) & 1, &sm->abort, 22);
                    before_shared = both;
                    // Shared: the second row tile starts when the first one's maxima
                    // are known, which puts the two half a round apart; in step both
                    // would want the tensor pipe, then the exponentials, together.
                    if (t == 1 && __shfl_sync(0xffffffffu, (int)run_apart(it), 0)) {
                        ok = ok && warp_wait_flag(&sm->offset, off_ph, &sm->abort, 21);
                        off_ph ^= 1;
                    }
                    tc_fence_after();
                    if (both) {
                        for (int j = 0; j < tiles && ok; ++j) {
                            scores(tile0 + j, s_t, &sm->s_full[t], j + 1 == tiles, std::false_type{});
                            uint64_t *v_free;
                            const uint32_t v = wait_tile(tile0 + j, 1, v_free);
#pragma unroll
                            for (int h = 0; h < kParts; ++h) {
                                ok = ok && warp_wait_flag(&sm->p_ready[t][h], (shared0 + j) & 1, &sm->abort, 7);
                                if (!ok) break;
                                product(v, s_t, h * (kSteps / kParts), (h + 1) * (kSteps / kParts), j == 0,
                                        &sm->o_done[t], v_free);
                            }
                        }
                        shared0 += tiles;
                    } else if (t == 0) {
                        scores(tile0, s_col, &sm->s_split[0], tiles == 1, std::true_type{});
                        for (int j = 0; j < tiles && ok; ++j) {
                            // (the last product with this memory's weights came before)
                            if (j + 1 < tiles)
                                scores(tile0 + j + 1, s_col + ((j + 1) & 1) * kKeys, &sm->s_split[(j + 1) & 1], j + 2 == tiles,
                                       std::true_type{});
                            uint64_t *v_free;
                            const uint32_t v = wait_tile(tile0 + j, 1, v_free);
                            ok = ok && warp_wait_flag(&sm->p_split[j & 1], split_ph >> (j & 1) & 1, &sm->abort, 7);
                            if (!ok) break;
                            split_ph ^= 1u << (j & 1);
                            product(v, s_col + (j & 1) * kKeys, 0, kSteps, j == 0, &sm->o_split[j & 1], v_free);
                        }
                    } else {
                        for (int j = 0; j < tiles && ok; ++j)  // (the first row tile's: done with)
                            for (int part = 0; part < 2; ++part) {
                                uint64_t *free;
                                wait_tile(tile0 + j, part, free);
                                if (ok && lane == 0) mbar_arrive(free);
                            }
                        if (ok && lane == 0) mbar_arrive(&sm->q_empty[t]);  // (not used)
                    }
                    __syncwarp();
                    if (elect_one()) tc_commit(&sm->item_done[t][n & 3]);
                    __syncwarp();
                    tile0 += tiles;
                }
                // everything issued has finished before the block ends
                if (elect_one()) tc_commit(&sm->finished);
                __syncwarp();
                wait_own(&sm->finished, 0);
            };
            if (warp == kMmaWarp)
                products(std::integral_constant<int, 0>{});
            else
                products(std::integral_constant<int, 1>{});
        } else if (FP8 && warp == kFixWarp) {
            // ---------------- copies of V's codes
            Item it;
            uint32_t tile = 0;
            bool ok = true;
            for (uint32_t n = 0; ok && take(n, it); ++n) {
                int pg = page_of(it.b, it.j0, it.nk);
                ok = a.test_no_copies || load_q(it, n);
                for (int i = 0; i < it.tiles && ok && !a.test_no_copies; ++i, ++tile) {
                    const int key0 = (it.j0 + i) * kKeys, key = key0 + ((lane % chunks) << box_shift);
                    int p = pg;
                    if ((unsigned)p >= (unsigned)a.kv.num_pages) p = 0;  // (the other copying warp reports it)
                    if (i + 1 < it.tiles) pg = page_of(it.b, it.j0 + i + 1, it.nk);
                    const uint32_t s = tile % C::kRaw;
                    ok = warp_wait_flag(&sm->raw_empty[s], ((tile / C::kRaw) & 1) ^ 1, &sm->abort, 3);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&sm->raw_full[s], min(kKeys, (it.nk - key0 + R - 1) & -R) * D);
                    __syncwarp();
                    if (lane < chunks && key < it.nk) {
                        const int64_t row = ((((int64_t)p * a.kv.Hkv + it.hk) * 2 + 1) << page_shift) + (key & page_mask);
                        bulk_g2s(smem_u32(raw_base + s * C::kKB) + lane * R * D, a.kv.data + row * D, R * D,
                                 &sm->raw_full[s]);
                    }
                    __syncwarp();
                }
            }
            land();
        } else if (!FP8 && warp == kFixWarp) {
            // ---------------- last value tiles: zeros past the sequence's end
            Item it;
            uint32_t op = 0, ph = 0;  // ph: one phase bit per stage
            for (uint32_t n = 0; take(n, it); ++n) {
                if (!a.test_no_copies && !load_q(it, n)) break;
                op += 2 * it.tiles;
                const int from = it.nk - (it.j0 + it.tiles - 1) * kKeys;
                if (from >= kKeys) continue;
                const uint32_t s = (op - 1) % S;
                if (!warp_wait_flag(&sm->tail[s], (ph >> s) & 1, &sm->abort, 8)) break;
                ph ^= 1u << s;
                uint8_t *v = op_base + s * C::kKvB;
                for (int h = 0; h < kHalves; ++h)
                    for (int i = from * 8 + lane; i < kKeys * 8; i += 32)
                        *reinterpret_cast<uint4 *>(v + h * kKvHalf + i * 16) = make_uint4(0, 0, 0, 0);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->op_full[s]);
            }
            land();
        } else if (FP8 && warp >= kConvWarp) {
            // ---------------- V's scales and codes into operands
            const int cw = warp - kConvWarp;
            Item it;
            uint32_t tile = 0;
            bool ok = true;
            for (uint32_t n = 0; ok && take(n, it); ++n) {
                int expo = -126;  // of the largest scale so far
                for (int j = 0; j < it.tiles && ok; ++j, ++tile) {
                    const int n_tile = it.nk - (it.j0 + j) * kKeys, n_live = n_tile - kConvKeys * cw;  // (this warp's)
                    const uint32_t buf = tile % kScaleBufs, s = tile % S, r = tile % C::kRaw;
                    const float *sc = scales + (buf * 2 + 1) * kKeys;
                    ok = warp_wait_flag(&sm->sc_full[buf], (tile / kScaleBufs) & 1, &sm->abort, 19);
                    if (!ok) break;
                    // (every warp looks at all of them)
                    const float4 v4 = *reinterpret_cast<const float4 *>(sc + 4 * lane);
                    const float v[4] = {v4.x, v4.y, v4.z, v4.w};
                    const float mine = sc[kConvKeys * cw + lane];
                    uint32_t most = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t bits = __float_as_uint(v[e]) & 0x7FFFFFFFu;
                        if (4 * lane + e < n_tile && bits < 0x7F800000u) most = max(most, bits);
                    }
                    most = __reduce_max_sync(0xffffffffu, most);
                    expo = max(expo, (int)(most >> 23) - 127);
                    const __half2 own = __float2half2_rn(mine * pow2(-expo));
                    if (tid == 32 * kConvWarp) sm->expo[buf] = expo;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm->sc_ready[buf]);
                    ok = warp_wait_flag(&sm->raw_full[r], (tile / C::kRaw) & 1, &sm->abort, 15);
                    ok = ok && warp_wait_flag(&sm->op_empty[s], ((tile / S) & 1) ^ 1, &sm->abort, 14);
                    if (!ok) break;
                    uint8_t *to = op_base + s * C::kKvB + kConvKeys * cw * 128;
                    const uint8_t *from = raw_base + r * C::kKB + kConvKeys * cw * D;
                    // A lane has 16 codes of a row at a time, and rows r8, r8 + 8, ...;
                    // of heads of 128, odd rows the other half of the columns, so that
                    // eight neighbouring lanes' loads and stores are in different banks.
                    constexpr int kEach = kConvKeys * D / 16 / 32;
                    const int r8 = lane >> 2, piece = lane & 3;
                    const uint32_t u0 = ((2 * piece) ^ r8) << 4, u1 = ((2 * piece + 1) ^ r8) << 4;
                    auto row_of = [&](int k) { return (D == 128 ? k >> 1 : k) * 8 + r8; };
                    auto half_of = [&](int k) { return D == 128 ? (k ^ r8) & 1 : 0; };
                    // Four at a time: what all warps run in turn has to stay near the schedulers
                    // (eight in one stretch: 166 us instead of 160 for 64 sequences of 4096 keys,
                    // 16 tokens, 64 heads of 128 over 8, and 312 instead of 279 for 32 of 8192, 64
                    // tokens, 32 heads over 4).
                    constexpr int kGroup = 4;
#pragma unroll 1
                    for (int k0 = 0; k0 < kEach; k0 += kGroup) {
                        uint4 c[kGroup];
#pragma unroll
                        for (int k = 0; k < kGroup; ++k)
                            c[k] = *reinterpret_cast<const uint4 *>(from + row_of(k0 + k) * D + half_of(k0 + k) * 64 + piece * 16);
                        if (n_live < kConvKeys)
#pragma unroll
                            for (int k = 0; k < kGroup; ++k)
                                if (row_of(k0 + k) >= n_live) c[k] = make_uint4(0, 0, 0, 0);
#pragma unroll
                        for (int k = 0; k < kGroup; ++k) {
                            const uint32_t fb = __shfl_sync(0xffffffffu, *reinterpret_cast<const uint32_t *>(&own), row_of(k0 + k));
                            // (a row that does not exist has zeros whatever its scale)
                            const uint32_t f = n_live < kConvKeys && row_of(k0 + k) >= n_live ? 0u : fb;
                            auto scaled = [&](uint32_t w) {
                                uint2 h = e4m3_f16(w);
                                __half2 x = __hmul2(*reinterpret_cast<__half2 *>(&h.x), *reinterpret_cast<const __half2 *>(&f));
                                __half2 y = __hmul2(*reinterpret_cast<__half2 *>(&h.y), *reinterpret_cast<const __half2 *>(&f));
                                h.x = *reinterpret_cast<uint32_t *>(&x);
                                h.y = *reinterpret_cast<uint32_t *>(&y);
                                return h;
                            };
                            const uint2 o0 = scaled(c[k].x), o1 = scaled(c[k].y), o2 = scaled(c[k].z), o3 = scaled(c[k].w);
                            uint8_t *at = to + half_of(k0 + k) * kKvHalf + row_of(k0 + k) * 128;
                            *reinterpret_cast<uint4 *>(at + u0) = make_uint4(o0.x, o0.y, o1.x, o1.y);
                            *reinterpret_cast<uint4 *>(at + u1) = make_uint4(o2.x, o2.y, o3.x, o3.y);
                        }
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sm->op_full[s]);
                        mbar_arrive(&sm->raw_empty[r]);
                    }
                    __syncwarp();
                }
            }
        }
    } else {
        // ---------------- softmax: warpgroup t has row tile t, a thread a row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
        const int t = warp >> 2;
        const int r = tid & 127;
        const uint32_t lane_base = (uint32_t)(warp & 3) * 32 << 16;
        const uint32_t s_t = s_col + t * kKeys + lane_base, o_t = o_col + t * D + lane_base;
        const int tok_r = r / Gt, gr = r % Gt;
        uint32_t tile0 = 0, shared0 = 0;  // key tiles of the items before, and of those shared
        uint32_t split_ph = 0, ex_ph = 0; // parities: a bit a half of S; the exchange
        bool before_shared = false;       // the item before
        // All 8 warps have come here.
        auto exchange = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm->exchange);
            bool done = C::kQuick && mbar_test_wait(&sm->exchange, ex_ph);
            if (C::kQuick)
                for (int i = 0; i < 32 && !done; ++i) done = mbar_test_wait(&sm->exchange, ex_ph);
            done = (C::kQuick && __all_sync(0xffffffffu, done)) || warp_wait_flag(&sm->exchange, ex_ph, &sm->abort, 12);
            ex_ph ^= 1;
            return done;
        };
        Item it;
        bool ok = true;
        for (uint32_t n = 0; ok && take(n, it); ++n) {
            const int tok = it.tok0 + (it.shared ? t * tpt : 0) + tok_r;
            const bool live = tok_r < tpt && tok < it.nq && gr < it.heads;
            const bool any_live = __any_sync(0xffffffffu, live);
            const int ctx = it.nk - it.nq;
            const uint64_t mask = live ? __ldg(a.tree + it.q0 + tok) & (~0ull >> (64 - it.nq)) : 0;
            float sl = a.scale * kLog2e;
            if (FP8) {
                // this row of Q, its largest value in [128, 256), as two rows of
                // e4m3 numbers, in its place or to tensor memory
                ok = warp_wait_flag(&sm->q_full[t], n & 1, &sm->abort, 16);
                // (the second row tile's sums of the item before are read)
                if (C::kQuick && !it.shared && before_shared) ok = ok && exchange();
                before_shared = it.shared;
                if (!ok) break;
                tc_fence_after();
                uint8_t *q = base + t * C::kQB + r * 128;
                auto unit = [&](int u) {  // 8 columns, 16 bytes
                    return reinterpret_cast<uint4 *>(q + (u >> 3) * kQHalf + (((u & 7) ^ (r & 7)) << 4));
                };
                float most = 0.f;
                auto look = [&](const uint4 &x) {
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        most = max3(most, fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xFFFF0000u)));
                };
                auto factors = [&](float &down) {
                    // (an infinity makes the row NaN, as its scores would)
                    const int e2 = max((int)(__float_as_uint(most) >> 23) - 127, -119);
                    down = e2 > 127 ? __uint_as_float(0x7FFFFFFFu) : pow2(7 - e2);
                    // (never 0, which times a masked score's -inf would be NaN)
                    sl = fmaxf(sl * pow2(min(e2, 127) - 7), __uint_as_float(1));
                };
                // 16 columns: 16 bytes of each term
                auto terms = [&](const uint4 &x, const uint4 &y, float down, uint32_t *h0, uint32_t *h1) {
                    const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float2 a0 = make_float2(__uint_as_float(w[2 * e] << 16) * down,
                                                __uint_as_float(w[2 * e] & 0xFFFF0000u) * down);
                        float2 a1 = make_float2(__uint_as_float(w[2 * e + 1] << 16) * down,
                                                __uint_as_float(w[2 * e + 1] & 0xFFFF0000u) * down);
                        const uint32_t c0 = take_e4m3(a0), c1 = take_e4m3(a1);
                        h0[e] = c0 | c1 << 16;
                        const uint32_t d0 = take_e4m3(a0), d1 = take_e4m3(a1);
                        h1[e] = d0 | d1 << 16;
                    }
                };
                if (C::kQuick && !it.shared) {
                    // each warpgroup, from its copy, half of the columns, to tensor memory
#pragma unroll
                    for (int u = 0; u < D / 8; ++u) look(*unit(u));
                    float down;
                    factors(down);
                    uint32_t h0[16], h1[16];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        terms(*unit(8 * t + 2 * u), *unit(8 * t + 2 * u + 1), down, h0 + 4 * u, h1 + 4 * u);
                    tmem_st16(q_col + lane_base + t * 16, h0);
                    tmem_st16(q_col + lane_base + D / 4 + t * 16, h1);
                } else if (any_live) {
                    uint4 v[D / 8];
#pragma unroll
                    for (int u = 0; u < D / 8; ++u) look(v[u] = *unit(u));
                    float down;
                    factors(down);
#pragma unroll
                    for (int u = 0; u < D / 16; ++u) {
                        uint32_t h0[4], h1[4];
                        terms(v[2 * u], v[2 * u + 1], down, h0, h1);
                        // (heads of 64: both terms in one row)
                        *unit(u) = make_uint4(h0[0], h0[1], h0[2], h0[3]);
                        *unit((D == 128 ? 8 : 4) + u) = make_uint4(h1[0], h1[1], h1[2], h1[3]);
                    }
                }
                tc_wait_st();
                tc_fence_before();
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->q_ready[t]);
            }
            float ref = -INFINITY;  // the row's reference, in log2 units
            float l = 0.f;
            int expo = 0;  // of the scales that O's sums were made with
            // Products with key tile j, whose scores have been here and no later ones'
            // weights.  (Up to 128 rows weights can be there two products ahead, hence
            // barriers for every other key tile; all three have the same counts.)
            auto wait_products = [&](int j) {
                if (it.shared) return warp_wait_flag(&sm->o_done[t], (shared0 + j) & 1, &sm->abort, 10);
                return warp_wait_flag(&sm->o_split[j & 1], ~(split_ph >> (j & 1)) & 1, &sm->abort, 11);
            };
            bool seen = false;  // the next key tile's scores and scales
            // Key tile j: W of its scores a thread, all, or this warpgroup's half.
            auto round = [&](auto width, int j) {
                constexpr int W = decltype(width)::value;
                constexpr bool kSplit = W < kKeys;
                const int half = j & 1, col0 = kSplit ? t * W : 0;
                const uint32_t s_at = kSplit ? s_col + half * kKeys + lane_base + col0 : s_t;
                const uint32_t p_at = kSplit ? s_col + half * kKeys + lane_base + col0 / 2 : s_t;
                const uint32_t buf = (tile0 + j) % kScaleBufs;
                if (kSplit && C::kQuick && !any_live) {
                    // (no row of this warp's is used: it is there when the others are)
                    split_ph ^= 1u << half;
                    if (!exchange()) return false;
                    if (lane == 0) {
                        if (FP8) mbar_arrive(&sm->sc_empty[buf]);
                        mbar_arrive(&sm->p_split[half]);
                    }
                    return true;
                }
                // (before the scores are)
                if (FP8 && !seen && !warp_wait_flag(&sm->sc_ready[buf], ((tile0 + j) / kScaleBufs) & 1, &sm->abort, 17)) return false;
                const int larger = FP8 ? sm->expo[buf] : 0;  // (the same for all rows)
                bool both_there = false;  // of the next key tile
                if (kSplit) {
                    if (!seen && !warp_wait_flag(&sm->s_split[half], split_ph >> half & 1, &sm->abort, 9)) return false;
                    split_ph ^= 1u << half;
                } else if (!warp_wait_flag(&sm->s_full[t], (shared0 + j) & 1, &sm->abort, 9)) {
                    return false;
                }
                const float *sc = scales + buf * 2 * kKeys + col0;
                tc_fence_after();
                const bool tells = !kSplit && t == 0 && j == 0 && run_apart(it) && lane == 0;
                if (!(kSplit && C::kQuick) && !any_live) {
                    if (tells) mbar_arrive(&sm->offset);
                    expo = larger;
                    tc_fence_before();
                    __syncwarp();
                    if (FP8 && lane == 0) mbar_arrive(&sm->sc_empty[buf]);
                    if (kSplit && !exchange()) return false;
                    if (lane == 0)
                        for (int h = 0; h < W / (kKeys / kParts); ++h)
                            mbar_arrive(kSplit ? &sm->p_split[half] : &sm->p_ready[t][h]);
                    return true;
                }
                float x[W];
#pragma unroll
                for (int c = 0; c < W; c += 32) tmem_ld32(s_at + c, x + c);
                tc_wait_ld();
                if (FP8) {
#pragma unroll
                    for (int c = 0; c < W; c += 4) {
                        const float4 k = *reinterpret_cast<const float4 *>(sc + c);
                        const float2 lo = mul2(make_float2(x[c], x[c + 1]), make_float2(k.x, k.y));
                        const float2 hi = mul2(make_float2(x[c + 2], x[c + 3]), make_float2(k.z, k.w));
                        x[c] = lo.x;
                        x[c + 1] = lo.y;
                        x[c + 2] = hi.x;
                        x[c + 3] = hi.y;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm->sc_empty[buf]);
                }
                const int key0 = (it.j0 + j) * kKeys + col0;
                if (key0 + W > ctx) {
#pragma unroll
                    for (int c = 0; c < W; c += 32) {
                        const int d = key0 + c - ctx;  // the drafted token of column c
                        if (d > -32) {
                            const uint32_t vis = d >= 64  ? 0u
                                                 : d >= 0 ? (uint32_t)(mask >> d)
                                                          : ((uint32_t)mask << -d) | ((1u << -d) - 1u);
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[c + e] = vis >> e & 1 ? x[c + e] : -INFINITY;
                        }
                    }
                }
                float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int c = 4; c + 8 <= W; c += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e) m4[e] = max3(m4[e], x[c + 2 * e], x[c + 2 * e + 1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) m4[e] = fmaxf(m4[e], x[W - 4 + e]);
                float most = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                if (kSplit) {
                    // (both warpgroups have their scores in registers after this, too: the
                    // weights of one lie where scores of the other were)
                    sm->halves[half][t][r] = most;
                    tc_fence_before();
                    if (!exchange()) return false;
                    tc_fence_after();
                    most = fmaxf(most, sm->halves[half][1 - t][r]);
                }
                const float top = most * sl;
                const bool raise = top > ref + kSlack;
                if (__any_sync(0xffffffffu, raise) || (FP8 && larger != expo)) {
                    const float to = raise ? top : ref;
                    float f = raise ? ex2(ref - to) : 1.f;
                    l *= f;
                    ref = to;
                    if (FP8) {
                        f *= pow2(max(expo - larger, -127));
                        expo = larger;
                    }
                    if (j > 0) {
                        // the last product into O has to be over; of one O each
                        // warpgroup has half of the columns
                        if (!wait_products(j - 1)) return false;
                        tc_fence_after();
                        const uint32_t o_at = kSplit ? o_col + lane_base + t * (D / 2) : o_t;
#pragma unroll
                        for (int c = 0; c < (kSplit ? D / 2 : D); c += 16) {
                            uint32_t o[16];
                            tmem_ld16(o_at + c, o);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st16(o_at + c, o);
                        }
                    }
                }
                if (tells) mbar_arrive(&sm->offset);
                const float z = (ref == -INFINITY ? 0.f : ref) - (FP8 ? kShift : 0);
                const float2 sl2 = make_float2(sl, sl), nz2 = make_float2(-z, -z);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < W; c += 32) {
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float2 y = fma2(make_float2(x[c + 2 * e], x[c + 2 * e + 1]), sl2, nz2);
                        y.x = ex2(y.x);
                        y.y = ex2(y.y);
                        sum[e & 1] = add2(sum[e & 1], y);
                        if (FP8) {
                            const __half2 w = __floats2half2_rn(y.x, y.y);
                            p[e] = *reinterpret_cast<const uint32_t *>(&w);
                        } else {
                            p[e] = pack_bf16(y.x, y.y);
                        }
                    }
                    if (kSplit && C::kQuick && c + 32 == W) {
                        const uint32_t i = tile0 + j + 1;
                        both_there = mbar_test_wait(&sm->s_split[1 - half], split_ph >> (1 - half) & 1);
                        both_there = both_there && mbar_test_wait(&sm->sc_ready[i % kScaleBufs], (i / kScaleBufs) & 1);
                    }
                    tmem_st16(p_at + c / 2, p);
                    if ((c + 32) % (kKeys / kParts) == 0) {  // their product may start
                        tc_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(kSplit ? &sm->p_split[half] : &sm->p_ready[t][c / (kKeys / kParts)]);
                    }
                }
                const float2 both = add2(sum[0], sum[1]);
                l += both.x + both.y;
                if (kSplit && C::kQuick) seen = __all_sync(0xffffffffu, both_there);
                return true;
            };
            if (it.shared)
                for (int j = 0; j < it.tiles && ok; ++j) ok = round(std::integral_constant<int, kKeys>{}, j);
            else
                for (int j = 0; j < it.tiles && ok; ++j) ok = round(std::integral_constant<int, kKeys / 2>{}, j);
            if (!ok) break;
            // ---- the rows' outputs
            float sum = l;
            if (!it.shared) {  // (the half that no reader of the last maxima can be at)
                sm->halves[it.tiles & 1][t][r] = l;
                ok = exchange();
                if (!ok) break;
                sum = sm->halves[it.tiles & 1][0][r] + sm->halves[it.tiles & 1][1][r];
            }
            ok = wait_products(it.tiles - 1);
            if (!ok) break;
            tc_fence_after();
            tile0 += it.tiles;
            if (it.shared) shared0 += it.tiles;
            const bool whole = it.slot < 0, none = sum == 0.f;  // (none: a row that sees nothing)
            // What the row's sums are multiplied by: 1 over the sum if these are all
            // keys; fp8: and the powers of two of the weights and of the scales.
            if (FP8) sum *= 1.f / (1 << kShift);
            float f = whole ? (none ? 0.f : 1.f / sum) : 1.f;
            if (FP8) f *= pow2(expo) * (1.f / (1 << kShift));
            // one O: each warpgroup has half of the columns
            const uint32_t o_at = it.shared ? o_t : o_col + lane_base;
            const int c0 = it.shared ? 0 : t * (D / 2), c1 = it.shared ? D : c0 + D / 2;
            const int row_tile = it.shared ? t : 0;
            uint16_t *to = a.out + (int64_t)(it.q0 + tok) * a.out_stride + (it.h0 + gr) * D;
            if (any_live)
#pragma unroll 1
                for (int c = c0; c < c1; c += 32) {
                    float o[32];
                    tmem_ld32(o_at + c, o);
                    tc_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] *= f;
                    if (!live) continue;
                    if (!whole) {
                        float *part = reinterpret_cast<float *>(a.workspace + L.sums);
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4 *>(part + part_at(it.slot, row_tile, c + e, r, D)) =
                                make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            *reinterpret_cast<uint4 *>(to + c + e) =
                                none ? make_uint4(0, 0, 0, 0)
                                     : make_uint4(pack_bf16(o[e], o[e + 1]), pack_bf16(o[e + 2], o[e + 3]),
                                                  pack_bf16(o[e + 4], o[e + 5]), pack_bf16(o[e + 6], o[e + 7]));
                    }
                }
            if (live && (it.shared || t == 0)) {
                if (!whole)
                    reinterpret_cast<float2 *>(a.workspace + L.ml)[((size_t)it.slot * kM + row_tile) * kTile + r] =
                        make_float2(ref, sum);
                else if (a.lse)
                    a.lse[(size_t)(it.q0 + tok) * a.Hq + it.h0 + gr] =
                        none ? -INFINITY : (ref + __log2f(sum)) * kLn2;
            }
            // (O and the sums are read: the next item's first p_ready comes after this)
            tc_fence_before();
            if (!it.shared) ok = exchange();
            tc_fence_after();
        }
    }
    __syncthreads();
    if (tid == 0) reinterpret_cast<Err *>(a.workspace + L.err)[g] = Err{sm->abort, sm->bad};
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_relinquish();
        tmem_dealloc(sm->tmem, 512);
    }
}

// Joins the parts of a range: blockIdx.x is its record, blockIdx.y a row tile and
// 32 columns of it; a thread has a row and 8 columns.  Latency counts: what the
// record does not say is not looked up, and the loads of up to kAhead parts are in
// flight together.
template <int D, bool REST>
__global__ void __launch_bounds__(4 * kTile) tree_join(const DecodeAttnArgs a, const int n_blocks) {
    __shared__ int red[2];
    constexpr int kAhead = 4;
    const TreeLayout L = tree_layout(D);
    const int tid = threadIdx.x, r = tid & (kTile - 1);
    const int Gt = tile_heads(a.Hq / a.kv.Hkv), tpt = kTile / Gt;
    const int t = blockIdx.y / (D / 32), c = blockIdx.y % (D / 32) * 32 + tid / kTile * 8;
    pdl_wait();
    const Join jn = reinterpret_cast<const Join *>(a.workspace + L.join)[blockIdx.x];
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
            if (REST) {  // what the launch before has found counts too
                if (ctrl->status == MOE_ERR_DEVICE_TIMEOUT) red[0] = max(red[0], ctrl->detail);
                if (ctrl->status == MOE_ERR_DEVICE_BAD_INDEX) red[1] = min(red[1], ctrl->detail);
            }
            ctrl->status = red[0] ? MOE_ERR_DEVICE_TIMEOUT
                                  : (red[1] != 0x7fffffff ? MOE_ERR_DEVICE_BAD_INDEX : MOE_OK);
            ctrl->detail = red[0] ? red[0] : (red[1] != 0x7fffffff ? red[1] : 0);
        }
    }
    if (jn.parts == 0 || t >= jn.tiles) return;
    const int tok = jn.tok0 + t * tpt + r / Gt, gr = r % Gt;
    if (r / Gt >= tpt || tok >= jn.nq || gr >= jn.heads) return;
    const float2 *ml = reinterpret_cast<const float2 *>(a.workspace + L.ml);
    const float *sums = reinterpret_cast<const float *>(a.workspace + L.sums);
    // the first part is its block's last one, the others are first ones
    auto slot_of = [&](int i) { return 2 * (jn.first + i) + (i == 0 ? 1 : 0); };
    float top = -INFINITY, sum = 0.f, o[8] = {};
    for (int i0 = 0; i0 < jn.parts; i0 += kAhead) {
        float2 v[kAhead];
        float4 x[kAhead][2];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = min(i0 + k, jn.parts - 1);
            v[k] = ml[((size_t)slot_of(i) * kM + t) * kTile + r];
            x[k][0] = *reinterpret_cast<const float4 *>(sums + part_at(slot_of(i), t, c, r, D));
            x[k][1] = *reinterpret_cast<const float4 *>(sums + part_at(slot_of(i), t, c + 4, r, D));
        }
        float to = top;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) to = fmaxf(to, v[k].x);
        const float z = to == -INFINITY ? 0.f : to, f0 = ex2(top - z);
        top = to;
        sum *= f0;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] *= f0;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (i0 + k >= jn.parts) break;
            const float f = ex2(v[k].x - z);
            const float e[8] = {x[k][0].x, x[k][0].y, x[k][0].z, x[k][0].w, x[k][1].x, x[k][1].y, x[k][1].z, x[k][1].w};
            sum = fmaf(f, v[k].y, sum);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = fmaf(f, e[i], o[i]);
        }
    }
    const bool none = sum == 0.f;
    const float inv = none ? 0.f : 1.f / sum;
    const int64_t row = (int64_t)jn.q0 + tok;
    const int h = jn.h0 + gr;
    *reinterpret_cast<uint4 *>(a.out + row * a.out_stride + h * D + c) =
        none ? make_uint4(0, 0, 0, 0)
             : make_uint4(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv),
                          pack_bf16(o[4] * inv, o[5] * inv), pack_bf16(o[6] * inv, o[7] * inv));
    if (a.lse && c == 0) a.lse[row * a.Hq + h] = none ? -INFINITY : (top + __log2f(sum)) * kLn2;
}

template <int D, bool FP8, bool REST>
cudaError_t run(const DecodeAttnArgs &a, int sms, cudaStream_t s) {
    using C = Cfg<D, FP8>;
    const int G = a.Hq / a.kv.Hkv, Gt = tile_heads(G), tpt = tile_tokens(G), HT = (G + Gt - 1) / Gt;
    CUtensorMap mq, mkv;
    {
        const uint64_t dims[4] = {64, (uint64_t)a.Hq, (uint64_t)a.T, D / 64};
        const uint64_t strides[3] = {D * 2, (uint64_t)a.q_stride * 2, 128};
        const uint32_t box[4] = {64, (uint32_t)Gt, (uint32_t)tpt, 1};
        if (!encode_tensor_map(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, a.q, dims, strides, box,
                               CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    }
    const int page = 1 << a.kv.page_shift;
    if (FP8) {  // K's codes (the rows of V are copied as they are)
        const uint64_t dims[3] = {D, (uint64_t)page, (uint64_t)a.kv.num_pages * a.kv.Hkv * 2};
        const uint64_t strides[2] = {D, (uint64_t)page * D};
        const uint32_t box[3] = {D, (uint32_t)(page < kKeys ? page : kKeys), 1};
        if (!encode_tensor_map(&mkv, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.kv.data, dims, strides, box,
                               D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
            return cudaErrorInvalidValue;
    } else {
        const uint64_t row_b = D * 2;
        const uint64_t dims[4] = {64, (uint64_t)page, D / 64, (uint64_t)a.kv.num_pages * a.kv.Hkv * 2};
        const uint64_t strides[3] = {row_b, 128, page * row_b};
        const uint32_t box[4] = {64, (uint32_t)(page < kKeys ? page : kKeys), 1, 1};
        if (!encode_tensor_map(&mkv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, a.kv.data, dims, strides, box,
                               CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    }
    // no more blocks than key tiles could exist
    const int64_t tiles = ((int64_t)a.table_stride * page + kKeys - 1) / kKeys;
    const int tokens = a.T < kTreeTokens ? a.T : kTreeTokens, rows = tokens * Gt;
    const int64_t rb = (tokens + kM * tpt - 1) / (kM * tpt);
    const int64_t most = (a.B < a.T ? a.B : a.T) * tiles * a.kv.Hkv * HT * rb;
    int grid = sms < kMaxGrid ? sms : kMaxGrid;
    if (most < grid) grid = (int)most;
    auto fn = tree_kernel<D, FP8, REST>;
    static SmemOnce once;
    cudaError_t err = once.set(reinterpret_cast<const void *>(fn), C::kSmem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    err = cudaLaunchKernelEx(&cfg, fn, a, HT, mq, mkv);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cj = {};
    cj.gridDim = dim3(grid, (rows > tpt * Gt ? kM : 1) * D / 32);
    cj.blockDim = dim3(4 * kTile);
    cj.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cj.attrs = at;
    cj.numAttrs = 1;
    return cudaLaunchKernelEx(&cj, tree_join<D, REST>, a, grid);
}

}  // namespace

size_t tree_workspace(int, int T, int Hq, int Hkv, int D) {
    const size_t small = tree_small_workspace(T, Hq, Hkv, D), large = align_up(tree_layout(D).total, 256);
    return small > large ? small : large;
}

// REST: the sequences of more than a.few tokens alone, over fp8.
template <bool REST>
static cudaError_t launch_large(const DecodeAttnArgs &a, cudaStream_t s) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const int sms = tc_grid(dev);
    if (sms < 1) return cudaErrorInvalidDevice;
    if (REST || a.cache_type == MOE_KV_FP8)
        return a.D == 128 ? run<128, true, REST>(a, sms, s) : run<64, true, REST>(a, sms, s);
    return a.D == 128 ? run<128, false, false>(a, sms, s) : run<64, false, false>(a, sms, s);
}

cudaError_t launch_attn_tree(const DecodeAttnArgs &args, cudaStream_t s) {
    DecodeAttnArgs a = args;
    // Tiles of 8 or 16 rows where none can have more, or where there are few on average
    // (what a sequence has the host does not know; any number is right either way).  64
    // sequences of 4096 keys, 4 key/value heads, here and in small tiles: 8 rows each,
    // heads of 128, bf16 91 and 90 us, fp8 81 and 55, heads of 64 53 and 49, 83 and 33; 16
    // rows 92 and 99, 81 and 76, 52 and 52, 83 and 51; 24 rows 93 and 175, 81 and 130, 52 and
    // 90, 83 and 84.  6 sequences of 4000 keys, one head, 4 rows, bf16 21 and 11; 162 of
    // 300, 2 heads, 6 rows, bf16 21 and 16, fp8 33 and 17.
    const int tokens = a.T < kTreeTokens ? a.T : kTreeTokens, G = a.Hq / a.kv.Hkv;
    const bool bf16 = a.cache_type == MOE_KV_BF16;
    const int few = bf16 && a.D == 128 ? 8 : 12;
    if (tokens * G <= kFewRows) return launch_attn_tree_small(a, s);
    if ((int64_t)a.T * G > (int64_t)a.B * few || G > kFewRows) return launch_large<false>(a, s);
    // A few sequences may have most of the rows, and small tiles read such a one's keys
    // for every 8 or 16 of them.  Where that could be many bytes (by the table's width),
    // it is large tiles over bf16, where the small ones gain little from there on, and
    // over fp8 small tiles for sequences of up to 16 rows, then large ones for the
    // others.  One sequence of 64 tokens and 63 without, 32 heads of 128 over 4, in small
    // tiles and so: bf16, 1024 keys (128 MB) 22 and 16 us, 4096 50 and 23, 8192 87 and 26;
    // fp8, 2048 (132 MB) 31 and 30, 4096 50 and 33, 8192 87 and 37.  64 sequences of 6
    // tokens, 4 heads over 4, 4096 keys: bf16 (384 MB) 90 and 91, heads of 64 49 and 52;
    // 64 of 2 tokens, 16 heads, fp8 (264 MB), where the second launch finds nothing, 55 and
    // 61.
    // (a double: with the widest tables this is past 64 bits)
    const double reads = (double)a.T * G / 8 * a.kv.Hkv * ((int64_t)a.table_stride << a.kv.page_shift) *
                         (bf16 ? 4 * a.D : 2 * a.D + 8);
    if (reads <= kFewBytes) return launch_attn_tree_small(a, s);
    if (bf16) return launch_large<false>(a, s);
    a.few = kFewRows / G;
    const cudaError_t err = launch_attn_tree_small(a, s);
    return err != cudaSuccess ? err : launch_large<true>(a, s);
}

}  // namespace moe
