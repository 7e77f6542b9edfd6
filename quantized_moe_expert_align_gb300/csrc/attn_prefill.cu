// attn_prefill.cu -- attention over packed prompts on the tensor cores.
//
// For a query row with keys 0 .. limit - 1:  o = sum_j p_j v_j / sum_j p_j,
// p_j = 2^(s_j - r), s_j = scale log2(e) q . k_j and r a reference close to
// the running maximum.  4 D multiply-adds' worth of work per visible pair
// and head against 4 D bytes per key and 256 rows: the tensor pipe bounds it.
//
// One persistent block per SM takes work items of 256 rows: two tiles of 128
// rows of one key/value head, a row being one (token, query head of the
// group) pair, so grouped heads share every key tile and short prompts fill
// the rows.  Key/value tiles have 128 keys.  Per tile t and key tile j:
//   S_t = Q_t K_j^T      tcgen05.mma, operands in shared memory (TMA, 128 B swizzle)
//   P_t = 2^(S_t - r)    one thread per row, in registers; rounded to bf16 (v's
//                        type, which the product wants) into tensor memory
//   O_t += P_t V_j       tcgen05.mma, P_t from tensor memory
// One warp per row tile issues its products, so that one tile's softmax runs
// under the other tile's products; one warp copies; one clears the rows of a
// last value tile that belong to the next sequence (a weight of 0 would not
// stop their NaN).  The reference r is raised, and O_t rescaled, only when a
// row's maximum exceeds it by 2^8: the sums are in fp32, where p <= 2^8 costs
// nothing (8192 causal tokens: 798 us when every rise rescales and 680 with this,
// when it was added).
//
// A planning kernel lists the items by falling number of key tiles; the
// blocks take them from a counter, longest first.  Where a few items have
// several times the key tiles of an SM's even share of the whole work, they are
// cut into parts, whose unscaled sums a last kernel joins in order.  Small calls (at
// most 32 sequences and kMinKeys keys in all, where nothing is cut) do
// without the plan: every block finds its own items.
//
// Measured on one GB300 (cuBLAS bf16 1876 TFLOP/s in a burst, 1697 sustained),
// in bursts of 20 calls and back to back for two seconds under the power limit;
// heads of 128: 8192 causal tokens, 64 heads over 8, 611 us (1801 TFLOP/s) and
// 669 (1643); six prompts up to 4096 tokens 350 (1599) and 381 to 389 (1471 to
// 1441).  A round of one row tile is softmax (1300 cycles) then its 1024 cycles
// of products and two hand-overs; the two tiles, half a round apart, keep the
// tensor pipe busy 75 to 85% of the time.  Heads of 64: 8192 causal tokens 455
// us (1209 TFLOP/s) and 467; there the two warps per scheduler cannot hide the
// softmax's latencies (tensor pipe, exponentials and issue all near 50%).  1024
// tokens take 18.4 us: eight key tiles in turn at 1.4 us.
#include <type_traits>

#include "attn_common.cuh"
#include "gemm_tc.h"

namespace moe {
namespace {

using namespace attn;

constexpr int kTile = 128;       // rows of a row tile
constexpr int kM = 2;            // row tiles of an item
constexpr int kKeys = 128;       // keys of a key tile
constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 1024;
constexpr float kSlack = 8.f;    // a row's maximum may exceed its reference by this

constexpr int kMinKeys = 1024;   // with no more keys in all, no key range is cut
constexpr int kMinPart = 4;      // key tiles of a part at least
// What the plan reckons with: a round of one key tile, a join, a part.
constexpr int kRound = 32, kJoinCost = 128, kPartCost = 1;
constexpr int kMaxSms = 160;     // blocks of the main kernel at most
constexpr int kMaxParts = 2 * kMaxSms;  // of one call, all heads together

struct PlanHead {
    int32_t items, next;   // (block, part) pairs; the next item to take
    int32_t joins, slots;  // blocks in parts; places for parts
};
// One sequence's block of rows for every head (what does not depend on the
// head), or one part of its keys.
struct __align__(16) Block {
    int32_t q0, nq, k0, nk;   // rows of the sequence
    int32_t tok0;             // the block's first token within the sequence
    int32_t j0;               // the first key tile
    int32_t tiles0, tiles1;   // key tiles of each row tile, from j0 on
    int32_t slot, parts, part, pad;  // slot: of the block's first head and part; -1: whole
};
struct __align__(16) Split {  // a block in parts
    int32_t q0, nq, tok0, slot, parts, pad[3];
};
struct PrefillLayout {
    size_t ctrl, head, list, splits, ml, sums, total;
};
// Every sequence has at most one partly filled block; parts beyond a block's
// first add up to at most kMaxSms.
__host__ __device__ inline PrefillLayout prefill_layout(int B, int Tq, int tokens, int D) {
    PrefillLayout l;
    l.ctrl = 0;
    l.head = 256;
    l.list = 512;
    l.splits = l.list + ((size_t)Tq / tokens + B + kMaxSms) * sizeof(Block);
    l.ml = l.splits + kMaxParts * sizeof(Split);
    const size_t rows = (size_t)kMaxParts * kM * kTile;
    l.sums = (l.ml + rows * 8 + 255) / 256 * 256;
    l.total = l.sums + rows * D * 4;
    return l;
}
// Place of a part's four columns c .. c + 3 of row r of row tile t: rows are
// neighbours, so a warp's stores and loads are whole lines.
__host__ __device__ inline size_t part_at(int slot, int t, int c, int r, int D) {
    return ((((size_t)slot * kM + t) * (D / 4) + c / 4) * kTile + r) * 4;
}
// Query heads of a row tile and tokens of a row tile, for groups of G heads.
__host__ __device__ inline int tile_heads(int G) { return G < kTile ? G : kTile; }
__host__ __device__ inline int tile_tokens(int G) { return kTile / tile_heads(G); }

constexpr int kParts = 2;        // in which a key tile's weights come
// Warps: two softmax warpgroups, one warp per row tile issuing products, one
// copying, one clearing.
constexpr int kMmaWarp = 4 * kM, kLoadWarp = 5 * kM, kFixWarp = 5 * kM + 1;
constexpr int kThreads = 32 * (5 * kM + 2);
// The launch's 168 registers a thread, shared out anew (88 and 208: the same
// for heads of 128, 237 us instead of 229 for prompt parts with heads of 64).
constexpr int kRoleRegs = 72, kSoftmaxRegs = 216;
static_assert(128 * kRoleRegs + 256 * kSoftmaxRegs <= 384 * 168, "register split");
// Items of at least this many key tiles run their row tiles offset.  The first
// tile's roles cannot signal twice before the second's have looked once: an
// item of kApart key tiles fills the ring of stages.
constexpr int kApart = 4;

template <int D>
struct Cfg {
    static constexpr int kQB = kTile * D * 2, kKvB = kKeys * D * 2;  // a Q tile, a K or V tile
    static constexpr int kStages = D == 128 ? 5 : 8;
    static_assert(kStages <= 2 * kApart, "see kApart");
    // Tensor memory (512 columns): S_t 2 x 128, O_t 2 x D.  Heads of 64 leave
    // 128 columns for the weights P_t, so that the next scores can be computed
    // as soon as S_t is in registers; heads of 128 put P_t over S_t.  (Heads
    // of 64 as three row tiles against key tiles of 64, for more warps to hide
    // the softmax's latencies: 205 us instead of 148, 2432 rows over 4096 keys.)
    static constexpr bool kOwnP = D == 64;
    static constexpr size_t kSmem = (size_t)kM * kQB + kStages * kKvB + 1024 + 1024;
    static_assert(kSmem > 114 * 1024, "one block per SM: all of tensor memory is its own");
};

// A work item as the roles see it.
struct Item {
    Block b;
    int hk, h0, heads;     // key/value head; first query head and their number
    int slot;              // this head's and part's place, -1: the block is whole
    int done;
};

struct Shared {
    uint64_t q_full[kM], q_empty[kM], kv_full[8], kv_empty[8], tail[8], s_full[kM], s_free[kM];
    uint64_t p_ready[kM][kParts], o_done[kM];
    uint64_t offset;            // the second row tile may start
    uint64_t item_full[2], item_empty[2], finished;
    uint32_t tmem;
    int abort;
    Item item[2];
};
static_assert(sizeof(Shared) <= 1024, "shared block");

__device__ __forceinline__ bool seq_ok(const PrefillArgs &a, int b) {
    const int q0 = __ldg(a.cu_q + b), q1 = __ldg(a.cu_q + b + 1);
    const int k0 = __ldg(a.cu_k + b), k1 = __ldg(a.cu_k + b + 1);
    return q0 >= 0 && q1 >= q0 && q1 <= a.Tq && k0 >= 0 && k1 >= k0 && k1 <= a.Tk;
}
// Keys that token `tok` of a sequence sees.
__device__ __forceinline__ int keys_seen(int causal, int tok, int nq, int nk) {
    return causal ? max(0, min(nk, tok + nk - nq + 1)) : nk;
}

// The block of a sequence that starts at its token t0, whole.
__device__ __forceinline__ Block block_at(int causal, int q0, int nq, int k0, int nk, int t0, int tpt) {
    auto tiles_of = [&](int t) {  // of the row tile from token t on
        const int last = min(nq, t + tpt) - 1;
        return last < t ? 0 : (keys_seen(causal, last, nq, nk) + kKeys - 1) / kKeys;
    };
    return Block{q0, nq, k0, nk, t0, 0, tiles_of(t0), tiles_of(t0 + tpt), -1, 1, 0, 0};
}
__device__ __forceinline__ int most_tiles(const Block &b) { return max(b.tiles0, b.tiles1); }
__device__ __forceinline__ int tiles_at(const Block &b, int t) { return t == 0 ? b.tiles0 : b.tiles1; }
__device__ __forceinline__ bool run_apart(const Block &b) { return min(b.tiles0, b.tiles1) >= kApart; }

// ------------------------------------------------------------------- planning
__device__ __forceinline__ unsigned long long warp_total(unsigned long long v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// Items are sorted by their key tiles into classes: one a number up to kExact,
// then 32 an octave (up to 2^24 tiles, all that 2^31 keys can make).
constexpr int kExactLog = 9, kExact = 1 << kExactLog;
static_assert(kExact + 32 * (25 - kExactLog) <= kBuckets, "classes");
__device__ __forceinline__ int class_of(int tiles) {
    if (tiles < kExact) return tiles;
    const int e = 31 - __clz(tiles);
    return kExact + (e - kExactLog) * 32 + (tiles >> (e - 5) & 31);
}
__device__ __forceinline__ int most_of_class(int c) {
    return c < kExact ? c : ((33 + (c & 31)) << ((c - kExact) / 32 + kExactLog - 5)) - 1;
}
__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(const PrefillArgs a, const int tpt, const int HV, const int n_blocks) {
    __shared__ int count[kBuckets], warp_sum[kPlanThreads / 32], first_bad, joins, slots, longest;
    __shared__ unsigned long long all_tiles, best;  // best: cost, key tiles of an item
    const int tokens = kM * tpt;  // of a block
    const PrefillLayout L = prefill_layout(a.B, a.Tq, tokens, a.D);
    const int tid = threadIdx.x, lane = tid & 31;
    pdl_trigger();
    count[tid] = 0;
    if (tid == 0) {
        first_bad = 0x7fffffff;
        joins = slots = longest = 0;
        all_tiles = 0;
        best = ~0ull;
    }
    __syncthreads();
    const int64_t room = (int64_t)a.Tq / tokens + a.B + kMaxSms;
    // one warp per sequence, one lane per block: f(block's first token, key tiles)
    auto blocks = [&](auto f) {
        for (int b = tid >> 5; b < a.B; b += kPlanThreads / 32) {
            if (!seq_ok(a, b)) {
                if (lane == 0) atomicMin(&first_bad, b);
                continue;
            }
            const int q0 = __ldg(a.cu_q + b), nq = __ldg(a.cu_q + b + 1) - q0;
            const int k0 = __ldg(a.cu_k + b), nk = __ldg(a.cu_k + b + 1) - k0;
            for (int t0 = lane * tokens; t0 < nq; t0 += 32 * tokens)
                f(block_at(a.causal, q0, nq, k0, nk, t0, tpt));
        }
    };
    auto bucket_of = [&](int tiles) {  // fewest key tiles last
        return kBuckets - 1 - class_of(tiles);
    };
    // Blocks by their key tiles, if none is cut; all key tiles; the most.
    unsigned long long mine_tiles = 0;
    int longest_mine = 0;
    blocks([&](const Block &e) {
        const int tiles = most_tiles(e);
        mine_tiles += tiles;
        longest_mine = max(longest_mine, tiles);
        atomicAdd(&count[bucket_of(tiles)], 1);
    });
    int most = 0x7fffff;  // key tiles of an item
    if (a.Tk > kMinKeys) {
        mine_tiles = warp_total(mine_tiles);
        longest_mine = __reduce_max_sync(0xffffffffu, longest_mine);
        if (lane == 0 && mine_tiles) {
            atomicAdd(&all_tiles, mine_tiles);
            atomicMax(&longest, longest_mine);
        }
        __syncthreads();
        // Warp n looks at the longest key range in n + 1 parts, the last one at
        // parts of an even share of everything, and what that leaves the
        // busiest block to do: its items one after another if they are few,
        // little more than the share if they are many; and parts have to be
        // written, read and joined.  (A cut of everything above the share: 76
        // us instead of 54 for 1024 rows over 4096 keys, 32 heads over 4, 65
        // instead of 37 for 16 sequences of 64 rows over 2048.)
        // (64-bit divisions take long, and these operands are small as a rule)
        auto by_blocks = [&](int64_t x) {
            return x >> 32 ? (x + n_blocks - 1) / n_blocks : (int64_t)(((uint32_t)x - 1) / n_blocks + 1);
        };
        const int64_t share = all_tiles ? by_blocks(all_tiles * HV) : 0;
        const int64_t least = max(share, (int64_t)kMinPart);
        if (longest > least) {
            const int n = tid >> 5;
            const uint32_t m = n == 31 ? (uint32_t)least : ((uint32_t)longest + n) / (n + 1);
            uint32_t big = 0, parts = 0;  // items above half of m; parts of cut ranges
            if (n == 0 || m >= least)
                for (int i = lane, last = class_of(longest); i <= last; i += 32) {
                    const uint32_t tiles = min(longest, most_of_class(i)), c = count[kBuckets - 1 - i];
                    if (c == 0 || 2 * tiles <= m) continue;
                    const uint32_t in = c * ((tiles + m - 1) / m);
                    big += in;
                    if (tiles > m) parts += in;
                }
            const int64_t all_big = (int64_t)__reduce_add_sync(0xffffffffu, big) * HV;
            const int64_t all_parts = (int64_t)__reduce_add_sync(0xffffffffu, parts) * HV;
            const int64_t rounds = max(share, min(all_big ? by_blocks(all_big) * m : 0, share + m));
            const int64_t cost = kRound * rounds + (all_parts ? kJoinCost + all_parts * kPartCost : 0);
            if (lane == 0 && (n == 0 || m >= least)) atomicMin(&best, (unsigned long long)cost << 32 | m);
            __syncthreads();
            most = (int)(best & 0xffffffffu);
        }
    }
    __syncthreads();
    const bool cut = longest > most;
    auto parts_of = [&](const Block &e) {
        return cut ? max(1, (most_tiles(e) + most - 1) / most) : 1;
    };
    if (cut) {  // count again, by parts
        count[tid] = 0;
        __syncthreads();
        blocks([&](const Block &e) {
            // n parts: the first `longer` of base + 1 key tiles, the others of base
            const int tiles = most_tiles(e), n = parts_of(e);
            const int base = tiles / n, longer = tiles % n;
            if (longer) atomicAdd(&count[bucket_of(base + 1)], longer);
            atomicAdd(&count[bucket_of(base)], n - longer);
        });
        __syncthreads();
    }
    // counts -> first places
    const int mine = count[tid];
    int scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) warp_sum[tid >> 5] = scan;
    __syncthreads();
    const int before = __reduce_add_sync(0xffffffffu, lane < tid >> 5 ? warp_sum[lane] : 0);
    count[tid] = before + scan - mine;
    const int total = before + scan;  // (of the last thread: of all)
    __syncthreads();
    blocks([&](const Block &e) {
        const int n = parts_of(e);
        int slot = -1;
        if (n > 1) {
            slot = atomicAdd(&slots, n * HV);
            const int at = atomicAdd(&joins, 1);
            // (a block of T > most key tiles has n < 2 T / most parts, and
            // most is at least all tiles / n_blocks: at most 2 n_blocks parts
            // in all)
            reinterpret_cast<Split *>(a.workspace + L.splits)[at] = Split{e.q0, e.nq, e.tok0, slot, n, {0, 0, 0}};
        }
        const int tiles = most_tiles(e), base = tiles / n, longer = tiles % n;
        const int at0 = longer ? atomicAdd(&count[bucket_of(base + 1)], longer) : 0;
        const int at1 = atomicAdd(&count[bucket_of(base)], n - longer);
        for (int p = 0; p < n; ++p) {
            Block x = e;
            x.j0 = p * base + min(p, longer);
            const int j1 = x.j0 + base + (p < longer ? 1 : 0);
            x.tiles0 = max(0, min(j1, e.tiles0) - x.j0);
            x.tiles1 = max(0, min(j1, e.tiles1) - x.j0);
            x.slot = slot;
            x.parts = n;
            x.part = p;
            const int at = p < longer ? at0 + p : at1 + p - longer;
            // (overlapping sequences may ask for more items than rows)
            if (at < room) reinterpret_cast<Block *>(a.workspace + L.list)[at] = x;
        }
    });
    __syncthreads();
    if (tid == kPlanThreads - 1) {
        *reinterpret_cast<PlanHead *>(a.workspace + L.head) =
            PlanHead{(int)min((int64_t)total, room), 0, joins, slots};
        Ctrl *ctrl = reinterpret_cast<Ctrl *>(a.workspace);
        ctrl->status = first_bad == 0x7fffffff ? MOE_OK : MOE_ERR_DEVICE_BAD_INDEX;
        ctrl->detail = first_bad == 0x7fffffff ? 0 : first_bad;
    }
}

// ------------------------------------------------------------------ the products
// kind::f16 with bf16 operands and fp32 sums; trans_b: B is stored along N.
__host__ __device__ constexpr uint32_t idesc_bf16(uint32_t n, bool trans_b) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((trans_b ? 1u : 0u) << 16) | ((n >> 3) << 17) |
           ((128u >> 4) << 24);
}
// Values [key][d] as the operand whose contraction runs over the keys:
// 128-byte rows of 64 columns, 8-row groups 1024 bytes apart (stride
// offset), the second 64 columns `half` bytes on (leading offset).
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t addr, uint32_t half) {
    uint64_t d = 0;
    d |= (uint64_t)((addr >> 4) & 0x3FFFu);
    d |= (uint64_t)(half >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
__device__ __forceinline__ void mma_bf16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
        "%30, %31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
          "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
          "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]),
          "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]),
          "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// x * a + b and x + y on pairs of fp32
__device__ __forceinline__ float2 fma2(float2 x, float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, a, b, r;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 a, {%4, %5};\n\t"
        "mov.b64 b, {%6, %7};\n\tfma.rn.f32x2 r, x, a, b;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, r;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 r, x, y;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return r;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
prefill_kernel(const PrefillArgs a, const int HT, const bool planned, const __grid_constant__ CUtensorMap map_q,
               const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
    using C = Cfg<D>;
    constexpr int S = C::kStages;
    constexpr int kHalves = D / 64;
    constexpr uint32_t kQHalf = kTile * 128, kKvHalf = kKeys * 128;  // 64 columns of a tile
    extern __shared__ uint8_t raw[];
    const uint32_t raw_u = smem_u32(raw);
    uint8_t *base = raw + ((1024 - (raw_u & 1023)) & 1023);
    uint8_t *kv_base = base + kM * C::kQB;
    const uint32_t q_smem = smem_u32(base), kv_smem = smem_u32(kv_base);
    Shared *sm = reinterpret_cast<Shared *>(kv_base + (size_t)S * C::kKvB);
    // (a broadcast tells the compiler that these are the same in all lanes:
    // the copy and product instructions want their operands in uniform registers)
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int G = a.Hq / a.Hkv, Gt = tile_heads(G), tpt = tile_tokens(G);
    const PrefillLayout L = prefill_layout(a.B, a.Tq, kM * tpt, D);
    Ctrl *ctrl = reinterpret_cast<Ctrl *>(a.workspace);

    if (warp == kMmaWarp) tmem_alloc(&sm->tmem, 512);
    if (threadIdx.x == 0) {
        for (int t = 0; t < kM; ++t) {
            mbar_init(&sm->q_full[t], 1);
            mbar_init(&sm->q_empty[t], 1);
            mbar_init(&sm->s_full[t], 1);
            mbar_init(&sm->s_free[t], 4);
            for (int h = 0; h < kParts; ++h) mbar_init(&sm->p_ready[t][h], 4);
            mbar_init(&sm->o_done[t], 1);
        }
        for (int n = 0; n < 2; ++n) {
            mbar_init(&sm->item_full[n], 1);
            mbar_init(&sm->item_empty[n], 5 * kM + 1);  // all warps but the copying one
        }
        for (int i = 0; i < S; ++i) {
            mbar_init(&sm->kv_full[i], 1);
            mbar_init(&sm->kv_empty[i], kM);
            mbar_init(&sm->tail[i], 1);
        }
        mbar_init(&sm->offset, C::kOwnP ? 1 : 4);
        mbar_init(&sm->finished, kM);
        fence_barrier_init();
        sm->abort = 0;
        prefetch_tensormap(&map_q);
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // S_t, O_t and P_t in tensor memory, all of which is this block's: its
    // address is 0 (anything else is reported like a wait that gave up)
    if (sm->tmem != 0) sm->abort = 20;
    constexpr uint32_t s_col = 0, o_col = kM * kKeys;
    constexpr uint32_t p_col = C::kOwnP ? o_col + kM * D : s_col;
    constexpr uint32_t kPStep = C::kOwnP ? kKeys / 2 : kKeys;
    static_assert(kM * (kKeys + D + (C::kOwnP ? kKeys / 2 : 0)) <= 512, "tensor memory");

    // The next item; false when there is none or a wait gave up.  Every role
    // but the copying one walks the items with this.
    auto take = [&](uint32_t n, Item &it) {
        if (!warp_wait_flag(&sm->item_full[n & 1], (n >> 1) & 1, &sm->abort, 1)) return false;
        it = sm->item[n & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->item_empty[n & 1]);
        return it.done == 0;
    };
    // A value tile whose rows past the sequence's end belong to others.
    auto ragged = [&](const Item &it, int j) {
        return (it.b.j0 + j + 1) * kKeys > it.b.nk && it.b.k0 + it.b.nk < a.Tk;
    };

    if (warp >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRoleRegs));
        if (warp == kLoadWarp) {
            // ---------------- copies, and the items for everyone
            const int HV = a.Hkv * HT;
            const Block *list = reinterpret_cast<const Block *>(a.workspace + L.list);
            int *counter = &reinterpret_cast<PlanHead *>(a.workspace + L.head)->next;
            // Without a plan, lane b has sequence b: its rows, and how many
            // blocks the sequences up to it have.
            int q0 = 0, nq = 0, k0 = 0, nk = 0, up_to = 0;
            int64_t total;
            if (planned) {
                pdl_wait();
                total = (int64_t)*(volatile const int32_t *)&reinterpret_cast<const PlanHead *>(
                            a.workspace + L.head)->items * HV;
            } else {
                const bool ok = lane >= a.B || seq_ok(a, lane);
                if (lane < a.B && ok) {
                    q0 = __ldg(a.cu_q + lane);
                    nq = __ldg(a.cu_q + lane + 1) - q0;
                    k0 = __ldg(a.cu_k + lane);
                    nk = __ldg(a.cu_k + lane + 1) - k0;
                }
                up_to = (nq + kM * tpt - 1) / (kM * tpt);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, up_to, o);
                    if (lane >= o) up_to += v;
                }
                total = (int64_t)__shfl_sync(0xffffffffu, up_to, 31) * HV;
                const uint32_t bad = __ballot_sync(0xffffffffu, !ok);
                if (blockIdx.x == 0 && lane == 0) {
                    ctrl->status = bad ? MOE_ERR_DEVICE_BAD_INDEX : MOE_OK;
                    ctrl->detail = bad ? __ffs(bad) - 1 : 0;
                }
            }
            auto entry = [&](int64_t i) {
                if (planned) return list[i];
                // the sequence whose blocks hold number i, its longest block first
                const int b = min(31, __popc(__ballot_sync(0xffffffffu, up_to <= i)));
                const int sq0 = __shfl_sync(0xffffffffu, q0, b), snq = __shfl_sync(0xffffffffu, nq, b);
                const int sk0 = __shfl_sync(0xffffffffu, k0, b), snk = __shfl_sync(0xffffffffu, nk, b);
                const int left = __shfl_sync(0xffffffffu, up_to, b) - 1 - (int)i;
                return block_at(a.causal, sq0, snq, sk0, snk, left * kM * tpt, tpt);
            };
            // Item n + 1's entry and item n + 2's number are fetched while
            // item n's copies are issued.
            int64_t idx = blockIdx.x;
            int64_t ahead = idx;  // (lane 0)
            auto next_ahead = [&]() {
                if (!planned)
                    ahead += gridDim.x;
                else if (lane == 0)
                    ahead = (int64_t)gridDim.x + atomicAdd(counter, 1);
            };
            next_ahead();
            Block blk = idx < total ? entry(idx / HV) : Block{};
            uint32_t n = 0, kv = 0;
            for (;; ++n) {
                Item it;
                it.b = blk;
                it.done = idx >= total;
                const int hv = (int)(idx % HV), g0 = (hv % HT) * Gt;
                it.hk = hv / HT;
                it.h0 = it.hk * G + g0;
                it.heads = min(Gt, G - g0);
                it.slot = blk.slot < 0 ? -1 : blk.slot + hv * blk.parts + blk.part;
                if (!warp_wait_flag(&sm->item_empty[n & 1], ((n >> 1) & 1) ^ 1, &sm->abort, 2)) break;
                if (lane == 0) {
                    sm->item[n & 1] = it;
                    mbar_arrive(&sm->item_full[n & 1]);
                }
                __syncwarp();
                if (it.done) break;
                idx = __shfl_sync(0xffffffffu, ahead, 0);
                if (idx < total) blk = entry(idx / HV);
                next_ahead();
                const int tiles = most_tiles(it.b);
                bool ok = true;
                auto copy_kv = [&](const CUtensorMap *map, int j, bool tail) {
                    const uint32_t s = kv % S, ph = (kv / S) & 1;
                    ok = ok && warp_wait_flag(&sm->kv_empty[s], ph ^ 1, &sm->abort, 3);
                    if (!ok) return;
                    if (lane == 0) {
                        uint64_t *bar = tail ? &sm->tail[s] : &sm->kv_full[s];
                        mbar_arrive_expect_tx(bar, C::kKvB);
                        tma_load_4d(kv_base + s * C::kKvB, map, 0, it.b.k0 + (it.b.j0 + j) * kKeys, it.hk, 0, bar);
                    }
                    __syncwarp();
                    ++kv;
                };
                for (int j = 0; j < tiles && ok && !a.test_no_copies; ++j) {
                    if (!C::kOwnP || j == 0) copy_kv(&map_k, j, false);
                    if (j == 0) {
                        for (int t = 0; t < kM && ok; ++t) {
                            ok = warp_wait_flag(&sm->q_empty[t], (n & 1) ^ 1, &sm->abort, 4);
                            if (ok && lane == 0) {
                                // (a tile without rows is loaded all the same: its phases go on)
                                mbar_arrive_expect_tx(&sm->q_full[t], (uint32_t)(Gt * tpt) * D * 2);
                                for (int h = 0; h < kHalves; ++h)
                                    tma_load_4d(base + t * C::kQB + h * kQHalf, &map_q, 0, it.h0,
                                                it.b.q0 + it.b.tok0 + t * tpt, h, &sm->q_full[t]);
                            }
                            __syncwarp();
                        }
                    }
                    // (in the order in which the products want them)
                    if (C::kOwnP && ok && j + 1 < tiles) copy_kv(&map_k, j + 1, false);
                    if (ok) copy_kv(&map_v, j, ragged(it, j));
                }
                if (!ok) break;
                if (tiles == 0) {
                    // no copies: the other roles' phases of q go on without them
                    for (int t = 0; t < kM && ok; ++t) {
                        ok = warp_wait_flag(&sm->q_empty[t], (n & 1) ^ 1, &sm->abort, 4);
                        if (ok && lane == 0) mbar_arrive(&sm->q_full[t]);
                        __syncwarp();
                    }
                    if (!ok) break;
                }
            }
            // (after a give-up) nothing of this warp's may still be in flight
            if (*(volatile int *)&sm->abort) {
                const long long t0 = clock64();
                while (clock64() - t0 < (1ll << 24)) __nanosleep(1000);
            }
        } else if (warp < kLoadWarp) {
            // ---------------- products of row tile t
            auto products = [&](auto tile) {
                constexpr int t = decltype(tile)::value;
                const uint64_t q_desc = sdesc_k_sw128(q_smem), k_desc = sdesc_k_sw128(kv_smem);
                const uint64_t v_desc = sdesc_mn_sw128(kv_smem, kKvHalf);
                constexpr uint32_t kIdS = idesc_bf16(kKeys, false), kIdO = idesc_bf16(D, true);
                uint32_t stage = 0, stage_ph = 0;         // the next key or value tile
                uint32_t p_ph = 0, f_ph = 1, off_ph = 0;
                Item it;
                bool ok = true;
                const uint64_t qd = q_desc + ((t * C::kQB) >> 4);
                constexpr uint32_t s_t = s_col + t * kKeys, o_t = o_col + t * D, p_t = p_col + t * kPStep;
                auto commit = [&](uint64_t *bar) {
                    if (elect_one()) tc_commit(bar);
                    __syncwarp();
                };
                auto next_stage = [&]() {  // waits for the next key or value tile
                    ok = ok && warp_wait_flag(&sm->kv_full[stage], stage_ph, &sm->abort, 5);
                    tc_fence_after();
                    const uint32_t s = stage;
                    if (++stage == S) {
                        stage = 0;
                        stage_ph ^= 1;
                    }
                    return s;
                };
                // S_t = Q_t K^T; `last`: of this item, so that Q_t is free after it
                auto qk = [&](uint32_t s, bool last) {
                    if (C::kOwnP) {  // (else the last product with P_t came before)
                        ok = ok && warp_wait_flag(&sm->s_free[t], f_ph, &sm->abort, 12);
                        if (!ok) return;
                        f_ph ^= 1;
                        tc_fence_after();
                    }
                    if (elect_one()) {
                        const uint64_t kd = k_desc + ((s * C::kKvB) >> 4);
#pragma unroll
                        for (int j = 0; j < D / 16; ++j) {
                            const uint32_t in = (j & 3) * 32;
                            mma_bf16_ss(s_t, qd + (((j >> 2) * kQHalf + in) >> 4), kd + (((j >> 2) * kKvHalf + in) >> 4),
                                        kIdS, j > 0);
                        }
                        tc_commit(&sm->s_full[t]);
                        tc_commit(&sm->kv_empty[s]);
                        if (last) tc_commit(&sm->q_empty[t]);
                    }
                    __syncwarp();
                };
                // O_t += P_t V, in the parts in which the weights come
                auto pv = [&](uint32_t s, bool first, bool tell) {
                    const uint64_t vd = v_desc + ((s * C::kKvB) >> 4);
                    constexpr int kSteps = kKeys / 16 / kParts;
#pragma unroll
                    for (int h = 0; h < kParts; ++h) {
                        ok = ok && warp_wait_flag(&sm->p_ready[t][h], p_ph, &sm->abort, 7);
                        if (!ok) return;
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int i = h * kSteps; i < (h + 1) * kSteps; ++i)
                                mma_f16_ts(o_t, p_t + i * 8, vd + ((i * 2048) >> 4), kIdO,
                                           i > 0 ? 1u : (first ? 0u : 1u));
                            if (h == kParts - 1) {
                                tc_commit(&sm->o_done[t]);
                                tc_commit(&sm->kv_empty[s]);
                            }
                        }
                        __syncwarp();
                        if (tell && h == 0 && lane == 0) mbar_arrive(&sm->offset);
                    }
                    p_ph ^= 1;
                };
                for (uint32_t n = 0; ok && take(n, it); ++n) {
                    const int nt = __shfl_sync(0xffffffffu, tiles_at(it.b, t), 0);
                    const int tiles = __shfl_sync(0xffffffffu, most_tiles(it.b), 0);
                    uint32_t s = 0;
                    if (tiles > 0) s = next_stage();
                    ok = ok && warp_wait_flag(&sm->q_full[t], n & 1, &sm->abort, 6);
                    if (!ok) break;
                    tc_fence_after();
                    // The second tile starts behind the first: two tiles in step
                    // would want the tensor pipe, and then the exponentials, at
                    // the same time.  Heads of 128: once the first tile's maxima
                    // are known, which puts the two half a round apart (8192
                    // causal tokens, 64 heads, when this was chosen: 606 us, 640
                    // with the signal below, 656 in step); heads of 64: once the
                    // first half of its weights is (455, 483 the other way, 484
                    // in step).
                    const bool apart = __shfl_sync(0xffffffffu, (int)run_apart(it.b), 0) != 0;
                    if (apart && t == 1) {
                        ok = warp_wait_flag(&sm->offset, off_ph, &sm->abort, 13);
                        if (!ok) break;
                        off_ph ^= 1;
                    }
                    if (nt > 0)
                        qk(s, nt == 1);
                    else {  // (the other tile's stages, and a Q_t that is not used)
                        commit(&sm->q_empty[t]);
                        if (tiles > 0) commit(&sm->kv_empty[s]);
                    }
                    // the scores of key tile j + 1
                    auto next_scores = [&](int j) {
                        if (j + 1 >= tiles) return;
                        const uint32_t k = next_stage();
                        if (!ok) return;
                        if (j + 1 < nt)
                            qk(k, j + 2 == nt);
                        else
                            commit(&sm->kv_empty[k]);
                    };
                    for (int j = 0; j < tiles && ok; ++j) {
                        if (C::kOwnP) next_scores(j);
                        const uint32_t v = next_stage();
                        if (!ok) break;
                        if (j < nt)
                            pv(v, j == 0, C::kOwnP && j == 0 && apart && t == 0);
                        else
                            commit(&sm->kv_empty[v]);
                        if (!C::kOwnP && ok) next_scores(j);
                    }
                }
                // everything issued has finished before the block ends
                commit(&sm->finished);
                wait_own(&sm->finished, 0);
            };
            if (warp == kMmaWarp)
                products(std::integral_constant<int, 0>{});
            else
                products(std::integral_constant<int, 1>{});
        } else if (warp == kFixWarp) {
            // ---------------- last value tiles: zeros past the sequence's end
            Item it;
            uint32_t kv = 0, ph = 0;  // ph: one phase bit per stage
            for (uint32_t n = 0; take(n, it); ++n) {
                const int tiles = most_tiles(it.b);
                kv += 2 * tiles;
                if (tiles == 0 || !ragged(it, tiles - 1)) continue;
                const uint32_t s = (kv - 1) % S;
                if (!warp_wait_flag(&sm->tail[s], (ph >> s) & 1, &sm->abort, 8)) break;
                ph ^= 1u << s;
                uint8_t *v = kv_base + s * C::kKvB;
                const int from = it.b.nk - (it.b.j0 + tiles - 1) * kKeys;
                for (int h = 0; h < kHalves; ++h)
                    for (int i = from * 8 + lane; i < kKeys * 8; i += 32)
                        *reinterpret_cast<uint4 *>(v + h * kKvHalf + i * 16) = make_uint4(0, 0, 0, 0);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->kv_full[s]);
            }
        }
    } else {
        // ---------------- softmax: warpgroup t has row tile t, a thread a row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int t = warp >> 2;
        const int r = threadIdx.x & 127;
        const uint32_t lane_base = (uint32_t)(warp & 3) * 32 << 16;
        const uint32_t s_t = s_col + t * kKeys + lane_base, o_t = o_col + t * D + lane_base;
        const uint32_t p_t = p_col + t * kPStep + lane_base;
        const int tok_r = r / Gt, g = r % Gt;
        const float sl = a.scale * kLog2e;
        uint32_t ph = 0;  // parity of this warpgroup's count of key tiles
        // A wait costs about 200 cycles even when its phase is over.  Where the
        // phases usually are (heads of 64), they are tested ahead, and the
        // answer used when it has come.
        bool s_seen = false, o_seen = false;
        Item it;
        bool ok = true;
        for (uint32_t n = 0; ok && take(n, it); ++n) {
            const int tok = it.b.tok0 + t * tpt + tok_r;
            const bool live = tok_r < tpt && tok < it.b.nq && g < it.heads;
            // (rows that do not exist ask for no masking)
            const int limit = live ? keys_seen(a.causal, tok, it.b.nq, it.b.nk) : 0x3fffffff;
            const int least = __reduce_min_sync(0xffffffffu, limit);
            float ref = -INFINITY;  // the row's reference, in log2 units
            float l = 0.f;
            const int tiles = tiles_at(it.b, t);
            const bool apart = run_apart(it.b);
            for (int j = 0; j < tiles; ++j) {
                if (!C::kOwnP || !__all_sync(0xffffffffu, s_seen)) {
                    ok = warp_wait_flag(&sm->s_full[t], ph, &sm->abort, 9);
                    if (!ok) break;
                }
                tc_fence_after();
                float x[kKeys];
#pragma unroll
                for (int c = 0; c < kKeys; c += 32) tmem_ld32(s_t + c, x + c);
                tc_wait_ld();
                if (C::kOwnP) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm->s_free[t]);
                    o_seen = mbar_test_wait(&sm->o_done[t], ph ^ 1);
                }
                const int key0 = (it.b.j0 + j) * kKeys;
                if (key0 + kKeys > least) {
                    const int lim = limit - key0;
#pragma unroll
                    for (int c = 0; c < kKeys; c += 32)
                        if (key0 + c + 32 > least) {
#pragma unroll
                            for (int e = c; e < c + 32; ++e) x[e] = e < lim ? x[e] : -INFINITY;
                        }
                }
                float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int c = 4; c + 8 <= kKeys; c += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e) m4[e] = max3(m4[e], x[c + 2 * e], x[c + 2 * e + 1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) m4[e] = fmaxf(m4[e], x[kKeys - 4 + e]);
                const float top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * sl;
                const bool raise = top > ref + kSlack;
                bool over = !C::kOwnP || j == 0;  // P_t may be written
                if (__any_sync(0xffffffffu, raise)) {
                    const float to = raise ? top : ref;
                    const float f = raise ? ex2(ref - to) : 1.f;
                    l *= f;
                    ref = to;
                    if (j > 0) {
                        // the last product into O_t has to be over
                        ok = warp_wait_flag(&sm->o_done[t], ph ^ 1, &sm->abort, 10);
                        if (!ok) break;
                        over = true;
                        tc_fence_after();
#pragma unroll
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(o_t + c, o);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st16(o_t + c, o);
                        }
                    }
                }
                // the last product with P_t has to be over
                if (!over && !__all_sync(0xffffffffu, o_seen)) {
                    ok = warp_wait_flag(&sm->o_done[t], ph ^ 1, &sm->abort, 10);
                    if (!ok) break;
                }
                if (C::kOwnP) tc_fence_after();
                if (!C::kOwnP && t == 0 && j == 0 && apart && lane == 0) mbar_arrive(&sm->offset);
                const float z = ref == -INFINITY ? 0.f : ref;
                const float2 sl2 = make_float2(sl, sl), nz2 = make_float2(-z, -z);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < kKeys; c += 32) {
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float2 y = fma2(make_float2(x[c + 2 * e], x[c + 2 * e + 1]), sl2, nz2);
                        y.x = ex2(y.x);
                        y.y = ex2(y.y);
                        sum[e & 1] = add2(sum[e & 1], y);
                        p[e] = pack_bf16(y.x, y.y);
                    }
                    if (C::kOwnP && c + 32 == kKeys) s_seen = mbar_test_wait(&sm->s_full[t], ph ^ 1);
                    tmem_st16(p_t + c / 2, p);
                    if ((c + 32) % (kKeys / kParts) == 0) {  // their product may start
                        tc_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm->p_ready[t][c / (kKeys / kParts)]);
                    }
                }
                const float2 both = add2(sum[0], sum[1]);
                l += both.x + both.y;
                ph ^= 1;
            }
            if (!ok) break;
            // ---- the rows' outputs
            const float inv = 1.f / l;
            const bool none = l == 0.f;  // no key: zeros
            if (it.slot >= 0) {  // one part of several: its sums as they are
                if (tiles > 0) {
                    ok = warp_wait_flag(&sm->o_done[t], ph ^ 1, &sm->abort, 11);
                    if (!ok) break;
                    tc_fence_after();
                }
                float *to = reinterpret_cast<float *>(a.workspace + L.sums);
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    if (tiles > 0) {
                        tmem_ld32(o_t + c, o);
                        tc_wait_ld();
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0.f;
                    }
                    if (live)
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4 *>(to + part_at(it.slot, t, c + e, r, D)) =
                                make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
                if (live)
                    reinterpret_cast<float2 *>(a.workspace + L.ml)[((size_t)it.slot * kM + t) * kTile + r] =
                        make_float2(ref, l);
                tc_fence_before();
                continue;
            }
            // Four neighbouring lanes hand each other 16-byte pieces, so that
            // a store covers 64 bytes of each of 8 rows: this lane's rows are
            // then those of its four, its piece lane % 4.
            uint16_t *rows[4];
            const int64_t at = live ? (int64_t)(it.b.q0 + tok) * a.out_stride + (it.h0 + g) * D : -1;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t v = __shfl_sync(0xffffffffu, at, (lane & ~3) + k);
                rows[k] = v < 0 ? nullptr : a.out + v + (lane & 3) * 8;
            }
            if (tiles > 0) {
                ok = warp_wait_flag(&sm->o_done[t], ph ^ 1, &sm->abort, 11);
                if (!ok) break;
                tc_fence_after();
            }
#pragma unroll
            for (int c = 0; c < D; c += 32) {
                float o[32];
                if (tiles > 0) {
                    tmem_ld32(o_t + c, o);
                    tc_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.f;
                }
                uint32_t u[4][4];  // [piece of 8 columns][word]
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    u[e / 4][e % 4] = none ? 0u : pack_bf16(o[2 * e] * inv, o[2 * e + 1] * inv);
                // a 4 x 4 transposition of pieces in two exchanges
#pragma unroll
                for (int b = 1; b < 4; b <<= 1) {
                    const bool up = (lane & b) != 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (k & b) continue;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t give = up ? u[k][e] : u[k | b][e];
                            const uint32_t got = __shfl_xor_sync(0xffffffffu, give, b);
                            if (up) u[k][e] = got; else u[k | b][e] = got;
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (rows[k])
                        *reinterpret_cast<uint4 *>(rows[k] + c) = make_uint4(u[k][0], u[k][1], u[k][2], u[k][3]);
            }
            if (a.lse && live)
                a.lse[(size_t)(it.b.q0 + tok) * a.Hq + it.h0 + g] =
                    none ? -INFINITY : (ref + __log2f(l)) * kLn2;
            // (O_t is read: the next item's first p_ready comes after this)
            tc_fence_before();
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && sm->abort) set_status(ctrl, MOE_ERR_DEVICE_TIMEOUT, sm->abort);
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_relinquish();
        tmem_dealloc(sm->tmem, 512);
    }
}

// Joins the parts of cut key ranges, 32 neighbouring rows (a lane each) and 8
// columns at a time.  Up to kFewParts parts: by one warp, all of its loads in
// flight (4 sequences of 100 rows over 3000 keys, 32 heads over 4: the call 45
// -> 41 us).  More: by a block, whose warps take every fourth part; their sums
// are then added in order.
constexpr int kJoinWarps = 4, kFewParts = 8;

// The sums of some parts of a row's 8 columns.
struct PartSums {
    float top = -INFINITY, sum = 0.f, o[8] = {};
};
// Parts first, first + step, ... of a block of `parts` whose first has place
// `slot`: row r of row tile t, columns c to c + 7.
template <int D>
__device__ __forceinline__ PartSums take_parts(const float2 *ml, const float *sums, int slot, int parts, int first,
                                               int step, int t, int c, int r) {
    PartSums x;
#pragma unroll 8
    for (int p = first; p < parts; p += step)
        x.top = fmaxf(x.top, ml[((size_t)(slot + p) * kM + t) * kTile + r].x);
    const float z = x.top == -INFINITY ? 0.f : x.top;
#pragma unroll 8
    for (int p = first; p < parts; p += step) {
        const float2 v = ml[((size_t)(slot + p) * kM + t) * kTile + r];
        const float4 lo = *reinterpret_cast<const float4 *>(sums + part_at(slot + p, t, c, r, D));
        const float4 hi = *reinterpret_cast<const float4 *>(sums + part_at(slot + p, t, c + 4, r, D));
        const float f = ex2(v.x - z);
        const bool empty = v.x == -INFINITY && v.y == 0.f;  // no key of this part
        const float e[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        x.sum = empty ? x.sum : fmaf(f, v.y, x.sum);
#pragma unroll
        for (int i = 0; i < 8; ++i) x.o[i] = empty ? x.o[i] : fmaf(f, e[i], x.o[i]);
    }
    return x;
}

template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const PrefillArgs a, const int HT) {
    __shared__ float shared[kJoinWarps][10][32];  // per warp: maximum, sum, 8 columns
    pdl_wait();
    const int G = a.Hq / a.Hkv, Gt = tile_heads(G), tpt = tile_tokens(G), HV = a.Hkv * HT;
    const PrefillLayout L = prefill_layout(a.B, a.Tq, kM * tpt, D);
    const PlanHead head = *reinterpret_cast<const PlanHead *>(a.workspace + L.head);
    const float2 *ml = reinterpret_cast<const float2 *>(a.workspace + L.ml);
    const float *sums = reinterpret_cast<const float *>(a.workspace + L.sums);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kCols = D / 8, kRowGroups = kTile / 32;
    const int64_t work = (int64_t)head.joins * HV * kM * kRowGroups * kCols;
    // What number w is: a lane's row (if it has one), its part and its columns.
    struct Work {
        int t, c, r, h, slot, parts, tok;
        int64_t row;  // of q, -1: none
    };
    auto work_of = [&](int64_t w) {
        Work k;
        k.c = (int)(w % kCols) * 8;
        k.r = (int)(w / kCols) % kRowGroups * 32 + lane;
        k.t = (int)(w / (kCols * kRowGroups)) % kM;
        const int64_t bh = w / (kM * kCols * kRowGroups);
        const Split sp = reinterpret_cast<const Split *>(a.workspace + L.splits)[bh / HV];
        const int hv = (int)(bh % HV), g0 = (hv % HT) * Gt, g = k.r % Gt;
        k.tok = sp.tok0 + k.t * tpt + k.r / Gt;
        const bool live = k.r / Gt < tpt && k.tok < sp.nq && g < min(Gt, G - g0);
        k.row = live ? (int64_t)sp.q0 + k.tok : -1;
        k.h = (hv / HT) * G + g0 + g;
        k.slot = sp.slot + hv * sp.parts;
        k.parts = sp.parts;
        return k;
    };
    auto put = [&](const Work &k, const PartSums &x) {
        const bool none = x.sum == 0.f;
        const float inv = 1.f / x.sum;
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = none ? 0.f : x.o[i] * inv;
        *reinterpret_cast<uint4 *>(a.out + k.row * a.out_stride + k.h * D + k.c) =
            make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
        if (a.lse && k.c == 0)
            a.lse[(size_t)k.row * a.Hq + k.h] = none ? -INFINITY : (x.top + __log2f(x.sum)) * kLn2;
    };
    for (int64_t w = (int64_t)blockIdx.x * kJoinWarps + warp; w < work; w += gridDim.x * kJoinWarps) {
        const Work k = work_of(w);
        if (k.parts <= kFewParts && k.row >= 0)
            put(k, take_parts<D>(ml, sums, k.slot, k.parts, 0, 1, k.t, k.c, k.r));
    }
    for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
        const Work k = work_of(w);
        // (both the same in all warps)
        if (k.parts <= kFewParts || !__any_sync(0xffffffffu, k.row >= 0)) continue;
        PartSums x;
        if (k.row >= 0) x = take_parts<D>(ml, sums, k.slot, k.parts, warp, kJoinWarps, k.t, k.c, k.r);
        shared[warp][0][lane] = x.top;
        shared[warp][1][lane] = x.sum;
#pragma unroll
        for (int i = 0; i < 8; ++i) shared[warp][2 + i][lane] = x.o[i];
        __syncthreads();
        if (warp == 0 && k.row >= 0) {
#pragma unroll
            for (int p = 1; p < kJoinWarps; ++p) x.top = fmaxf(x.top, shared[p][0][lane]);
            const float z = x.top == -INFINITY ? 0.f : x.top;
            x.sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) x.o[i] = 0.f;
#pragma unroll
            for (int p = 0; p < kJoinWarps; ++p) {
                const float m = shared[p][0][lane], f = m == -INFINITY ? 0.f : ex2(m - z);
                // (a warp without a key has sums of 0; NaN has no maximum)
                const float s1 = shared[p][1][lane];
                x.sum += m == -INFINITY ? s1 : f * s1;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float e = shared[p][2 + i][lane];
                    x.o[i] += m == -INFINITY ? e : f * e;
                }
            }
            put(k, x);
        }
        __syncthreads();
    }
}

template <int D>
cudaError_t run(const PrefillArgs &a, int sms, cudaStream_t s) {
    using C = Cfg<D>;
    const int G = a.Hq / a.Hkv, Gt = tile_heads(G), tpt = tile_tokens(G), HT = (G + Gt - 1) / Gt;
    CUtensorMap mq, mk, mv;
    {
        const uint64_t dims[4] = {64, (uint64_t)a.Hq, (uint64_t)a.Tq, D / 64};
        const uint64_t strides[3] = {D * 2, (uint64_t)a.q_stride * 2, 128};
        const uint32_t box[4] = {64, (uint32_t)Gt, (uint32_t)tpt, 1};
        if (!encode_tensor_map(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, a.q, dims, strides, box,
                               CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    }
    for (int i = 0; i < 2; ++i) {
        // (no keys at all: nothing is copied, any valid map will do)
        const uint16_t *p = a.Tk > 0 ? (i ? a.v : a.k) : a.q;
        const uint64_t dims[4] = {64, (uint64_t)(a.Tk > 0 ? a.Tk : 1), (uint64_t)a.Hkv, D / 64};
        const uint64_t strides[3] = {(uint64_t)(i ? a.v_stride : a.k_stride) * 2, D * 2, 128};
        const uint32_t box[4] = {64, kKeys, 1, D / 64};
        if (!encode_tensor_map(i ? &mv : &mk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, p, dims, strides,
                               box, CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    }
    // (no key range is cut below this many keys: then no joins either)
    const bool cuts = a.Tk > kMinKeys;
    const int64_t most = ((int64_t)a.Tq / (kM * tpt) + a.B) * a.Hkv * HT;
    if (sms > kMaxSms) sms = kMaxSms;
    const int grid = (int)(cuts || most > sms ? sms : most);
    // (1024 tokens, 32 heads: 20.8 us with a plan, 18.7 without)
    const bool planned = cuts || a.B > 32;
    cudaError_t err = cudaSuccess;
    if (planned) {
        plan_kernel<<<1, kPlanThreads, 0, s>>>(a, tpt, a.Hkv * HT, grid);
        err = cudaGetLastError();
    }
    if (err != cudaSuccess) return err;
    auto fn = prefill_kernel<D>;
    static SmemOnce once;
    err = once.set(reinterpret_cast<const void *>(fn), C::kSmem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = planned ? 1 : 0;
    err = cudaLaunchKernelEx(&cfg, fn, a, HT, planned, mq, mk, mv);
    if (err != cudaSuccess || !cuts) return err;
    cudaLaunchConfig_t cj = {};
    cj.gridDim = dim3(8 * sms);  // (16: up to 2 us more where there is nothing to join)
    cj.blockDim = dim3(32 * kJoinWarps);
    cj.stream = s;
    cj.attrs = at;
    cj.numAttrs = 1;
    return cudaLaunchKernelEx(&cj, join_kernel<D>, a, HT);
}

}  // namespace

size_t prefill_workspace(int B, int Tq, int Hq, int Hkv, int D) {
    return align_up(prefill_layout(B, Tq, kM * tile_tokens(Hq / Hkv), D).total, 256);
}

cudaError_t launch_attn_prefill(const PrefillArgs &a, cudaStream_t s) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const int sms = tc_grid(dev);
    if (sms < 1) return cudaErrorInvalidDevice;
    return a.D == 128 ? run<128>(a, sms, s) : run<64>(a, sms, s);
}

}  // namespace moe
