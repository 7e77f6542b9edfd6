// attn_tree_small.cu -- attention of drafted tokens over the paged cache, in
// tiles of 8 or 16 rows: for sequences that have few (attn_tree.cu has the rule).
#include "attn_decode.cuh"

namespace moe {

size_t tree_small_workspace(int T, int Hq, int Hkv, int D) {
    const int tokens = T < kTreeTokens ? T : kTreeTokens;
    return align_up(decode_layout(8 * tiles_of(Hq / Hkv * tokens), D).total, 256);
}

cudaError_t launch_attn_tree_small(const DecodeAttnArgs &a, cudaStream_t s) {
    // Tiles of 8 rows where that is what a sequence has on average, or can have: of 8 rows
    // each (64 sequences of 4096 keys, 4 key/value heads, fp8) heads of 128 in 55 us, not
    // 70, heads of 64 in 33, not 49; of 5 to 11 rows 69 and 71, 40 and 49.
    const int G = a.Hq / a.kv.Hkv;
    const bool few = (int64_t)a.T * G <= (int64_t)a.B * 8;
    return launch<kTree>(a, few ? 8 : G * (a.T < kTreeTokens ? a.T : kTreeTokens), s);
}

}  // namespace moe
