// attn_tree_small.cu -- attention of drafted tokens over the paged cache, in
// tiles of up to 16 rows: for sequences that have few (attn_tree.cu has the rule).
#include "attn_decode.cuh"

namespace moe {

size_t tree_small_workspace(int T, int Hq, int Hkv, int D) {
    const int tokens = T < kTreeTokens ? T : kTreeTokens;
    return align_up(decode_layout(8 * tiles_of(Hq / Hkv * tokens), D).total, 256);
}

cudaError_t launch_attn_tree_small(const DecodeAttnArgs &a, cudaStream_t s) {
    return launch<kTree>(a, a.Hq / a.kv.Hkv * (a.T < kTreeTokens ? a.T : kTreeTokens), s);
}

}  // namespace moe
