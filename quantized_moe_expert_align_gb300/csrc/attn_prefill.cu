// attn_prefill.cu -- attention over packed prompts: all keys, or up to one's own.
#include "attn_prefill.cuh"

namespace moe {

size_t prefill_workspace(int B, int Tq, int Hq, int Hkv, int D) {
    return align_up(prefill_layout(B, Tq, kM * tile_tokens(Hq / Hkv), D).total, 256);
}

cudaError_t launch_attn_prefill(const PrefillArgs &a, cudaStream_t s) { return launch<false>(a, s); }

}  // namespace moe
