// attn_prefill_window.cu -- attention over packed prompts through a sliding
// window: the last `window` keys up to one's own and the first `sinks`.
#include "attn_prefill.cuh"

namespace moe {

cudaError_t launch_attn_prefill_window(const PrefillArgs &a, cudaStream_t s) { return launch<true>(a, s); }

}  // namespace moe
