// attn_decode_window.cu -- attention of single tokens over the paged cache
// through a sliding window: the last `window` keys and the first `sinks`.
#include "attn_decode.cuh"

namespace moe {

cudaError_t launch_attn_decode_window(const DecodeAttnArgs &args, cudaStream_t s) {
    DecodeAttnArgs a = args;
    a.box_shift = a.window < 1024 ? 4 : a.kv.page_shift < 6 ? a.kv.page_shift : 6;
    return launch<kWindow>(a, a.Hq / a.kv.Hkv, s);
}

}  // namespace moe
