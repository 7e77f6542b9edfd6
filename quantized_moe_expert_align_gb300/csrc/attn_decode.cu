// attn_decode.cu -- attention of single tokens over the paged cache: every key.
#include "attn_decode.cuh"

namespace moe {

size_t decode_attn_workspace(int, int Hq, int Hkv, int D) {
    return align_up(decode_layout(8 * tiles_of(Hq / Hkv), D).total, 256);
}

cudaError_t launch_attn_decode(const DecodeAttnArgs &a, cudaStream_t s) {
    return launch<kPlain>(a, a.Hq / a.kv.Hkv, s);
}

}  // namespace moe
