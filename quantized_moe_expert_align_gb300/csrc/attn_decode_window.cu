// attn_decode_window.cu -- attention of single tokens over the paged cache
// through a sliding window: the last `window` keys and the first `sinks`.
#include "attn_decode.cuh"

namespace moe {

// Rows of a copy.  Small ones bring less that is not seen, large ones are fewer.  64
// sequences, 64 heads over 8.  bf16, heads of 128, with 16, 32 and 64 rows: window 128
// 15.3, 15.5 and 17.4 us, 512 30.0, 31.4 and 35.8, 2000 87.9, 89.1 and 91.2.  fp8, with 32
// and 64: heads of 128, 1000 35.2 and 36.1, 2000 56.3 and 57.2, 2500 66.0 and 66.0, 6000
// 135.6 and 132.8 (256 sequences: 182.2 and 183.3, 221.4 and 220.7, 492.7 and 485.9); heads
// of 64, 128 11.8 and 12.0, 500 16.6 and 16.4, 1000 22.8 and 22.2, 4000 57.2 and 55.0.
static int box_rows_log(const DecodeAttnArgs &a) {
    const int log = a.cache_type == MOE_KV_BF16 ? 4 : a.window < (a.D == 128 ? 2300 : 500) ? 5 : 6;
    return log < a.kv.page_shift ? log : a.kv.page_shift;
}

cudaError_t launch_attn_decode_window(const DecodeAttnArgs &args, cudaStream_t s) {
    DecodeAttnArgs a = args;
    a.box_shift = box_rows_log(a);
    return launch<kWindow>(a, a.Hq / a.kv.Hkv, s);
}

}  // namespace moe
