// attn_decode_window.cu -- attention of single tokens over the paged cache
// through a sliding window: the last `window` keys and the first `sinks`.
#include "attn_decode.cuh"

namespace moe {

// Rows of a copy.  Small ones bring less that is not seen, large ones are fewer.  64
// sequences, 64 heads of 128 over 8, with 16, 32 and 64 rows: bf16, window 128 15.3,
// 15.5 and 17.4 us, 512 30.0, 31.4 and 35.8, 2000 87.9, 89.1 and 91.2; fp8, half the
// bytes a row, 128 15.2, 15.3 and 15.6, 1000 35.7, 34.9 and 35.4, 4096 102, 97.4 and
// 96.5.
static int box_rows_log(const DecodeAttnArgs &a) {
    const int log = a.cache_type == MOE_KV_BF16 ? 4 : a.window < 4096 ? 5 : 6;
    return log < a.kv.page_shift ? log : a.kv.page_shift;
}

cudaError_t launch_attn_decode_window(const DecodeAttnArgs &args, cudaStream_t s) {
    DecodeAttnArgs a = args;
    a.box_shift = box_rows_log(a);
    return launch<kWindow>(a, a.Hq / a.kv.Hkv, s);
}

}  // namespace moe
