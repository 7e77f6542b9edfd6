/*
 * moe_attn.h -- C ABI of the attention half of a decoder layer on GB300
 * (sm_103a), in the same library as the MoE half (moe_w4a16.h): per-head
 * norms of queries and keys with the position rotation and the cache write
 * in one pass, the read-back of cached tokens, attention of single tokens
 * over the paged cache, attention over packed prompts.
 *
 * Conventions are those of moe_w4a16.h: the caller owns every buffer, calls
 * are asynchronous on `stream`, host-detectable errors return before
 * anything is launched, errors found on the device never trap and are
 * recorded in the workspace's status word, which each call sets anew and
 * moe_w4a16_get_device_status() reads back.  A workspace must not be used by
 * two calls that overlap on the GPU; it need not be initialised.
 *
 * Activations are bf16.  Strides are in elements, between the rows of one
 * token and the next; the heads of a token are D elements apart, so the
 * three parts of one fused projection can be passed without copying.  All
 * strides are multiples of 8 and all activation pointers 16-byte aligned.
 * D is 64 or 128; Hq % Hkv == 0, query head h reads key/value head
 * h / (Hq / Hkv).
 */
#ifndef MOE_ATTN_H
#define MOE_ATTN_H

#include "moe_w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How a cache holds keys and values. */
typedef enum {
    MOE_KV_BF16 = 0, /* bf16 */
    MOE_KV_FP8 = 1   /* fp8 e4m3 codes, one fp32 scale per token, head and K / V */
} moe_kv_type_t;

/*
 * A paged key/value cache (caller-owned device memory).
 *  data   [num_pages][Hkv][2][page_size][D] bf16 or e4m3: K rows, then V rows
 *         of one head of one page, contiguous (one copy brings both on chip);
 *         16-byte aligned.
 *  scales [num_pages][Hkv][2][page_size] fp32 (MOE_KV_FP8; 16-byte aligned),
 *         NULL for MOE_KV_BF16.  A value is code * scale.
 * page_size is 16, 32, 64, 128 or 256 and num_pages * page_size < 2^31;
 * num_pages * Hkv * 2 * page_size < 2^31.
 * A slot number is page * page_size + position in the page.
 */
typedef struct {
    void *data;
    float *scales;
    int32_t type; /* moe_kv_type_t */
    int32_t num_pages, page_size, Hkv, D;
} moe_kv_cache_t;

/* Bytes of a cache's two arrays (*scale_bytes = 0 for bf16). */
moe_status_t moe_kv_cache_size(int type, int num_pages, int page_size, int Hkv, int D,
                               size_t *data_bytes, size_t *scale_bytes);

/* Workspace of moe_qk_rope_append and moe_kv_gather (256-byte aligned). */
#define MOE_ATTN_STATUS_BYTES 256u

/*
 * Norm, rotation and cache write of T new tokens.  For every head of q and k
 * (a row x of D values), all in fp32:
 *   x <- x * rsqrt(mean(x^2) + eps) * w      (w = q_norm or k_norm [D] bf16;
 *                                             NULL: left out)
 *   pairs i < rot/2, with c = cos_sin[p][i], s = cos_sin[p][rot/2 + i] of the
 *   token's position p = positions[t]:  (a, b) <- (a c - b s, b c + a s),
 *   where (a, b) = (x[i], x[i + rot/2]), or (x[2i], x[2i+1]) if interleaved;
 *   values from rot on are not rotated.
 * q goes to q_out and k to k_out (NULL: not written), rounded to bf16; each
 * may be its own input with the same stride.  k and v (as given) go to slot
 * slots[t] of the cache (-1: this token is not cached; cache NULL: none is):
 * rounded to bf16, or, MOE_KV_FP8, as scale = amax / 448 with amax the row's
 * largest magnitude, and code = e4m3(x * (448 / amax)), nearest-even (amax
 * 0: scale and codes 0; an amax below 2^-119 counts as 2^-119; a row holding
 * an infinity or a NaN: scale NaN).  (A cache that others filled may hold NaN
 * codes with any scale: such a value is NaN to all that read it.)
 * Two tokens must not name the same slot.
 *  cos_sin [max_pos][rot] fp32, 16-byte aligned (NULL if rot == 0): scaling
 *          for long contexts is a matter of the table's angles.
 * Limits: 0 <= rot <= D, rot % 16 == 0, 0 <= T, T * (Hq + 2 Hkv) < 2^31.
 * A position outside [0, max_pos) or a slot outside [-1, num_pages *
 * page_size) leaves that token out (nothing of it is written) and reports
 * MOE_ERR_DEVICE_BAD_INDEX (detail: the first such token).
 */
moe_status_t moe_qk_rope_append(const uint16_t *q, int64_t q_stride, const uint16_t *k,
                                int64_t k_stride, const uint16_t *v, int64_t v_stride,
                                const uint16_t *q_norm, const uint16_t *k_norm, float eps,
                                const float *cos_sin, int max_pos, int rot, int interleaved,
                                const int32_t *positions, const int32_t *slots, uint16_t *q_out,
                                int64_t q_out_stride, uint16_t *k_out, int64_t k_out_stride,
                                const moe_kv_cache_t *cache, int T, int Hq, int Hkv, int D,
                                void *workspace, size_t ws_bytes, moe_stream_t stream);

/*
 * Read-back of cached tokens as packed bf16 rows, for a prompt attention over
 * an earlier context: row cu_k[b] + i of k_out / v_out [Tk][Hkv][D] = token i
 * of sequence b, the value code * scale rounded once.
 *  page_table [B][table_stride] int32: page of token i is entry i / page_size.
 *  cu_k [B+1] int32: first row of each sequence; cu_k[0] = 0, cu_k[B] = Tk.
 * A page number outside [0, num_pages), a decreasing cu_k, one that does not
 * start at 0 and end at Tk, or a sequence longer than its table reports
 * MOE_ERR_DEVICE_BAD_INDEX (detail: the first such sequence, B for the
 * ends of cu_k); rows that have no page are written as zeros.
 */
moe_status_t moe_kv_gather(const moe_kv_cache_t *cache, const int32_t *page_table,
                           int table_stride, const int32_t *cu_k, int B, int Tk, uint16_t *k_out,
                           int64_t k_out_stride, uint16_t *v_out, int64_t v_out_stride,
                           void *workspace, size_t ws_bytes, moe_stream_t stream);

/* Workspace bytes of moe_attn_decode (0 for sizes it rejects). */
size_t moe_attn_decode_workspace_size(int B, int Hq, int Hkv, int D);

/*
 * Attention of one new token of each of B sequences over its cached tokens
 * (its own among them, appended before): for head h of sequence b
 *   s_j = scale * q . k_j,  out = sum_j exp(s_j) v_j / sum_j exp(s_j),
 *   lse = ln sum_j exp(s_j),   j < seq_lens[b];
 * seq_lens[b] = 0 gives zeros and lse = -inf.  What the pages hold from
 * seq_lens[b] on is never used, whatever it is.
 *  q [B][Hq][D], out [B][Hq][D] bf16; lse [B][Hq] fp32 or NULL.
 *  page_table, table_stride: as in moe_kv_gather.
 * Results do not depend on timing: keys are split over the GPU by the
 * lengths alone and the parts are joined in a fixed order.
 * Rounding: sums are in fp32 and the result is rounded once to bf16.  Over a
 * bf16 cache the weights exp(s - max) enter the product with v as sums of two
 * bf16 (2^-16).  Over an fp8 cache each weight times its v's scale is rounded
 * to one bf16, which moves a result by at most 2^-8 sum_j p_j |v_j| (p the
 * normalised weights; with one key, all values of a head by one factor), and
 * values of q below 2^-14 of their head's largest are off by up to 2^-25 of it.
 * Limits: 0 <= B <= 65535, Hq <= 1024, scale > 0.
 * A page number out of range, a negative length or one beyond the table (or
 * 2^30) reports MOE_ERR_DEVICE_BAD_INDEX (detail: the first such sequence),
 * and that sequence's output is undefined.
 * For testing the failure path only, MOE_ATTN_TEST_NO_COPIES=1 (read once per
 * process) makes this call and moe_attn_prefill issue no copies: their
 * bounded waits give up after about a second, the call reports
 * MOE_ERR_DEVICE_TIMEOUT (detail: the role) and its output is undefined.
 */
moe_status_t moe_attn_decode(const uint16_t *q, int64_t q_stride, const moe_kv_cache_t *cache,
                             const int32_t *page_table, int table_stride, const int32_t *seq_lens,
                             float scale, uint16_t *out, int64_t out_stride, float *lse, int B,
                             int Hq, void *workspace, size_t ws_bytes, moe_stream_t stream);

/* Workspace bytes of moe_attn_prefill (0 for sizes it rejects). */
size_t moe_attn_prefill_workspace_size(int B, int Tq, int Hq, int Hkv, int D);

/*
 * Attention over packed sequences: sequence b has the query rows
 * [cu_q[b], cu_q[b+1]) of q and the key/value rows [cu_k[b], cu_k[b+1]) of k
 * and v; its last query row stands at its last key.  Row i of nq sees the
 * keys j <= i + nk - nq of nk (causal != 0) or all of them; a row that sees
 * none gets zeros and lse = -inf.
 *  q [Tq][Hq][D], k and v [Tk][Hkv][D], out [Tq][Hq][D] bf16;
 *  lse [Tq][Hq] fp32 or NULL.
 * Rows of out and lse that belong to no sequence are not written.
 * Other sequences' rows never matter, whatever they hold.  Within a
 * sequence an infinity or NaN in v may also reach up to 255 rows before the
 * first that sees it (its weight there is 0, the product NaN).
 * Weights exp(s - max) are rounded to bf16 for the product with v (sums are
 * in fp32).
 * Limits: 0 <= B <= 65535, Hq <= 1024, Tq * Hq < 2^31, scale > 0.
 * A cu_q or cu_k that decreases or leaves [0, Tq] / [0, Tk] reports
 * MOE_ERR_DEVICE_BAD_INDEX (detail: the first such sequence); that
 * sequence's rows are not written.
 */
moe_status_t moe_attn_prefill(const uint16_t *q, int64_t q_stride, const uint16_t *k,
                              int64_t k_stride, const uint16_t *v, int64_t v_stride,
                              const int32_t *cu_q, const int32_t *cu_k, int B, int Tq, int Tk,
                              int Hq, int Hkv, int D, int causal, float scale, uint16_t *out,
                              int64_t out_stride, float *lse, void *workspace, size_t ws_bytes,
                              moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ATTN_H */
