/*
 * moe_attn_serve.h -- C ABI of what a server needs around the paged cache of
 * moe_attn.h, in the same library: page tables and slots from the requests'
 * lengths, attention through a sliding window with first tokens that stay
 * visible, attention of trees of drafted tokens, and the move of the accepted
 * ones to their places.
 *
 * Conventions are those of moe_attn.h: caller-owned buffers, asynchronous
 * calls on `stream`, host-detectable errors before anything is launched,
 * device errors in the workspace's status word (moe_w4a16_get_device_status).
 * All index arrays are int32 on the device, 4-byte aligned.  With
 * MOE_ATTN_TEST_NO_COPIES=1 the attentions here fail as moe_attn_decode does.
 */
#ifndef MOE_ATTN_SERVE_H
#define MOE_ATTN_SERVE_H

#include "moe_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Workspace bytes of moe_page_plan (0 for sizes it rejects). */
size_t moe_page_plan_workspace_size(int B);

/*
 * One step's page tables, slots and positions for B sequences of which
 * sequence b has seq_lens[b] cached tokens and gets new_lens[b] more (0: none;
 * -1: it has finished and gives all its pages back).
 *
 * Free pages are a ring of `ring_size` places: state[0] is the place of the
 * first, state[1] their number.  Pages are taken from there in the order of
 * the sequences (and of each one's tokens) and entered into page_table
 * [B][table_stride]; pages given back go behind the last free one, in the same
 * order, and can be taken by the next call.  ring_size is at least the number
 * of pages that the ring and the table hold together.
 *
 * window > 0: pages all of whose tokens are behind the window of every token
 * from seq_lens[b] on, and not among the first `sinks`, are given back too:
 * page p with p >= ceil(sinks / page_size) and (p + 1) * page_size <=
 * seq_lens[b] + 1 - window.  kept[b] says up to which page (its number in the
 * sequence; 0 for a new one) earlier calls have done so, kept_out[b] the same
 * after this one.  Their entries keep their old numbers: only attention through
 * such a window may use that row from then on, not moe_attn_tree.  moe_kv_gather
 * brings what those pages hold by now, and moe_attn_prefill_window of the tokens from
 * seq_lens[b] on over what it brought takes nothing from there.  window 0: kept and
 * kept_out are not used.
 *
 * dropped (NULL: none) says how many tokens sequence b has lost since its last
 * step, rejected drafts: its table holds pages for seq_lens[b] + dropped[b].  New
 * tokens use those first; what the new length does not need goes back.  No token is
 * dropped whose page has gone back behind a window: kept[b] is at most seq_lens[b] /
 * page_size rounded down (or ceil(sinks / page_size): then no page has).
 *
 * Outputs (each input array that has an output may be that output):
 *  state_out [2];  seq_lens_out [B] (0 for a finished one);  kept_out [B];
 *  cu_q [B+1]: first row of each sequence's new tokens;
 *  cu_k [B+1]: sums of seq_lens_out (NULL: not written);
 *  positions, slots [rows]: of new token i of sequence b, in row cu_q[b] + i:
 *  its slot in the cache (moe_attn.h) and its position, seq_lens[b] + i or, with
 *  offsets [rows], seq_lens[b] + offsets[row] (a drafted token's depth in its
 *  tree).  Rows from cu_q[B] on get position 0 and slot -1, which
 *  moe_qk_rope_append does not cache.
 * All or nothing: if there are too few free pages or rows, a sequence outgrows
 * its table (or 2^30 tokens), a number is out of range, or cu_k would pass 2^31,
 * nothing is taken or given back: state, lengths and kept come out as they were,
 * cu_q and cu_k are 0, slots -1, and the status is MOE_ERR_DEVICE_BAD_INDEX
 * (detail: the first sequence that failed; B: state or a page given back twice).
 * Limits: 0 <= B <= 65535, 0 <= rows < 2^31 - 256, page_size as in moe_attn.h,
 * 1 <= ring_size < 2^30, window >= 0, sinks >= 0.
 */
moe_status_t moe_page_plan(int32_t *ring, int ring_size, const int32_t *state, int32_t *state_out,
                           int32_t *page_table, int table_stride, int page_size,
                           const int32_t *seq_lens, const int32_t *new_lens,
                           const int32_t *dropped, const int32_t *kept, const int32_t *offsets,
                           int window, int sinks, int B, int rows,
                           int32_t *seq_lens_out, int32_t *kept_out, int32_t *cu_q, int32_t *cu_k,
                           int32_t *positions, int32_t *slots, void *workspace, size_t ws_bytes,
                           moe_stream_t stream);

/*
 * moe_attn_decode through a window: the token, which is the sequence's last
 * (place n - 1, n = seq_lens[b]), sees the keys j >= n - window and j < sinks.
 * Entries of page_table whose page holds no such key are not read, whatever
 * they hold.  All else, and the workspace, as in moe_attn_decode; window >= 1,
 * sinks >= 0.
 */
moe_status_t moe_attn_decode_window(const uint16_t *q, int64_t q_stride,
                                    const moe_kv_cache_t *cache, const int32_t *page_table,
                                    int table_stride, const int32_t *seq_lens, int window, int sinks,
                                    float scale, uint16_t *out, int64_t out_stride, float *lse, int B,
                                    int Hq, void *workspace, size_t ws_bytes, moe_stream_t stream);

/*
 * moe_attn_prefill, causal and through a window: a row at place p of its
 * sequence's keys (row i of nq stands at p = i + nk - nq) sees the keys j <= p
 * with j > p - window or j < sinks.  An infinity or NaN in v may reach the up to
 * 255 rows before the first that sees it, and those up to 270 rows after the
 * last one.  All else, and the workspace, as in moe_attn_prefill; window >= 1,
 * sinks >= 0.
 */
moe_status_t moe_attn_prefill_window(const uint16_t *q, int64_t q_stride, const uint16_t *k,
                                     int64_t k_stride, const uint16_t *v, int64_t v_stride,
                                     const int32_t *cu_q, const int32_t *cu_k, int B, int Tq, int Tk,
                                     int Hq, int Hkv, int D, int window, int sinks, float scale,
                                     uint16_t *out, int64_t out_stride, float *lse, void *workspace,
                                     size_t ws_bytes, moe_stream_t stream);

/* Drafted tokens of a sequence at most. */
#define MOE_TREE_TOKENS 64

/* Workspace bytes of moe_attn_tree (0 for sizes it rejects). */
size_t moe_attn_tree_workspace_size(int B, int T, int Hq, int Hkv, int D);

/*
 * Attention of drafted tokens over the paged cache: sequence b has the rows
 * [cu_q[b], cu_q[b+1]) of q, at most 64, which are the last of its seq_lens[b]
 * cached tokens (appended before).  Its row i sees every token before the
 * drafted ones, and drafted token j where bit j of tree[row] is set (a tree: the
 * row's ancestors and itself; (2 << i) - 1: plain causal order).  A row that
 * sees nothing gets zeros and lse = -inf.  (There is no window: all of a sequence's
 * pages are read, so none may have gone back.)
 *  q [T][Hq][D], out [T][Hq][D] bf16; tree [T] uint64, 8-byte aligned;
 *  lse [T][Hq] fp32 or NULL; page_table as in moe_kv_gather.
 * Rows of out and lse that belong to no sequence are not written.  What the
 * pages hold from seq_lens[b] on is never used.  An infinity or NaN in the v of
 * a drafted token may reach all rows of its tree.
 * Results do not depend on timing.  Rounding: sums are in fp32 and the result is
 * rounded once to bf16; beside that weights may be rounded to one bf16, which moves
 * a result by at most 2^-8 sum_j p_j |v_j|, as in moe_attn_decode over fp8.  Over an
 * fp8 cache values of q below 2^-9 of their head's largest may be off by up to 2^-17
 * of it, and values of v by up to 2^-24 of the sequence's largest scale of v,
 * rounded up to a power of two, and 2^-9 of themselves (the weights then are fp16:
 * the bound above holds for both together).  Which of these a sequence's rows have may
 * depend on the other sequences and on the table's width.
 * Limits: 0 <= B <= 65535, Hq <= 1024, 0 <= T, T * Hq < 2^31, scale > 0.
 * A page number out of range, a length that is negative or beyond the table (or
 * 2^30), a cu_q that decreases or leaves [0, T], more than 64 rows, or more than
 * the sequence is long, reports MOE_ERR_DEVICE_BAD_INDEX (detail: the first such
 * sequence), and that sequence's output is undefined.
 */
moe_status_t moe_attn_tree(const uint16_t *q, int64_t q_stride, const moe_kv_cache_t *cache,
                           const int32_t *page_table, int table_stride, const int32_t *seq_lens,
                           const int32_t *cu_q, const uint64_t *tree, float scale, uint16_t *out,
                           int64_t out_stride, float *lse, int B, int T, int Hq, void *workspace,
                           size_t ws_bytes, moe_stream_t stream);

/*
 * Accepted tokens to their places: cached token base[b] + accept[b][i] of
 * sequence b becomes token base[b] + i (keys, values and scales, all heads), as
 * if all were read before the first is written.  accept [B][P] holds rising
 * numbers from 0 on, ended by -1 if there are fewer than P.
 * Workspace: MOE_ATTN_STATUS_BYTES.  Limits: 0 <= B <= 65535, 0 <= P <= 64.
 * A negative base, numbers that do not rise, a token beyond the table (or 2^30)
 * or a page number out of range reports MOE_ERR_DEVICE_BAD_INDEX (detail: the
 * first such sequence); nothing of that sequence moves.
 */
moe_status_t moe_kv_accept(const moe_kv_cache_t *cache, const int32_t *page_table, int table_stride,
                           const int32_t *base, const int32_t *accept, int B, int P, void *workspace,
                           size_t ws_bytes, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ATTN_SERVE_H */
