/*
 * bitmm: decoding several continuations of one prompt (beams, samples, guesses) over the 4-bit
 * paged cache of bitmm_attn.h. Part of libbitmm; the conventions of bitmm.h and the cache,
 * the activation rows and the status word of bitmm_attn.h hold here too.
 *
 *   bitmm_qk_norm_rope_append   head norms, position rotation and the append to the cache
 *   bitmm_kv_attention_shared   attention of sequences that share their first tokens, in groups
 *   bitmm_beam_select           the best continuations of a group of beams
 *   bitmm_kv_beam_reorder       the cached states in the order of the beams that go on
 *
 * The calls are for inference: there is no backward form.
 */
#ifndef BITMM_BEAM_H
#define BITMM_BEAM_H

#include "bitmm_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * bitmm_qk_norm_rope on q and k and bitmm_kv_append of k and v in one launch:
 *   q [T, q_heads, head_dim] -> q_out, as bitmm_qk_norm_rope has it (q = NULL with q_heads = 0
 *   leaves that side out; q_out may be q);
 *   k [T, kv_heads, head_dim], normed and rotated, and v as it is -> the cache's slots [T].
 * head_dim and kv_heads are the cache's. Keys are quantized as they come out of the rotation, in
 * f64, with no rounding to 16 bits on the way: their codes are nearer than those of the two
 * calls one after the other, and may differ from them where a key lies next to the border of
 * two codes. Values get the codes that bitmm_kv_append gives them. A token with slot -1 is
 * not stored, nor is one whose slot lies outside the cache, which sets *status; their q_out is
 * written all the same. Slots of one call are distinct (of two tokens with one slot, which
 * one's pieces stay is not defined). A key or value that is not finite makes its group NaN.
 * T <= 2^24 and T * (q_heads + kv_heads) < 2^30.
 */
bitmm_status bitmm_qk_norm_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                       const void* v, int64_t v_stride, const void* q_weight,
                                       const void* k_weight, const int32_t* positions,
                                       const float* inv_freq, void* q_out, int64_t q_out_stride,
                                       const int64_t* slots, const bitmm_kv_cache* cache, int64_t T,
                                       int64_t q_heads, int64_t rot_dim, int interleaved, float eps,
                                       float weight_offset, float rope_scale, bitmm_dtype dtype,
                                       uint32_t* status, void* stream);

/*
 * Attention of sequences that share their first tokens with the others of their group: a prompt's
 * beams or samples, or requests behind one system prompt. What they share is stored and read once.
 *   cu_groups    int32 [groups + 1]: the sequences of group g are cu_groups[g] .. cu_groups[g + 1] - 1
 *   prefix_table int32 [groups, pages_per_prefix], prefix_lens int32 [groups]: the shared tokens' pages and
 *                their number
 *   page_table   int32 [B, pages_per_seq], kv_lens int32 [B]: each sequence's own tokens, the queries' among
 *                them, on pages of their own (a prefix may end within a page)
 *   cu_q         int32 [B + 1]: the rows of each sequence's queries
 * q, out, lse, scale, types and status are bitmm_kv_attention's. A query sees all shared tokens of its group
 * and its sequence's own ones up to its own position, which is that of bitmm_kv_attention over the own
 * tokens alone. A sequence of no group has its own tokens alone. The result is that of bitmm_kv_attention
 * over shared and own tokens in a row, with another order of sums; there is no window (the shared part of one
 * is short: use bitmm_kv_attention). Where prefixes end with a page, bitmm_kv_attention over tables that name the shared
 * pages gives that too, and is the faster of the two where sequences and tokens are few.
 * max_group_q bounds the queries of a group, max_prefix the shared tokens, max_q and max_kv the queries
 * and own tokens of a sequence; what passes them is cut and sets *status, and rows past them are not written.
 * `workspace`: bitmm_kv_attention_shared_workspace_bytes(...) bytes, 16-byte aligned, no initialisation
 * needed; two calls that share it must be ordered on one stream.
 * Limits (else BITMM_ERR_UNSUPPORTED): q_heads / kv_heads <= 64; B and groups <= 65535; launches of
 * less than 2^23 workgroups.
 */
size_t bitmm_kv_attention_shared_workspace_bytes(int64_t T, int64_t B, int64_t groups, int64_t max_group_q,
                                                 int64_t max_prefix, int64_t max_q, int64_t max_kv,
                                                 int64_t q_heads, int64_t kv_heads, int64_t head_dim);
bitmm_status bitmm_kv_attention_shared(const void* q, int64_t q_stride, const bitmm_kv_cache* cache,
                                       const int32_t* prefix_table, int64_t pages_per_prefix,
                                       const int32_t* prefix_lens, const int32_t* cu_groups,
                                       const int32_t* page_table, int64_t pages_per_seq,
                                       const int32_t* kv_lens, const int32_t* cu_q, void* out,
                                       int64_t out_stride, float* lse, int64_t T, int64_t B, int64_t groups,
                                       int64_t q_heads, int64_t max_group_q, int64_t max_prefix,
                                       int64_t max_q, int64_t max_kv, float scale, bitmm_dtype dtype,
                                       bitmm_out out_type, void* workspace, size_t workspace_bytes,
                                       uint32_t* status, void* stream);

/*
 * Beam search's selection. Row r = g * beams + b holds the logits of beam b of group g (a prompt),
 * rows `row_stride` values apart, of which the first `vocab` count. A candidate is a token t after a
 * beam b, and stands for
 *   total = scores[g, b] + (logits[r, t] - log sum_u exp(logits[r, u]))
 * Of each group the k candidates of the largest total come out, in order: scores_out, parents (the
 * beam, 0 .. beams - 1) and tokens, all [groups, k]. Equal totals go to the lowest (beam, token); of
 * one beam the order is that of its logits. Sums, totals and comparisons are f64 (sums exact to 2^-32 or so of
 * themselves, whatever the logits' size), scores_out is rounded once.
 * A beam whose finished[r] (uint8 [groups, beams], or NULL for none) is not 0 has one candidate: end_token with
 * its score as it is; its logits are not read. finished_out (uint8 [groups, k], or NULL) is 1
 * where the parent was finished or the token is end_token (-1: no such token).
 * No candidates are: logits of -infinity, beams whose score is -infinity, and beams with a NaN or
 * +infinity among score or logits, which set *status. Where fewer than k are left the last places
 * hold -infinity, parent -1 and token -1.
 * With k = beams the outputs may be the inputs of the same kind; otherwise they do not overlap.
 * beams and k 1 to 64, vocab up to 2^30, groups * beams up to 2^22 (else BITMM_ERR_SHAPE); logits aligned
 * to their type. `workspace`: at least bitmm_beam_select_workspace_bytes(...) bytes, 16-byte aligned,
 * no initialisation needed; two calls that share it must be ordered on one stream.
 */
size_t bitmm_beam_select_workspace_bytes(int64_t groups, int64_t beams, int64_t vocab, int64_t k,
                                         bitmm_out logits_type);
bitmm_status bitmm_beam_select(const void* logits, int64_t row_stride, const float* scores,
                               const uint8_t* finished, float* scores_out, int32_t* parents,
                               int32_t* tokens, uint8_t* finished_out, int64_t groups, int64_t beams,
                               int64_t vocab, int64_t k, int32_t end_token, bitmm_out logits_type,
                               void* workspace, size_t workspace_bytes, uint32_t* status, void* stream);

/*
 * The cached states in the order of the beams that go on, with room for one more token each.
 * Row r = g * beams + j, beam j of group g, has lens[r] tokens on the pages that page_table
 * [groups * beams, pages_per_seq] names. After the call it has those of beam parents[r] of its
 * group (0 .. beams - 1; -1: none, an empty row) and one more, which is to be stored at slots[r]
 * (as bitmm_kv_append takes it) and which lens_out counts. Pages that are full are shared: rows of
 * the table name the same ones. A last page that is partly filled is kept by one row, if it
 * is of the group's pool and no longer row has it full in the same place: that with the most tokens on it, the first of
 * those with as many. The others get a page each, to which the tokens are copied, in all `layers` caches (one for each
 * layer of a model, of the same sizes; their pages share one table). A row whose last page is full, or that is empty,
 * gets a page for the next token.
 * New pages are the lowest ones of the group's pool that no row of the group holds afterwards, in the
 * order of the rows: pages [first_page + g * pages_per_group, + pages_per_group). A pool of beams *
 * pages_per_seq pages never ends. Pages outside it, as those of a prompt, may be named and are never written;
 * they lie in no other group's pool.
 * A row for which no page or no place in the table is left keeps its parent's tokens and gets no room:
 * its slot is -1, lens_out is its parent's, and *status is set, as it is by parents and lengths out of range
 * (taken as -1, and cut) and by a partly filled page outside the cache, whose tokens are lost: the row that would keep
 * it gets no room, any other a page of its own, of which the slots before its next token hold what lay there before.
 * Empty rows have slot -1 and a length of 0.
 * Entries of the table past a row's pages are passed on as they are. An output may be its input (same
 * pointer), otherwise they do not overlap.
 * beams 1 to 64, groups * beams up to 2^22, layers up to 4096, pages_per_seq up to 2^22, pages_per_group up to 2^18
 * (else BITMM_ERR_SHAPE). `workspace`: bitmm_kv_beam_reorder_workspace_bytes(...) bytes, 16-byte aligned, no
 * initialisation needed; two calls that share it must be ordered on one stream.
 */
size_t bitmm_kv_beam_reorder_workspace_bytes(int64_t groups, int64_t beams);
bitmm_status bitmm_kv_beam_reorder(const bitmm_kv_cache* caches, int64_t layers, const int32_t* page_table,
                                   int32_t* page_table_out, int64_t pages_per_seq, const int32_t* lens,
                                   int32_t* lens_out, const int32_t* parents, int64_t* slots,
                                   int64_t groups, int64_t beams, int64_t first_page,
                                   int64_t pages_per_group, void* workspace, size_t workspace_bytes,
                                   uint32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BITMM_BEAM_H */
