/*
 * bitmm: the attention block between the quantized projections, on AMD Instinct MI355X
 * (gfx950). Part of libbitmm, beside the products of bitmm.h, whose conventions hold here
 * too: caller-owned device pointers, work enqueued on `stream`, no synchronisation, no
 * allocation, arguments validated on the host before any HIP call, no exception across the
 * interface, bitwise deterministic results, and bitmm_last_launches names the kernels of
 * the thread's latest call.
 *
 *   bitmm_qk_norm_rope   RMS norm of each query and key head, with the position rotation
 *   bitmm_kv_append      quantizes keys and values to 4 bits, into the pages of a cache
 *   bitmm_kv_read        the values that given slots of the cache stand for
 *   bitmm_kv_attention   attention of queries over the 4-bit cache
 *
 * Activations are bf16 or binary16 (`dtype`). The calls are for inference: there is no
 * backward form.
 *
 * The cache. Tokens live in pages of page_size slots; slot s is place s % page_size of page
 * s / page_size. A key or value head is stored as the library stores weights: unsigned
 * 4-bit codes with a bf16 scale and bias for each group of group_size consecutive dims,
 * value = scale * code + bias. All arrays are contiguous:
 *   k_codes, v_codes    uint32 [num_pages, kv_heads, page_size, head_dim / 8]; dim d is in
 *                       bits [4 (d % 8), 4 (d % 8) + 4) of word d / 8
 *   k_scales, v_scales  bf16   [num_pages, kv_heads, page_size, head_dim / group_size, 2]:
 *                       the pair (scale, bias) of each group
 * A head of 128 dims in groups of 64 takes 72 bytes a token and side, against 256 in bf16.
 */
#ifndef BITMM_ATTN_H
#define BITMM_ATTN_H

#include "bitmm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  void* k_codes;
  void* k_scales;
  void* v_codes;
  void* v_scales;
  int64_t num_pages;  /* >= 1                                                            */
  int32_t page_size;  /* 16, 32, 64, 128 or 256                                          */
  int32_t kv_heads;   /* >= 1                                                            */
  int32_t head_dim;   /* 64, 128 or 256                                                  */
  int32_t group_size; /* 32, 64 or 128, at most head_dim                                 */
} bitmm_kv_cache;

/*
 * Every call below returns, for a cache: BITMM_ERR_NULL if the descriptor or one of its
 * pointers is NULL; BITMM_ERR_SHAPE if a count is out of range; BITMM_ERR_UNSUPPORTED for
 * other page sizes, head dims, groups or types; BITMM_ERR_ALIGN if one of its pointers is
 * not 16-byte aligned. Activation rows (q, k, v and their outputs) hold the heads of one
 * token side by side, heads * head_dim values; consecutive tokens are `*_stride` values
 * apart, so the slices of a fused projection's output are taken as they are. Strides are
 * at least heads * head_dim (BITMM_ERR_SHAPE) and multiples of 8, pointers 16-byte aligned
 * (BITMM_ERR_ALIGN).
 *
 * `status` (optional, device, uint32, 4-byte aligned) is set to 1 if the call met an
 * out-of-range index that the host could not see (a slot, a page id, a length). It is
 * never cleared by the library: the caller zeroes it when it wants to start afresh. Such
 * an index is never followed.
 */

/*
 * Head norms and position rotation, in one pass:
 *   n = x * rsqrt(mean(x^2) + eps) * (weight_offset + w)      (n = x where w is NULL)
 * over each head of q and k, then for each pair i < rot_dim / 2
 *   (a, b) -> rope_scale * (a cos t - b sin t, b cos t + a sin t),  t = positions[r] * inv_freq[i]
 * where the pair is dims (i, i + rot_dim / 2), or (2 i, 2 i + 1) when `interleaved`; dims
 * from rot_dim on are passed on as they are.
 *   q: [T, q_heads, head_dim], k: [T, kv_heads, head_dim] (k = NULL with kv_heads = 0, or
 *   q = NULL with q_heads = 0, leaves that side out); q_weight, k_weight: [head_dim] of the
 *   same type, or NULL; positions: int32 [T] (any value); inv_freq: f32 [rot_dim / 2],
 *   radians a position. Scaling for long contexts is a matter of that table and rope_scale.
 * An output may be its own input (same pointer and stride), otherwise they do not overlap.
 * The norm and the rotation are computed in f32, the angle reduced to a fraction of a turn
 * in f64, and the result is rounded once. head_dim 64, 128 or 256; rot_dim a multiple of 8
 * from 0 to head_dim. T * (q_heads + kv_heads) < 2^31.
 */
bitmm_status bitmm_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                const void* q_weight, const void* k_weight,
                                const int32_t* positions, const float* inv_freq, void* q_out,
                                int64_t q_out_stride, void* k_out, int64_t k_out_stride, int64_t T,
                                int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                int64_t rot_dim, int interleaved, float eps, float weight_offset,
                                float rope_scale, bitmm_dtype dtype, void* stream);

/*
 * Quantizes the keys and values of T tokens into the cache: k, v: [T, kv_heads, head_dim];
 * slots: int64 [T]. For each group of dims
 *   bias = bf16(min), scale = bf16((max - min) / 15), code = (x - bias) / scale rounded to
 *   nearest even and clamped to 0..15 (0 where scale is 0),
 * the difference and quotients in f32. A group that holds an infinity or NaN gets NaN for
 * both, and attention over it gives NaN. A slot of -1 skips its token (padding); any other
 * slot outside the cache skips it and sets *status. Two tokens of one call must not have
 * the same slot. T * kv_heads < 2^30.
 */
bitmm_status bitmm_kv_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                             const int64_t* slots, int64_t T, const bitmm_kv_cache* cache,
                             bitmm_dtype dtype, uint32_t* status, void* stream);

/*
 * The keys and values held at `slots`, as scale * code + bias rounded to `dtype`: k_out,
 * v_out: [T, kv_heads, head_dim] (either may be NULL). Tokens of slot -1 come back as
 * zeros, and so do those of other slots outside the cache, which also set *status.
 */
bitmm_status bitmm_kv_read(const bitmm_kv_cache* cache, const int64_t* slots, int64_t T,
                           void* k_out, int64_t k_out_stride, void* v_out, int64_t v_out_stride,
                           bitmm_dtype dtype, uint32_t* status, void* stream);

/*
 * Bytes of device workspace that bitmm_kv_attention needs (a multiple of 256; 0 if an
 * argument is out of range): partial results where few queries meet a long cache and its
 * tokens are split over several workgroups.
 */
size_t bitmm_kv_attention_workspace_bytes(int64_t T, int64_t B, int64_t max_q, int64_t max_kv,
                                          int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                          int64_t window, int64_t sinks);

/*
 * Causal attention over the 4-bit cache, for any number of new tokens of each sequence (one
 * when decoding, a prompt or a chunk of it in prefill), whose keys and values have been
 * appended before:
 *   out[i, h] = sum_j p_j v_j,  p = softmax_j(scale * q[i, h] . k_j)
 * over the tokens j of the query's sequence that it sees: j <= pos, and with window > 0
 * also j > pos - window or j < sinks (the first tokens that stay visible). Query head h
 * reads kv head h / (q_heads / kv_heads).
 *   q: [T, q_heads, head_dim]; page_table: int32 [B, pages_per_seq], token j of sequence b
 *   is place j % page_size of page page_table[b, j / page_size]; kv_lens: int32 [B], the
 *   tokens of each sequence in the cache; cu_q: int32 [B + 1], sequence b's queries are rows
 *   cu_q[b] .. cu_q[b + 1] - 1, the last of them at position kv_lens[b] - 1;
 *   out: [T, q_heads, head_dim] of type `out_type`; lse: f32 [T, q_heads] or NULL, the log
 *   of each softmax's sum.
 * A query that sees no token gives zeros and an lse of -infinity; a query that sees a token
 * whose scale or bias is not finite gives NaN, others are not touched by it, whatever stands
 * in slots they do not see. max_q and max_kv bound the sequences' queries and tokens; a
 * length or offset on the device that is negative, decreasing or passes these bounds, T or
 * the page table is cut to them and sets *status. A token on a page outside the cache is
 * seen by nobody, and sets *status if a query would see it: pages that a window has left behind
 * need no entry in the table. Rows of q that belong to no sequence are not written.
 * Scores, softmax and sums are f32; keys, values and probabilities enter the matrix cores
 * as binary16, and so do bf16 queries times `scale` in the form for many query rows (with
 * binary16 ones neither they nor keys are rounded there). Units are chosen from the stored
 * scales so that a token's key and value have 11 bits, or an error of 2^-18, of the largest
 * 15 |scale| + |bias| among its head's groups, whatever other tokens hold; probabilities have
 * 11 bits, or an error of 2^-11 of the weight of 32 tokens near them. Which form runs, how the
 * tokens are split, and with it the order of sums, follows from the arguments and all the
 * lengths of the call; the values decide whether its units need a second pass over the tokens.
 * `workspace`: caller-owned device memory of bitmm_kv_attention_workspace_bytes(...) bytes,
 * 16-byte aligned, no initialisation needed (NULL if that is 0); two calls that share it
 * must be ordered on one stream.
 * Limits (else BITMM_ERR_UNSUPPORTED): q_heads / kv_heads <= 64; B <= 65535.
 */
bitmm_status bitmm_kv_attention(const void* q, int64_t q_stride, const bitmm_kv_cache* cache,
                                const int32_t* page_table, int64_t pages_per_seq,
                                const int32_t* kv_lens, const int32_t* cu_q, void* out,
                                int64_t out_stride, float* lse, int64_t T, int64_t B,
                                int64_t q_heads, int64_t max_q, int64_t max_kv, float scale,
                                int64_t window, int64_t sinks, bitmm_dtype dtype,
                                bitmm_out out_type, void* workspace, size_t workspace_bytes,
                                uint32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BITMM_ATTN_H */
