/*
 * bitmm: decoding several continuations of one prompt (beams, samples, guesses) over the 4-bit
 * paged cache of bitmm_attn.h. Part of libbitmm; the conventions of bitmm.h and the cache,
 * the activation rows and the status word of bitmm_attn.h hold here too.
 *
 *   bitmm_qk_norm_rope_append   head norms, position rotation and the append to the cache
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
 * T * (q_heads + kv_heads) < 2^30.
 */
bitmm_status bitmm_qk_norm_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                       const void* v, int64_t v_stride, const void* q_weight,
                                       const void* k_weight, const int32_t* positions,
                                       const float* inv_freq, void* q_out, int64_t q_out_stride,
                                       const int64_t* slots, const bitmm_kv_cache* cache, int64_t T,
                                       int64_t q_heads, int64_t rot_dim, int interleaved, float eps,
                                       float weight_offset, float rope_scale, bitmm_dtype dtype,
                                       uint32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BITMM_BEAM_H */
