// C ABI of the attention block (declared in include/bitmm_attn.h): argument validation and
// dispatch. As in api.cpp, validation is host logic alone: no pointer is followed and no HIP
// call made before it is done.
#include "bitmm_attn.h"

#include "attn.hpp"
#include "checks.hpp"

using namespace bitmm::attn;

extern "C" {

bitmm_status bitmm_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                const void* q_weight, const void* k_weight,
                                const int32_t* positions, const float* inv_freq, void* q_out,
                                int64_t q_out_stride, void* k_out, int64_t k_out_stride, int64_t T,
                                int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                int64_t rot_dim, int interleaved, float eps, float weight_offset,
                                float rope_scale, bitmm_dtype dtype, void* stream) {
  try {
    bitmm::launch_log_begin();
    if (!dtype_ok(dtype) || !head_dim_ok(head_dim)) return BITMM_ERR_UNSUPPORTED;
    if (!fits_int(T) || !fits_int(q_heads) || !fits_int(kv_heads)) return BITMM_ERR_SHAPE;
    if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 8 != 0) return BITMM_ERR_SHAPE;
    const int64_t heads = q_heads + kv_heads;
    if (heads > INT32_MAX || T * heads > INT32_MAX) return BITMM_ERR_SHAPE;
    if (T == 0 || heads == 0) return BITMM_OK;
    bitmm_status st;
    if (q_heads > 0) {
      if ((st = check_rows(q, q_stride, q_heads, head_dim)) != BITMM_OK) return st;
      if ((st = check_rows(q_out, q_out_stride, q_heads, head_dim)) != BITMM_OK) return st;
    }
    if (kv_heads > 0) {
      if ((st = check_rows(k, k_stride, kv_heads, head_dim)) != BITMM_OK) return st;
      if ((st = check_rows(k_out, k_out_stride, kv_heads, head_dim)) != BITMM_OK) return st;
    }
    if (rot_dim > 0 && (!positions || !inv_freq)) return BITMM_ERR_NULL;
    if (!aligned(q_weight, 2) || !aligned(k_weight, 2) || !aligned(positions, 4) || !aligned(inv_freq, 4))
      return BITMM_ERR_ALIGN;
    if ((st = device_check()) != BITMM_OK) return st;
    bitmm::attn::RopeParams p = {};
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.q_weight = static_cast<const uint16_t*>(q_weight);
    p.k_weight = static_cast<const uint16_t*>(k_weight);
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.q_out = static_cast<uint16_t*>(q_out);
    p.k_out = static_cast<uint16_t*>(k_out);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.q_out_stride = q_out_stride;
    p.k_out_stride = k_out_stride;
    p.T = (int)T;
    p.q_heads = (int)q_heads;
    p.kv_heads = (int)kv_heads;
    p.rot_dim = (int)rot_dim;
    p.eps = eps;
    p.weight_offset = weight_offset;
    p.rope_scale = rope_scale;
    return launched(bitmm::attn::launch_qk_norm_rope(p, (int)head_dim, interleaved != 0, (int)dtype,
                                                     static_cast<hipStream_t>(stream)));
  } catch (...) {
    return BITMM_ERR_LAUNCH;
  }
}

bitmm_status bitmm_kv_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                             const int64_t* slots, int64_t T, const bitmm_kv_cache* cache,
                             bitmm_dtype dtype, uint32_t* status, void* stream) {
  try {
    bitmm::launch_log_begin();
    bitmm_status st = check_cache(cache);
    if (st != BITMM_OK) return st;
    if (!dtype_ok(dtype)) return BITMM_ERR_UNSUPPORTED;
    if (!fits_int(T) || T * cache->kv_heads >= (int64_t)1 << 30) return BITMM_ERR_SHAPE;
    if (T == 0) return BITMM_OK;
    if ((st = check_rows(k, k_stride, cache->kv_heads, cache->head_dim)) != BITMM_OK) return st;
    if ((st = check_rows(v, v_stride, cache->kv_heads, cache->head_dim)) != BITMM_OK) return st;
    if (!slots) return BITMM_ERR_NULL;
    if (!aligned(slots, 8) || !aligned(status, 4)) return BITMM_ERR_ALIGN;
    if ((st = device_check()) != BITMM_OK) return st;
    bitmm::attn::AppendParams p = {};
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.slots = slots;
    p.T = (int)T;
    p.cache = view(cache);
    p.status = status;
    return launched(bitmm::attn::launch_kv_append(p, (int)dtype, static_cast<hipStream_t>(stream)));
  } catch (...) {
    return BITMM_ERR_LAUNCH;
  }
}

bitmm_status bitmm_kv_read(const bitmm_kv_cache* cache, const int64_t* slots, int64_t T,
                           void* k_out, int64_t k_out_stride, void* v_out, int64_t v_out_stride,
                           bitmm_dtype dtype, uint32_t* status, void* stream) {
  try {
    bitmm::launch_log_begin();
    bitmm_status st = check_cache(cache);
    if (st != BITMM_OK) return st;
    if (!dtype_ok(dtype)) return BITMM_ERR_UNSUPPORTED;
    if (!fits_int(T) || T * cache->kv_heads >= (int64_t)1 << 30) return BITMM_ERR_SHAPE;
    if (T == 0 || (!k_out && !v_out)) return BITMM_OK;
    if (k_out && (st = check_rows(k_out, k_out_stride, cache->kv_heads, cache->head_dim)) != BITMM_OK) return st;
    if (v_out && (st = check_rows(v_out, v_out_stride, cache->kv_heads, cache->head_dim)) != BITMM_OK) return st;
    if (!slots) return BITMM_ERR_NULL;
    if (!aligned(slots, 8) || !aligned(status, 4)) return BITMM_ERR_ALIGN;
    if ((st = device_check()) != BITMM_OK) return st;
    bitmm::attn::ReadParams p = {};
    p.cache = view(cache);
    p.slots = slots;
    p.T = (int)T;
    p.k_out = static_cast<uint16_t*>(k_out);
    p.v_out = static_cast<uint16_t*>(v_out);
    p.k_stride = k_out_stride;
    p.v_stride = v_out_stride;
    p.status = status;
    return launched(bitmm::attn::launch_kv_read(p, (int)dtype, static_cast<hipStream_t>(stream)));
  } catch (...) {
    return BITMM_ERR_LAUNCH;
  }
}

size_t bitmm_kv_attention_workspace_bytes(int64_t T, int64_t B, int64_t max_q, int64_t max_kv,
                                          int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                          int64_t window, int64_t sinks) {
  if (!attention_sizes_ok(T, B, max_q, max_kv, q_heads, kv_heads, window, sinks) || !head_dim_ok(head_dim))
    return 0;
  if (T == 0 || B == 0 || max_q == 0) return 0;
  const AttentionPlan plan =
      bitmm::attn::plan_attention(B, max_q, max_kv, q_heads, kv_heads, head_dim, window, sinks);
  if (plan.splits == 1) return 0;
  const size_t bytes = (size_t)plan.splits * (size_t)(B * kv_heads) * (size_t)plan.tail_rows * (size_t)(head_dim + 2) * 4;
  return (bytes + 255) / 256 * 256;
}

bitmm_status bitmm_kv_attention(const void* q, int64_t q_stride, const bitmm_kv_cache* cache,
                                const int32_t* page_table, int64_t pages_per_seq,
                                const int32_t* kv_lens, const int32_t* cu_q, void* out,
                                int64_t out_stride, float* lse, int64_t T, int64_t B,
                                int64_t q_heads, int64_t max_q, int64_t max_kv, float scale,
                                int64_t window, int64_t sinks, bitmm_dtype dtype,
                                bitmm_out out_type, void* workspace, size_t workspace_bytes,
                                uint32_t* status, void* stream) {
  try {
    bitmm::launch_log_begin();
    bitmm_status st = check_cache(cache);
    if (st != BITMM_OK) return st;
    if (!dtype_ok(dtype)) return BITMM_ERR_UNSUPPORTED;
    if (out_type != BITMM_OUT_BF16 && out_type != BITMM_OUT_F32 && out_type != BITMM_OUT_F16)
      return BITMM_ERR_UNSUPPORTED;
    if (!attention_sizes_ok(T, B, max_q, max_kv, q_heads, cache->kv_heads, window, sinks) || pages_per_seq < 0 ||
        pages_per_seq > INT32_MAX)
      return BITMM_ERR_SHAPE;
    if (q_heads / cache->kv_heads > 64 || B > 65535) return BITMM_ERR_UNSUPPORTED;
    if (T == 0 || B == 0 || max_q == 0) return BITMM_OK;
    if ((st = check_rows(q, q_stride, q_heads, cache->head_dim)) != BITMM_OK) return st;
    if ((st = check_rows(out, out_stride, q_heads, cache->head_dim)) != BITMM_OK) return st;
    if ((pages_per_seq > 0 && !page_table) || !kv_lens || !cu_q) return BITMM_ERR_NULL;
    if (!aligned(page_table, 4) || !aligned(kv_lens, 4) || !aligned(cu_q, 4) || !aligned(lse, 4) ||
        !aligned(status, 4) || !aligned(workspace, 16))
      return BITMM_ERR_ALIGN;
    const AttentionPlan plan = bitmm::attn::plan_attention(B, max_q, max_kv, q_heads, cache->kv_heads,
                                                           cache->head_dim, window, sinks);
    // Workgroups of a launch are counted in 31 bits.
    const int64_t groups = B * cache->kv_heads;
    if (plan.workgroups(groups) > INT32_MAX || groups * plan.tail_rows > INT32_MAX) return BITMM_ERR_UNSUPPORTED;
    const size_t need = bitmm_kv_attention_workspace_bytes(T, B, max_q, max_kv, q_heads, cache->kv_heads,
                                                           cache->head_dim, window, sinks);
    if (need > 0 && (!workspace || workspace_bytes < need)) return BITMM_ERR_WORKSPACE;
    if ((st = device_check()) != BITMM_OK) return st;
    AttentionParams p = {};
    p.q = static_cast<const uint16_t*>(q);
    p.cache = view(cache);
    p.page_table = page_table;
    p.kv_lens = kv_lens;
    p.cu_q = cu_q;
    p.out = out;
    p.lse = lse;
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = p.part_o ? p.part_o + (size_t)plan.splits * groups * plan.tail_rows * cache->head_dim : nullptr;
    p.status = status;
    p.q_stride = q_stride;
    p.out_stride = out_stride;
    p.pages_per_seq = pages_per_seq;
    p.T = (int)T;
    p.B = (int)B;
    p.q_heads = (int)q_heads;
    p.share = (int)(q_heads / cache->kv_heads);
    p.max_q = (int)max_q;
    p.max_kv = (int)max_kv;
    p.window = (int)window;
    p.sinks = (int)sinks;
    p.otype = out_type == BITMM_OUT_F32 ? bitmm::kOutF32 : (out_type == BITMM_OUT_F16 ? bitmm::kOutF16 : bitmm::kOutBf16);
    p.scale = scale;
    return launched(bitmm::attn::launch_kv_attention(p, plan, (int)dtype, static_cast<hipStream_t>(stream)));
  } catch (...) {
    return BITMM_ERR_LAUNCH;
  }
}

}  // extern "C"
