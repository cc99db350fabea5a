// C ABI of the attention block (declared in include/bitmm_attn.h): argument validation and
// dispatch. As in api.cpp, validation is host logic alone: no pointer is followed and no HIP
// call made before it is done.
#include "bitmm_attn.h"

#include <string.h>

#include <atomic>

#include "attn.hpp"

namespace {

using bitmm::attn::AttentionParams;
using bitmm::attn::AttentionPlan;

// Whether the current device is a gfx950, asked once a device.
bitmm_status device_check() {
  static std::atomic<int> known[64];  // 0: not asked, 1: gfx950, 2: other
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) {
    (void)hipGetLastError();
    return BITMM_ERR_DEVICE;
  }
  int k = known[dev].load(std::memory_order_relaxed);
  if (k == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
      (void)hipGetLastError();
      return BITMM_ERR_DEVICE;
    }
    k = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
    known[dev].store(k, std::memory_order_relaxed);
  }
  return k == 1 ? BITMM_OK : BITMM_ERR_DEVICE;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool head_dim_ok(int64_t d) { return d == 64 || d == 128 || d == 256; }

bool dtype_ok(bitmm_dtype t) { return t == BITMM_DTYPE_BF16 || t == BITMM_DTYPE_F16; }

bool fits_int(int64_t v) { return v >= 0 && v <= INT32_MAX; }

bitmm_status check_cache(const bitmm_kv_cache* c) {
  if (!c) return BITMM_ERR_NULL;
  if (c->num_pages < 1 || c->kv_heads < 1) return BITMM_ERR_SHAPE;
  if (c->num_pages > INT32_MAX || c->kv_heads > 65535) return BITMM_ERR_SHAPE;
  const int p = c->page_size, g = c->group_size;
  if (p != 16 && p != 32 && p != 64 && p != 128 && p != 256) return BITMM_ERR_UNSUPPORTED;
  if (!head_dim_ok(c->head_dim)) return BITMM_ERR_UNSUPPORTED;
  if ((g != 32 && g != 64 && g != 128) || g > c->head_dim) return BITMM_ERR_UNSUPPORTED;
  if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales) return BITMM_ERR_NULL;
  if (!aligned(c->k_codes, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_codes, 16) ||
      !aligned(c->v_scales, 16))
    return BITMM_ERR_ALIGN;
  return BITMM_OK;
}

bitmm::attn::Cache view(const bitmm_kv_cache* c) {
  bitmm::attn::Cache v;
  v.k_codes = static_cast<uint32_t*>(c->k_codes);
  v.k_scales = static_cast<uint32_t*>(c->k_scales);
  v.v_codes = static_cast<uint32_t*>(c->v_codes);
  v.v_scales = static_cast<uint32_t*>(c->v_scales);
  v.num_pages = (int)c->num_pages;
  v.page_shift = __builtin_ctz((unsigned)c->page_size);
  v.kv_heads = c->kv_heads;
  v.head_dim = c->head_dim;
  v.group = c->group_size;
  return v;
}

// Rows of `heads` heads, `stride` values apart.
bitmm_status check_rows(const void* p, int64_t stride, int64_t heads, int64_t head_dim) {
  if (!p) return BITMM_ERR_NULL;
  if (stride < heads * head_dim) return BITMM_ERR_SHAPE;
  if (!aligned(p, 16) || stride % 8 != 0) return BITMM_ERR_ALIGN;
  return BITMM_OK;
}

bitmm_status launched(hipError_t e) { return e == hipSuccess ? BITMM_OK : BITMM_ERR_LAUNCH; }

bool attention_sizes_ok(int64_t T, int64_t B, int64_t max_q, int64_t max_kv, int64_t q_heads,
                        int64_t kv_heads, int64_t window, int64_t sinks) {
  // max_kv leaves room for the last step past it.
  return fits_int(T) && fits_int(B) && fits_int(max_q) && max_kv >= 0 && max_kv <= INT32_MAX - 1024 &&
         q_heads >= 1 && q_heads <= INT32_MAX && kv_heads >= 1 && kv_heads <= 65535 && q_heads % kv_heads == 0 &&
         fits_int(window) && fits_int(sinks) && max_q * (q_heads / kv_heads) <= INT32_MAX - 1024;
}

}  // namespace

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
