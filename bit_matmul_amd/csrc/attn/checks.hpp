// Host checks shared by the attention block's entry points.
#pragma once

#include <string.h>

#include <atomic>

#include "attn.hpp"
#include "bitmm_attn.h"

namespace bitmm {
namespace attn {

// Whether the current device is a gfx950, asked once a device.
inline bitmm_status device_check() {
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

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool head_dim_ok(int64_t d) { return d == 64 || d == 128 || d == 256; }

inline bool dtype_ok(bitmm_dtype t) { return t == BITMM_DTYPE_BF16 || t == BITMM_DTYPE_F16; }

inline bool fits_int(int64_t v) { return v >= 0 && v <= INT32_MAX; }

inline bitmm_status check_cache(const bitmm_kv_cache* c) {
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

inline Cache view(const bitmm_kv_cache* c) {
  Cache v;
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
inline bitmm_status check_rows(const void* p, int64_t stride, int64_t heads, int64_t head_dim) {
  if (!p) return BITMM_ERR_NULL;
  if (stride < heads * head_dim) return BITMM_ERR_SHAPE;
  if (!aligned(p, 16) || stride % 8 != 0) return BITMM_ERR_ALIGN;
  return BITMM_OK;
}

inline bitmm_status launched(hipError_t e) { return e == hipSuccess ? BITMM_OK : BITMM_ERR_LAUNCH; }

inline bool attention_sizes_ok(int64_t T, int64_t B, int64_t max_q, int64_t max_kv, int64_t q_heads,
                        int64_t kv_heads, int64_t window, int64_t sinks) {
  // max_kv leaves room for the last step past it.
  return fits_int(T) && fits_int(B) && fits_int(max_q) && max_kv >= 0 && max_kv <= INT32_MAX - 1024 &&
         q_heads >= 1 && q_heads <= INT32_MAX && kv_heads >= 1 && kv_heads <= 65535 && q_heads % kv_heads == 0 &&
         fits_int(window) && fits_int(sinks) && max_q * (q_heads / kv_heads) <= INT32_MAX - 1024;
}

}  // namespace attn
}  // namespace bitmm
