// Slots of the 4-bit paged cache, and the codes of eight values, as described in cache.hip.
#pragma once

#include "attn.hpp"

namespace bitmm {
namespace attn {

// Word offset of dims [8 l, 8 l + 8) of (slot, head), and of group g's pair. False when the
// slot is outside the cache; -1 is padding, anything else is reported.
__device__ __forceinline__ bool find_slot(const Cache& c, int64_t slot, uint32_t* status,
                                          int64_t& row_base, int head) {
  const int64_t page = slot >> c.page_shift;
  if (slot < 0 || page >= c.num_pages) {
    if (slot != -1 && status) *status = 1;
    return false;
  }
  const int64_t off = slot & (((int64_t)1 << c.page_shift) - 1);
  row_base = ((page * c.kv_heads + head) << c.page_shift) + off;
  return true;
}

// Codes and the pair of a lane's eight values, in a group of GS / 8 lanes.
template <int GS, int DT>
__device__ __forceinline__ uint32_t quantise(u32x4_t raw, uint32_t& pair) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack_half2<DT>(raw[i], x[2 * i], x[2 * i + 1]);
  float lo = x[0], hi = x[0], odd = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
    odd += x[i] * 0.f;  // NaN for an infinity or NaN, else 0
  }
  lo = reduce_lanes<GS / 8>(lo, Min());
  hi = reduce_lanes<GS / 8>(hi, Max());
  odd = reduce_lanes<GS / 8>(odd, Add());
  pair = pack_bf16x2((hi - lo) / 15.f, lo);
  if (!(odd == 0.f)) pair = 0x7FC07FC0u;
  const float s = bf16_lo(pair), b = bf16_hi(pair);
  if (!(s > 0.f)) return 0;
  // A product with the reciprocal is off by less than 2^-17 of a code; where that could decide
  // between two codes, the quotient itself does. So it does for scales below f32's normal numbers,
  // whose reciprocal the instruction does not give.
  const float r = __builtin_amdgcn_rcpf(s);
  uint32_t word = 0;
  float edge = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = (x[i] - b) * r, c = rintf(t);
    edge = fmaxf(edge, fabsf(t - c));
    word |= (uint32_t)fminf(fmaxf(c, 0.f), 15.f) << (4 * i);
  }
  if (edge >= 0.4999f || s < __FLT_MIN__) {
    word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) word |= (uint32_t)fminf(fmaxf(rintf((x[i] - b) / s), 0.f), 15.f) << (4 * i);
  }
  return word;
}

}  // namespace attn
}  // namespace bitmm
