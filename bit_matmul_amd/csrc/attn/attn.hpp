// Internal interface of the attention block's kernels (declared to callers in
// include/bitmm_attn.h). Callers of the launch functions have validated every argument.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"
#include "kernels.hpp"

namespace bitmm {
namespace attn {

// The 4-bit cache as the kernels see it.
struct Cache {
  uint32_t* k_codes;
  uint32_t* k_scales;  // (scale, bias) pairs: scale in the low half
  uint32_t* v_codes;
  uint32_t* v_scales;
  int num_pages;
  int page_shift;  // log2 of the page size
  int kv_heads;
  int head_dim;
  int group;
};

struct RopeParams {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* q_weight;
  const uint16_t* k_weight;
  const int32_t* positions;
  const float* inv_freq;
  uint16_t* q_out;
  uint16_t* k_out;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;
  int T, q_heads, kv_heads, rot_dim;
  int waves_per_token;
  float eps, weight_offset, rope_scale;
};
hipError_t launch_qk_norm_rope(RopeParams p, int head_dim, bool interleaved, int dtype,
                               hipStream_t stream);

struct AppendParams {
  const uint16_t* k;
  const uint16_t* v;
  int64_t k_stride, v_stride;
  const int64_t* slots;
  int T;
  Cache cache;
  uint32_t* status;
};
hipError_t launch_kv_append(const AppendParams& p, int dtype, hipStream_t stream);

struct ReadParams {
  Cache cache;
  const int64_t* slots;
  int T;
  uint16_t* k_out;
  uint16_t* v_out;
  int64_t k_stride, v_stride;
  uint32_t* status;
};
hipError_t launch_kv_read(const ReadParams& p, int dtype, hipStream_t stream);

struct AttentionParams {
  const uint16_t* q;
  Cache cache;
  const int32_t* page_table;
  const int32_t* kv_lens;
  const int32_t* cu_q;
  void* out;
  float* lse;
  float* part_o;    // [splits * B, kv_heads, tail_rows, head_dim] f32, not normalised
  float* part_ml;   // [splits * B, kv_heads, tail_rows, 2]: reference exponent (base 2) and sum
  uint32_t* status;
  int64_t q_stride, out_stride, pages_per_seq;
  int T, B, q_heads, share;  // share: query heads of one kv head
  int max_q, max_kv;
  int window, sinks;
  int row_tiles, tail_tiles, tail_rows, splits;  // as in AttentionPlan
  bool balanced;
  int otype;
  float scale;
  // In a pass over what groups of sequences share, else null: the sequences of group g are cu_groups[g] ..
  // cu_groups[g + 1] of `sequences`, cu_q has the rows of each, and all else is the groups'.
  const int32_t* cu_groups;
  int sequences;
};

// How a call is cut up, from sizes alone, so that the workspace query and the call agree: the
// rows of each sequence and kv head into row tiles, a workgroup each, and the tokens that the first
// tail_tiles of them see over `splits` workgroups each. (All of them where there are few; where
// there are many, those that would otherwise run alone at the end.)
struct AttentionPlan {
  bool tiles;      // the kernel for many query rows
  int waves;       // of a workgroup, in the kernel for few rows
  int rows_each;   // rows of a tile
  int row_tiles;
  int tail_tiles;  // 0 where nothing is split
  int tail_rows;   // rows that they hold
  int splits;
  bool balanced;   // splits are an average: longer sequences get more, shorter ones fewer
  int64_t workgroups(int64_t groups) const { return groups * (row_tiles + (int64_t)tail_tiles * (splits - 1)); }
};
AttentionPlan plan_attention(int64_t B, int64_t max_q, int64_t max_kv, int64_t q_heads,
                             int64_t kv_heads, int64_t head_dim, int64_t window, int64_t sinks);
hipError_t launch_kv_attention(AttentionParams p, const AttentionPlan& plan, int dtype,
                               hipStream_t stream);

// Attention of groups of sequences that share their first tokens: a pass over what they share and a pass over
// what each has of its own, whose partial results are joined.
struct SharedParams {
  AttentionParams own, prefix;  // in this order: a kernel's parameters begin with those of its pass
};
struct SharedPlan {
  AttentionPlan own, prefix;
  bool both;  // in one launch, a workgroup for all tokens that a row tile sees
};
// A kernel's part in it: none, the pass over the shared tokens, whose results are all partial, that over the own
// ones, whose results take in the former's, or both in one, each sequence by itself.
enum Pass { kAlone = 0, kPrefix = 1, kOwn = 2, kBoth = 3 };
template <int PASS>
struct PassParams {
  typedef AttentionParams Type;
};
template <>
struct PassParams<kOwn> {
  typedef SharedParams Type;
};
template <>
struct PassParams<kBoth> {
  typedef SharedParams Type;
};
__device__ __forceinline__ const AttentionParams& params_of(const AttentionParams& p) { return p; }
__device__ __forceinline__ const AttentionParams& params_of(const SharedParams& p) { return p.own; }
SharedPlan plan_attention_shared(int64_t groups, int64_t B, int64_t max_group_q, int64_t max_prefix, int64_t max_q,
                                 int64_t max_kv, int64_t q_heads, int64_t kv_heads, int64_t head_dim);
hipError_t launch_kv_attention_shared(SharedParams p, const SharedPlan& plan, int dtype, hipStream_t stream);

// Its passes for many query rows (prefill_shared.hip).
hipError_t launch_attention_tiles_prefix(const AttentionParams& p, int rows_each, unsigned workgroups, int dtype,
                                         hipStream_t stream);
hipError_t launch_attention_tiles_own(const SharedParams& p, int rows_each, unsigned workgroups, int dtype,
                                      hipStream_t stream);

// The kernel for many query rows (prefill.hip).
hipError_t launch_attention_tiles(const AttentionParams& p, int rows_each, unsigned workgroups, int dtype,
                                  hipStream_t stream);

// ---- device helpers -------------------------------------------------------------------

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

// 16-bit activation to f32 and back (rounded to nearest even). DT 0: bf16, 1: binary16.
template <int DT>
__device__ __forceinline__ float half_to_f32(uint32_t bits) {
  if constexpr (DT == 0)
    return __uint_as_float(bits << 16);
  else
    return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}
template <int DT>
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  if constexpr (DT == 0) {
    return pack_bf16x2(lo, hi);
  } else {
    f16x2_t v;
    v[0] = (_Float16)lo;
    v[1] = (_Float16)hi;
    return __builtin_bit_cast(uint32_t, v);
  }
}
// The two 16-bit values of a word as f32.
template <int DT>
__device__ __forceinline__ void unpack_half2(uint32_t w, float& lo, float& hi) {
  if constexpr (DT == 0) {
    lo = bf16_lo(w);
    hi = bf16_hi(w);
  } else {
    const f16x2_t v = __builtin_bit_cast(f16x2_t, w);
    lo = (float)v[0];
    hi = (float)v[1];
  }
}

// Value of lane ^ 16 combined with the own one, and the same for lane ^ 32: a swap of two
// copies of v leaves the one half's values in the first result and the other's in the
// second, in every lane.
template <typename F>
__device__ __forceinline__ float across16(float v, F f) {
  const uint32_t u = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return f(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
template <typename F>
__device__ __forceinline__ float across32(float v, F f) {
  const uint32_t u = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return f(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(v), CTRL, 0xF, 0xF, true));
}

// f over each aligned group of L lanes (4 to 64), the result in all of them.
template <int L, typename F>
__device__ __forceinline__ float reduce_lanes(float v, F f) {
  static_assert(L == 4 || L == 8 || L == 16 || L == 32 || L == 64, "group width");
  v = f(v, dpp<0xB1>(v));                           // lane ^ 1
  v = f(v, dpp<0x4E>(v));                           // lane ^ 2
  if constexpr (L >= 8) v = f(v, dpp<0x141>(v));    // mirrored within 8
  if constexpr (L >= 16) v = f(v, dpp<0x140>(v));   // mirrored within 16
  if constexpr (L >= 32) v = across16(v, f);
  if constexpr (L >= 64) v = across32(v, f);
  return v;
}

struct Add {
  __device__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
  __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct Min {
  __device__ float operator()(float a, float b) const { return fminf(a, b); }
};

struct AddInt {  // of integers
  __device__ float operator()(float a, float b) const {
    return __uint_as_float(__float_as_uint(a) + __float_as_uint(b));
  }
};
struct Or {  // of bit patterns
  __device__ float operator()(float a, float b) const {
    return __uint_as_float(__float_as_uint(a) | __float_as_uint(b));
  }
};

// A lane's value that the compiler knows nothing of: what a rare branch computes from it is not
// moved ahead of a loop, where it would hold registers throughout.
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

__device__ __forceinline__ float opaque(float v) {
  asm volatile("" : "+v"(v));
  return v;
}

}  // namespace attn
}  // namespace bitmm
