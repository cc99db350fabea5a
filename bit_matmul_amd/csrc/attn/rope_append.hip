// RMS norm and rotation of queries and keys, and the append of keys and values to the 4-bit paged cache,
// in one launch: rope.hip's and cache.hip's kernels without the keys' way through memory.
//
// Queries go as in rope.hip, by waves of their own. A key's wave holds eight consecutive dims a lane, as the
// cache has them in a word, and each lane also reads the eight dims that the rotation pairs them with
// (a second read of the same lines), so nothing but the reductions passes between lanes.
//
// Precision. A key next to the border of two codes takes one or the other by its last bit, a step of a
// fifteenth of its group's range; so from the sum of squares to the quotient, keys are f64, whose
// instructions run at the rate of f32's here. Nothing is rounded but the group's scale and bias (to f32 and
// bf16, as stored) and the code. Values are 16-bit numbers as they come and are quantized by cache.hip's steps.
#include "beam.hpp"
#include "cache.hpp"
#include "rope.hpp"

namespace bitmm {
namespace attn {
namespace {

__device__ __forceinline__ double two_words(uint32_t lo, uint32_t hi) {
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ uint32_t low_word(double v) { return (uint32_t)__double_as_longlong(v); }
__device__ __forceinline__ uint32_t high_word(double v) { return (uint32_t)((uint64_t)__double_as_longlong(v) >> 32); }

template <int CTRL>
__device__ __forceinline__ double dpp64(double v) {
  return two_words(__builtin_amdgcn_mov_dpp(low_word(v), CTRL, 0xF, 0xF, true),
                   __builtin_amdgcn_mov_dpp(high_word(v), CTRL, 0xF, 0xF, true));
}
// f over each aligned group of L lanes (4 to 32), the result in all of them.
template <int L, typename F>
__device__ __forceinline__ double reduce_lanes64(double v, F f) {
  static_assert(L == 4 || L == 8 || L == 16 || L == 32, "group width");
  v = f(v, dpp64<0xB1>(v));
  v = f(v, dpp64<0x4E>(v));
  if constexpr (L >= 8) v = f(v, dpp64<0x141>(v));
  if constexpr (L >= 16) v = f(v, dpp64<0x140>(v));
  if constexpr (L >= 32) {
    const auto lo = __builtin_amdgcn_permlane16_swap(low_word(v), low_word(v), false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(high_word(v), high_word(v), false, false);
    v = f(two_words(lo[0], hi[0]), two_words(lo[1], hi[1]));
  }
  return v;
}

// Codes and the pair of a lane's eight values, in a group of GS / 8 lanes.
template <int GS>
__device__ __forceinline__ uint32_t quantise64(const double (&x)[8], uint32_t& pair) {
  double lo = x[0], hi = x[0];
  float odd = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fmin(lo, x[i]);
    hi = fmax(hi, x[i]);
    odd = fabs(x[i]) < __DBL_MAX__ ? odd : 1.f;  // an infinity or NaN
  }
  lo = reduce_lanes64<GS / 8>(lo, [](double a, double b) { return fmin(a, b); });
  hi = reduce_lanes64<GS / 8>(hi, [](double a, double b) { return fmax(a, b); });
  odd = reduce_lanes<GS / 8>(odd, Max());
  // By way of f32, as frameworks convert 64-bit numbers; left to itself the compiler rounds once, and codes
  // made elsewhere from the same keys would differ where f32's rounding ends halfway between two bf16 numbers.
  pair = pack_bf16x2(opaque((float)((hi - lo) / 15.0)), opaque((float)lo));
  // Past bf16's range the pair would not be finite either.
  if (odd != 0.f || (pair & 0x7F80u) == 0x7F80u || (pair & 0x7F800000u) == 0x7F800000u) pair = 0x7FC07FC0u;
  const double s = bf16_lo(pair), b = bf16_hi(pair);
  if (!(s > 0.)) return 0;
  // A product with the reciprocal is off by less than 2^-46 of a code; where that could decide between two
  // codes, the quotient itself does.
  const double r = 1.0 / s;
  uint32_t word = 0;
  double edge = 0.;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double t = (x[i] - b) * r, c = rint(t);
    edge = fmax(edge, fabs(t - c));
    word |= (uint32_t)fmin(fmax(c, 0.), 15.) << (4 * i);
  }
  if (edge >= 0.5 - 0x1p-40) {
    word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) word |= (uint32_t)fmin(fmax(rint((x[i] - b) / s), 0.), 15.) << (4 * i);
  }
  return word;
}

template <int DT>
__device__ __forceinline__ void unpack4(u32x2_t raw, double* to) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float lo, hi;
    unpack_half2<DT>(raw[i], lo, hi);
    to[2 * i] = lo;
    to[2 * i + 1] = hi;
  }
}

// A wave's part of a token's key and value heads: HPW of them at a time.
template <int D, int GS, bool INTERLEAVED, int DT>
__device__ __forceinline__ void append_heads(const RopeAppendParams& p, int64_t token, int part, int lane) {
  constexpr int L = D / 8, HPW = kWave / L;
  const int l = lane % L, sub = lane / L;
  int64_t row0 = 0;
  if (!find_slot(p.cache, p.slots[token], p.status, row0, 0)) return;  // the wave's one token

  // Of each piece of four dims: where its partners are, and its angles. Dims that are not turned are
  // their own partners, with a sine of zero.
  const int rot = p.rope.rot_dim, half = rot / 2;
  int partner[2];
  double c[8], s[8];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int d = 8 * l + 4 * e;
    const bool turned = d < rot, lower = d < half;
    partner[e] = INTERLEAVED || !turned ? d : lower ? d + half : d - half;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[4 * e + i] = 1.;
      s[4 * e + i] = 0.;
    }
    if (!turned) continue;
    const double pos = (double)p.rope.positions[token];
#pragma unroll
    for (int i = 0; i < (INTERLEAVED ? 2 : 4); ++i) {
      const int pair = INTERLEAVED ? d / 2 + i : lower ? d + i : d - half + i;
      double t = pos * (double)p.rope.inv_freq[pair] * 0.15915494309189533577;
      t -= rint(t);
      double sine, cosine;
      sincospi(2. * t, &sine, &cosine);
      sine *= p.rope.rope_scale;
      cosine *= p.rope.rope_scale;
      if constexpr (INTERLEAVED) {
        c[4 * e + 2 * i] = c[4 * e + 2 * i + 1] = cosine;
        s[4 * e + 2 * i] = -sine;
        s[4 * e + 2 * i + 1] = sine;
      } else {
        c[4 * e + i] = cosine;
        s[4 * e + i] = lower ? -sine : sine;
      }
    }
  }
  const bool norm = p.rope.k_weight != nullptr;
  double w[8], wp[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int d = 8 * l + i, o = partner[i / 4] + i % 4;
    w[i] = norm ? (double)p.rope.weight_offset + (double)half_to_f32<DT>(p.rope.k_weight[d]) : 1.;
    wp[i] = norm ? (double)p.rope.weight_offset + (double)half_to_f32<DT>(p.rope.k_weight[o]) : 1.;
  }

  const int heads = p.cache.kv_heads;
  for (int h0 = part * HPW; h0 < heads; h0 += p.kv_waves * HPW) {
    const int h = min(h0 + sub, heads - 1);
    const uint16_t* src = p.rope.k + token * p.rope.k_stride + (int64_t)h * D;
    const u32x4_t raw = load_u128(src + 8 * l);
    const u32x4_t value = load_u128(p.v + token * p.v_stride + (int64_t)h * D + 8 * l);
    double x[8], y[8];
    unpack4<DT>(u32x2_t{raw[0], raw[1]}, x);
    unpack4<DT>(u32x2_t{raw[2], raw[3]}, x + 4);
    if constexpr (INTERLEAVED) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
    } else {
      unpack4<DT>(*reinterpret_cast<const u32x2_t*>(src + partner[0]), y);
      unpack4<DT>(*reinterpret_cast<const u32x2_t*>(src + partner[1]), y + 4);
    }
    double sq = 0.;
#pragma unroll
    for (int i = 0; i < 8; ++i) sq = fma(x[i], x[i], sq);
    sq = reduce_lanes64<L>(sq, [](double a, double b) { return a + b; });
    const double r = norm ? 1.0 / sqrt(sq * (1.0 / D) + (double)p.rope.eps) : 1.;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i] * c[i] + y[i] * r * (INTERLEAVED ? w[i ^ 1] : wp[i]) * s[i];
    uint32_t k_pair, v_pair;
    const uint32_t k_word = quantise64<GS>(x, k_pair), v_word = quantise<GS, DT>(value, v_pair);
    if (h0 + sub < heads) {
      const int64_t row = row0 + ((int64_t)h << p.cache.page_shift);
      p.cache.k_codes[row * (D / 8) + l] = k_word;
      p.cache.v_codes[row * (D / 8) + l] = v_word;
      if (l % (GS / 8) == 0) {
        p.cache.k_scales[row * (D / GS) + l / (GS / 8)] = k_pair;
        p.cache.v_scales[row * (D / GS) + l / (GS / 8)] = v_pair;
      }
    }
  }
}

template <int D, int GS, bool INTERLEAVED, int DT>
__global__ __launch_bounds__(256) void qk_norm_rope_append_kernel(RopeAppendParams p) {
  const int lane = threadIdx.x & 63;
  if (blockIdx.x < p.kv_blocks) {
    const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t token = wave / p.kv_waves;
    if (token < p.rope.T) append_heads<D, GS, INTERLEAVED, DT>(p, token, (int)(wave - token * p.kv_waves), lane);
  } else {
    const int64_t wave = (int64_t)(blockIdx.x - p.kv_blocks) * 4 + (threadIdx.x >> 6);
    const int64_t token = wave / p.rope.waves_per_token;
    if (token < p.rope.T)
      norm_rope_heads<D, INTERLEAVED, DT>(p.rope, token, (int)(wave - token * p.rope.waves_per_token), lane);
  }
}

template <int D, int GS, bool INTERLEAVED, int DT>
hipError_t launch(RopeAppendParams p, hipStream_t stream) {
  constexpr int HPW = kWave / (D / 8);
  auto waves = [&](int heads) {  // of a token: its heads spread over more waves where tokens are few
    const int64_t want = 8 * (int64_t)device_compute_units() / p.rope.T, units = (heads + HPW - 1) / HPW;
    return (int)(want < 1 ? 1 : want > units ? units : want);
  };
  auto blocks = [&](int each) { return (unsigned)(((int64_t)p.rope.T * each + 3) / 4); };
  p.kv_waves = waves(p.cache.kv_heads);
  p.kv_blocks = blocks(p.kv_waves);
  p.rope.waves_per_token = p.rope.q_heads > 0 ? waves(p.rope.q_heads) : 0;
  const dim3 grid(p.kv_blocks + blocks(p.rope.waves_per_token));
  hipLaunchKernelGGL((qk_norm_rope_append_kernel<D, GS, INTERLEAVED, DT>), grid, dim3(256), 0, stream, p);
  launch_log(grid, dim3(256), 0, "qk_norm_rope_append_kernel<%d, %d, %d, %d>", D, GS, (int)INTERLEAVED, DT);
  return hipGetLastError();
}

template <int D, int GS>
hipError_t launch_sizes(const RopeAppendParams& p, bool interleaved, int dtype, hipStream_t stream) {
  if (interleaved) return dtype == 0 ? launch<D, GS, true, 0>(p, stream) : launch<D, GS, true, 1>(p, stream);
  return dtype == 0 ? launch<D, GS, false, 0>(p, stream) : launch<D, GS, false, 1>(p, stream);
}

template <int D>
hipError_t launch_groups(const RopeAppendParams& p, bool interleaved, int dtype, hipStream_t stream) {
  if (p.cache.group == 32) return launch_sizes<D, 32>(p, interleaved, dtype, stream);
  if (p.cache.group == 64) return launch_sizes<D, 64>(p, interleaved, dtype, stream);
  if constexpr (D >= 128) return launch_sizes<D, 128>(p, interleaved, dtype, stream);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_qk_norm_rope_append(const RopeAppendParams& p, bool interleaved, int dtype, hipStream_t stream) {
  return p.cache.head_dim == 64    ? launch_groups<64>(p, interleaved, dtype, stream)
         : p.cache.head_dim == 128 ? launch_groups<128>(p, interleaved, dtype, stream)
                                   : launch_groups<256>(p, interleaved, dtype, stream);
}

}  // namespace attn
}  // namespace bitmm
