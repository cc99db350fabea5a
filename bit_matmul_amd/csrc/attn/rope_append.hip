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
//
// What bounds it: 8191 tokens of 40 + 8 heads of 128 dims, 211 MB: 53 us, 4.0 TB/s (a copy 41). Calls take 55.8, where
// queries alone take 38.0 (rope.hip's kernel) and keys and values alone 20.4 (of it 5 for f64 arithmetic over the append's
// 16: scattered pieces of 64 and 8 bytes): the two overlap little, and mixing their workgroups made it slower. The two
// calls one after the other take 68.0. 8 tokens: 4.4 us, a launch and the latencies of slot, loads and stores; calls
// 8.7 against 13.4.
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

// The instruction's 2^-26 or so, and two steps of Newton's.
__device__ __forceinline__ double rsqrt_f64(double a) {
  const double first = __builtin_amdgcn_rsq(a), half = 0.5 * a;
  double r = first;
#pragma unroll
  for (int i = 0; i < 2; ++i) r = fma(r, fma(-half * r, r, 0.5), r);
  return fabs(r) < __DBL_MAX__ ? r : first;  // of zero and infinity
}

// Sine and cosine of t turns: the nearest quarter taken off, the series of the rest, up to an eighth of a turn, to the
// 13th and 14th power, whose next terms are 2e-14 and 1e-15.
__device__ __forceinline__ void sincos_turns(double t, double& sine, double& cosine) {
  const double quarter = rint(4. * t), y = fma(quarter, -0.25, t) * 6.28318530717958647693, z = y * y;
  double s = 1. / 6227020800., c = -1. / 87178291200.;
  s = fma(s, z, -1. / 39916800.);
  s = fma(s, z, 1. / 362880.);
  s = fma(s, z, -1. / 5040.);
  s = fma(s, z, 1. / 120.);
  s = fma(s, z, -1. / 6.);
  s = fma(s * z, y, y);
  c = fma(c, z, 1. / 479001600.);
  c = fma(c, z, -1. / 3628800.);
  c = fma(c, z, 1. / 40320.);
  c = fma(c, z, -1. / 720.);
  c = fma(c, z, 1. / 24.);
  c = fma(c, z, -0.5);
  c = fma(c, z, 1.);
  const int n = (int)fma(rint(t), -4., quarter) & 3;  // within a turn, which may be far from the first
  const double a = n & 1 ? c : s, b = n & 1 ? s : c;
  sine = n & 2 ? -a : a;
  cosine = (n + 1) & 2 ? -b : b;
}

// Codes and the pair of a lane's eight values, in a group of GS / 8 lanes.
template <int GS>
__device__ __forceinline__ uint32_t quantise64(const double (&x)[8], uint32_t& pair) {
  double lo = x[0], hi = x[0], sum = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = fmin(lo, x[i]);
    hi = fmax(hi, x[i]);
    sum += x[i];
  }
  float odd = sum == sum ? 0.f : 1.f;  // a NaN; an infinity is a largest or smallest one, or two make a NaN
  lo = reduce_lanes64<GS / 8>(lo, [](double a, double b) { return fmin(a, b); });
  hi = reduce_lanes64<GS / 8>(hi, [](double a, double b) { return fmax(a, b); });
  odd = reduce_lanes<GS / 8>(odd, Max());
  // By way of f32, as frameworks convert 64-bit numbers; left to itself the compiler rounds once, and codes
  // made elsewhere from the same keys would differ where f32's rounding ends halfway between two bf16 numbers.
  // (A product with 1/15 is the f64 quotient, or next to it, and as f32 the same but once in 2^28.)
  pair = pack_bf16x2(opaque((float)((hi - lo) * (1. / 15.))), opaque((float)lo));
  // Past bf16's range, and for infinities, the pair would not be finite either.
  if (odd != 0.f || (pair & 0x7F80u) == 0x7F80u || (pair & 0x7F800000u) == 0x7F800000u) pair = 0x7FC07FC0u;
  const double s = bf16_lo(pair), b = bf16_hi(pair);
  if (!(s > 0.)) return 0;
  // An f32 product with the reciprocal is off by less than 2^-17 of a code; where that could decide between two
  // codes, the f64 quotient does. So it does for scales below f32's normal numbers, whose reciprocal the
  // instruction does not give.
  const float r = __builtin_amdgcn_rcpf(bf16_lo(pair));
  uint32_t word = 0;
  float edge = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = (float)(x[i] - b) * r, c = rintf(t);
    edge = fmaxf(edge, fabsf(t - c));
    word |= (uint32_t)fminf(fmaxf(c, 0.f), 15.f) << (4 * i);
  }
  if (edge >= 0.4999f || bf16_lo(pair) < __FLT_MIN__) {
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

// A wave's part of a token's key and value heads: HPW of them at a time. All that the token needs is asked for
// before any of it is waited for, and the next heads before the present ones are worked on.
template <int D, int GS, bool INTERLEAVED, int DT>
__device__ __forceinline__ void append_heads(const RopeAppendParams& p, int64_t token, int part, int lane, double2* angles) {
  constexpr int L = D / 8, HPW = kWave / L;
  const int l = lane % L, sub = lane / L;
  const int heads = p.cache.kv_heads;
  // Of each piece of four dims: where the partners lie that the rotation pairs it with. Dims that are not turned
  // are their own, with a sine of zero.
  const int rot = p.rope.rot_dim, half = rot / 2;
  int partner[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int d = 8 * l + 4 * e;
    partner[e] = INTERLEAVED || d >= rot ? d : d < half ? d + half : d - half;
  }
  u32x4_t next_k, next_v;
  u32x2_t next_p[2];
  auto load = [&](int h0) {
    const int h = min(h0 + sub, heads - 1);
    const uint16_t* src = p.rope.k + token * p.rope.k_stride + (int64_t)h * D;
    next_k = load_u128(src + 8 * l);
    if constexpr (!INTERLEAVED)
#pragma unroll
      for (int e = 0; e < 2; ++e) next_p[e] = *reinterpret_cast<const u32x2_t*>(src + partner[e]);
    next_v = load_u128(p.v + token * p.v_stride + (int64_t)h * D + 8 * l);
  };
  const int64_t slot = p.slots[token];
  load(part * HPW);

  // Each angle once, by a lane of its own (by each lane for its dims: 30 us for the keys and values of 8191 tokens of
  // 8 heads of 128 dims). The wave's own part of LDS: its operations are in order.
  if (rot > 0) {
    const double pos = (double)p.rope.positions[token];
    for (int i = lane; i < half; i += 64) {
      double sine, cosine;
      sincos_turns(pos * (double)p.rope.inv_freq[i] * 0.15915494309189533577, sine, cosine);
      angles[i] = make_double2(sine * p.rope.rope_scale, cosine * p.rope.rope_scale);
    }
  }
  __builtin_amdgcn_wave_barrier();

  // own[i] and other[i]: what a dim and its partner are multiplied by, but for the norm.
  double own[8], other[8];
  {
    const bool norm = p.rope.k_weight != nullptr;
    double w[8], c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = other[i] = 1.;
    if (norm) {  // of any even address
      typedef u32x2_t Four __attribute__((aligned(2)));
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        unpack4<DT>(*reinterpret_cast<const Four*>(p.rope.k_weight + 8 * l + 4 * e), w + 4 * e);
        if constexpr (!INTERLEAVED) unpack4<DT>(*reinterpret_cast<const Four*>(p.rope.k_weight + partner[e]), other + 4 * e);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[i] += (double)p.rope.weight_offset;
        other[i] += (double)p.rope.weight_offset;
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int d = 8 * l + 4 * e;
      const bool turned = d < rot, lower = d < half;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[4 * e + i] = 1.;
        s[4 * e + i] = 0.;
      }
      if (!turned) continue;
#pragma unroll
      for (int i = 0; i < (INTERLEAVED ? 2 : 4); ++i) {
        const int pair = INTERLEAVED ? d / 2 + i : lower ? d + i : d - half + i;
        const double sine = angles[pair].x, cosine = angles[pair].y;
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
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      own[i] = w[i] * c[i];
      other[i] = (INTERLEAVED ? w[i ^ 1] : other[i]) * s[i];
    }
  }
  int64_t row0 = 0;
  if (!find_slot(p.cache, slot, p.status, row0, 0)) return;  // the wave's one token

  for (int h0 = part * HPW; h0 < heads; h0 += p.kv_waves * HPW) {
    const u32x4_t raw = next_k, value = next_v;
    double x[8], y[8];
    unpack4<DT>(u32x2_t{raw[0], raw[1]}, x);
    unpack4<DT>(u32x2_t{raw[2], raw[3]}, x + 4);
    if constexpr (INTERLEAVED) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
    } else {
      unpack4<DT>(next_p[0], y);
      unpack4<DT>(next_p[1], y + 4);
    }
    if (h0 + p.kv_waves * HPW < heads) load(h0 + p.kv_waves * HPW);
    double r = 1.;
    if (p.rope.k_weight) {
      double sq = 0.;
#pragma unroll
      for (int i = 0; i < 8; ++i) sq = fma(x[i], x[i], sq);
      sq = reduce_lanes64<L>(sq, [](double a, double b) { return a + b; });
      r = rsqrt_f64(sq * (1.0 / D) + (double)p.rope.eps);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fma(x[i], own[i], y[i] * other[i]) * r;
    uint32_t k_pair, v_pair;
    const uint32_t k_word = quantise64<GS>(x, k_pair), v_word = quantise<GS, DT>(value, v_pair);
    if (h0 + sub < heads) {
      const int64_t row = row0 + ((int64_t)(h0 + sub) << p.cache.page_shift);
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
  __shared__ double2 angles[4][D / 2];
  const int in_block = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (blockIdx.x < p.kv_blocks) {
    const unsigned wave = blockIdx.x * 4 + in_block, token = wave / (unsigned)p.kv_waves;
    if (token < (unsigned)p.rope.T)
      append_heads<D, GS, INTERLEAVED, DT>(p, token, (int)(wave - token * p.kv_waves), lane, angles[in_block]);
  } else {
    const unsigned wave = (blockIdx.x - p.kv_blocks) * 4 + in_block, token = wave / (unsigned)p.rope.waves_per_token;
    if (token < (unsigned)p.rope.T)
      // five turns ahead: keys' registers let a SIMD hold half as many waves as rope.hip's kernel (8191 tokens of
      // 40 + 8 heads of 128 dims: 62.5 us one turn ahead, 54.0 three, 52.6 five; calls 64.7, 57.5, 55.7)
      norm_rope_heads<D, INTERLEAVED, DT, 5>(p.rope, token, (int)(wave - token * p.rope.waves_per_token), lane);
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
