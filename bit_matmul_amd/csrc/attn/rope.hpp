// RMS norm and rotation of a token's heads, as described in rope.hip: a wave's part of them.
#pragma once

#include "attn.hpp"

namespace bitmm {
namespace attn {

// AHEAD: how many turns ahead its heads are loaded.
template <int D, bool INTERLEAVED, int DT, int AHEAD = 1>
__device__ __forceinline__ void norm_rope_heads(const RopeParams& p, int64_t token64, int part, int lane) {
  constexpr int L = D / 8;        // lanes of a head
  constexpr int HPW = kWave / L;  // heads of a wave at a time
  const int l = lane % L;
  const int sub = lane / L;

  // The lane's two pieces of four dims, at offsets a and b of the head; `turned` pairs them.
  const int half = p.rot_dim / 2;
  int a, b;
  bool turned;
  if constexpr (INTERLEAVED) {
    a = 8 * l;
    b = a + 4;
    turned = a < p.rot_dim;
  } else {
    turned = 4 * l < half;
    a = turned ? 4 * l : p.rot_dim + 8 * (l - half / 4);
    b = turned ? a + half : a + 4;
  }
  float c[4], s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = 1.f;
    s[i] = 0.f;
  }
  if (turned) {
    const double pos = (double)p.positions[token64];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      double t = pos * (double)p.inv_freq[4 * l + i] * 0.15915494309189533577;
      t -= rint(t);
      sincospif(2.f * (float)t, &s[i], &c[i]);
      s[i] *= p.rope_scale;
      c[i] *= p.rope_scale;
    }
  }

  float wq[8], wk[8];
  auto load_weight = [&](const uint16_t* w, float* to) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      to[i] = w ? p.weight_offset + half_to_f32<DT>(w[a + i]) : 1.f;
      to[4 + i] = w ? p.weight_offset + half_to_f32<DT>(w[b + i]) : 1.f;
    }
  };
  load_weight(p.q_weight, wq);
  load_weight(p.k_weight, wk);

  const int heads = p.q_heads + p.kv_heads;
  u32x2_t next_a[AHEAD] = {}, next_b[AHEAD] = {};
  auto load = [&](int e, int h) {
    if (h >= heads) return;
    const uint16_t* src = h < p.q_heads ? p.q + token64 * p.q_stride + (int64_t)h * D
                                        : p.k + token64 * p.k_stride + (int64_t)(h - p.q_heads) * D;
    next_a[e] = *reinterpret_cast<const u32x2_t*>(src + a);
    next_b[e] = *reinterpret_cast<const u32x2_t*>(src + b);
  };
  const int each = p.waves_per_token * HPW;
#pragma unroll
  for (int e = 0; e < AHEAD; ++e) load(e, part * HPW + sub + e * each);
  auto turn = [&](int h0, int e) {
    const int h = h0 + sub;
    const bool live = h < heads;
    const bool is_q = h < p.q_heads;
    const u32x2_t xa = next_a[e], xb = next_b[e];
    load(e, h + AHEAD * each);  // the next heads while these are worked on
    float x[8];
    unpack_half2<DT>(xa[0], x[0], x[1]);
    unpack_half2<DT>(xa[1], x[2], x[3]);
    unpack_half2<DT>(xb[0], x[4], x[5]);
    unpack_half2<DT>(xb[1], x[6], x[7]);
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sq = fmaf(x[i], x[i], sq);
    sq = reduce_lanes<L>(sq, Add());
    const bool norm = (is_q ? p.q_weight : p.k_weight) != nullptr;
    const float r = norm ? rsqrtf(sq * (1.f / D) + p.eps) : 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * (is_q ? wq[i] : wk[i]);
    // Which product is rounded is written out, so that every kernel with these turns gives the same bits.
    float y[8];
    if (!turned) {  // passed on, without rope_scale
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = x[i];
    } else if constexpr (INTERLEAVED) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[2 * i] = fmaf(x[2 * i], c[i], -(x[2 * i + 1] * s[i]));
        y[2 * i + 1] = fmaf(x[2 * i], s[i], x[2 * i + 1] * c[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[i] = fmaf(x[i], c[i], -(x[4 + i] * s[i]));
        y[4 + i] = fmaf(x[i], s[i], x[4 + i] * c[i]);
      }
    }
    if (live) {
      uint16_t* dst = is_q ? p.q_out + token64 * p.q_out_stride + (int64_t)h * D
                           : p.k_out + token64 * p.k_out_stride + (int64_t)(h - p.q_heads) * D;
      *reinterpret_cast<u32x2_t*>(dst + a) =
          u32x2_t{pack_half2<DT>(y[0], y[1]), pack_half2<DT>(y[2], y[3])};
      *reinterpret_cast<u32x2_t*>(dst + b) =
          u32x2_t{pack_half2<DT>(y[4], y[5]), pack_half2<DT>(y[6], y[7])};
    }
  };
  for (int h0 = part * HPW; h0 < heads; h0 += AHEAD * each) {
#pragma unroll
    for (int e = 0; e < AHEAD; ++e)
      if (h0 + e * each < heads) turn(h0 + e * each, e);
  }
}

}  // namespace attn
}  // namespace bitmm
