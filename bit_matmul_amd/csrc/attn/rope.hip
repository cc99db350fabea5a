// RMS norm of each query and key head with the position rotation in the same pass:
//   n = x * rsqrt(mean(x^2) + eps) * (offset + w),
//   (a, b) -> rope_scale * (a cos t - b sin t, b cos t + a sin t), t = position * inv_freq.
//
// One read and one write of q and k. A head sits on head_dim / 8 lanes, so a wave takes 8, 4
// or 2 heads at a time; each lane holds the four pairs whose angles it computed, as two
// 8-byte pieces of the head (neighbouring dims, or dims rot_dim / 2 apart), so the rotation
// moves nothing between lanes. A wave stays on one token and goes over its heads: the
// angles (an f64 product and a sine and cosine each, more arithmetic than all the rest of a
// head) are computed once a token. With few tokens their heads are spread over more waves.
//
// Angles. position * inv_freq is formed in f64 and reduced to a fraction of a turn there: at
// position 2^20 an f32 product is off by up to 2^-5 radians. The fraction goes to sincospi
// in f32.
//
// What bounds it: HBM. 8191 tokens of 16 + 2 heads of 256 dims: 151 MB in 31 to 35 us, 4.3 to 4.9 TB/s, the
// rate of a large copy (4.86); the heads of the next turn are loaded before the present ones are
// finished. 8 tokens of 40 + 8 heads: 4 us, a launch and the latency of a load and a store. 600 tokens of
// them: 7 us, where three waves a token take four turns each.
#include "attn.hpp"

namespace bitmm {
namespace attn {
namespace {

template <int D, bool INTERLEAVED, int DT>
__global__ __launch_bounds__(256) void qk_norm_rope_kernel(RopeParams p) {
  constexpr int L = D / 8;        // lanes of a head
  constexpr int HPW = kWave / L;  // heads of a wave at a time
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t token64 = wave / p.waves_per_token;
  if (token64 >= p.T) return;
  const int part = (int)(wave - token64 * p.waves_per_token);
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
  u32x2_t next_a = {0, 0}, next_b = {0, 0};
  auto load = [&](int h) {
    if (h >= heads) return;
    const uint16_t* src = h < p.q_heads ? p.q + token64 * p.q_stride + (int64_t)h * D
                                        : p.k + token64 * p.k_stride + (int64_t)(h - p.q_heads) * D;
    next_a = *reinterpret_cast<const u32x2_t*>(src + a);
    next_b = *reinterpret_cast<const u32x2_t*>(src + b);
  };
  load(part * HPW + sub);
  for (int h0 = part * HPW; h0 < heads; h0 += p.waves_per_token * HPW) {
    const int h = h0 + sub;
    const bool live = h < heads;
    const bool is_q = h < p.q_heads;
    const u32x2_t xa = next_a, xb = next_b;
    load(h + p.waves_per_token * HPW);  // the next heads while these are worked on
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
    float y[8];
    if (!turned) {  // passed on, without rope_scale
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = x[i];
    } else if constexpr (INTERLEAVED) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[2 * i] = x[2 * i] * c[i] - x[2 * i + 1] * s[i];
        y[2 * i + 1] = x[2 * i + 1] * c[i] + x[2 * i] * s[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[i] = x[i] * c[i] - x[4 + i] * s[i];
        y[4 + i] = x[4 + i] * c[i] + x[i] * s[i];
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
  }
}

template <int D, bool INTERLEAVED, int DT>
hipError_t launch(RopeParams p, hipStream_t stream) {
  constexpr int HPW = kWave / (D / 8);
  const int units = (p.q_heads + p.kv_heads + HPW - 1) / HPW;
  const int64_t want = 8 * (int64_t)device_compute_units();  // waves that fill the chip
  int64_t wpt = want / p.T;
  wpt = wpt < 1 ? 1 : (wpt > units ? units : wpt);
  p.waves_per_token = (int)wpt;
  const dim3 grid((unsigned)((p.T * wpt + 3) / 4));
  hipLaunchKernelGGL((qk_norm_rope_kernel<D, INTERLEAVED, DT>), grid, dim3(256), 0, stream, p);
  launch_log(grid, dim3(256), 0, "qk_norm_rope_kernel<%d, %d, %d>", D, (int)INTERLEAVED, DT);
  return hipGetLastError();
}

template <int D, int DT>
hipError_t launch_pairs(const RopeParams& p, bool interleaved, hipStream_t stream) {
  return interleaved ? launch<D, true, DT>(p, stream) : launch<D, false, DT>(p, stream);
}

}  // namespace

hipError_t launch_qk_norm_rope(RopeParams p, int head_dim, bool interleaved, int dtype,
                               hipStream_t stream) {
  if (dtype == 0)
    return head_dim == 64    ? launch_pairs<64, 0>(p, interleaved, stream)
           : head_dim == 128 ? launch_pairs<128, 0>(p, interleaved, stream)
                             : launch_pairs<256, 0>(p, interleaved, stream);
  return head_dim == 64    ? launch_pairs<64, 1>(p, interleaved, stream)
         : head_dim == 128 ? launch_pairs<128, 1>(p, interleaved, stream)
                           : launch_pairs<256, 1>(p, interleaved, stream);
}

}  // namespace attn
}  // namespace bitmm
