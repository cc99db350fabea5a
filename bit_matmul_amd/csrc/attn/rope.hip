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
#include "rope.hpp"

namespace bitmm {
namespace attn {
namespace {

template <int D, bool INTERLEAVED, int DT>
__global__ __launch_bounds__(256) void qk_norm_rope_kernel(RopeParams p) {
  const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t token64 = wave / p.waves_per_token;
  if (token64 >= p.T) return;
  norm_rope_heads<D, INTERLEAVED, DT>(p, token64, (int)(wave - token64 * p.waves_per_token), threadIdx.x & 63);
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
