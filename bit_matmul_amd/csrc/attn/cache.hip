// Writing and reading the 4-bit paged cache. A lane holds eight consecutive dims of a key or
// value head: 16 bytes of activations, one word of codes. A group of dims sits on 4, 8 or 16
// neighbouring lanes, so its minimum and maximum are DPP reductions within a row of lanes,
// and the first lane of the group writes the (scale, bias) pair.
#include "attn.hpp"

namespace bitmm {
namespace attn {
namespace {

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

// Each thread's place: dims 8 l .. 8 l + 7 of head `head` of the keys (side 0) or values of
// token `token`.
template <int D>
__device__ __forceinline__ bool place(int T, int kv_heads, int& token, int& side, int& head, int& l) {
  constexpr int L = D / 8;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  l = (int)(id % L);
  const uint32_t unit = (uint32_t)(id / L);
  token = (int)(unit / (uint32_t)(2 * kv_heads));
  const int h = (int)(unit - (uint32_t)token * (uint32_t)(2 * kv_heads));
  side = h >= kv_heads;
  head = h - side * kv_heads;
  return token < T;
}

template <int D, int GS, int DT>
__global__ __launch_bounds__(256) void kv_append_kernel(AppendParams p) {
  int token, side, head, l;
  if (!place<D>(p.T, p.cache.kv_heads, token, side, head, l)) return;
  int64_t row = 0;
  if (!find_slot(p.cache, p.slots[token], p.status, row, head)) return;  // a head's lanes go together
  const uint16_t* src = (side ? p.v + (int64_t)token * p.v_stride : p.k + (int64_t)token * p.k_stride) +
                        (int64_t)head * D + 8 * l;
  const u32x4_t raw = load_u128(src);
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
  uint32_t pair = pack_bf16x2((hi - lo) / 15.f, lo);
  if (!(odd == 0.f)) pair = 0x7FC07FC0u;
  const float s = bf16_lo(pair), b = bf16_hi(pair);
  uint32_t word = 0;
  if (s > 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // A true quotient: a product with the reciprocal would put values next to a border
      // on the wrong side of it.
      const float t = fminf(fmaxf(rintf((x[i] - b) / s), 0.f), 15.f);
      word |= (uint32_t)t << (4 * i);
    }
  }
  uint32_t* codes = side ? p.cache.v_codes : p.cache.k_codes;
  uint32_t* scales = side ? p.cache.v_scales : p.cache.k_scales;
  codes[row * (D / 8) + l] = word;
  if (l % (GS / 8) == 0) scales[row * (D / GS) + l / (GS / 8)] = pair;
}

template <int D, int GS, int DT>
__global__ __launch_bounds__(256) void kv_read_kernel(ReadParams p) {
  int token, side, head, l;
  if (!place<D>(p.T, p.cache.kv_heads, token, side, head, l)) return;
  uint16_t* out = side ? p.v_out : p.k_out;
  if (!out) return;
  int64_t row = 0;
  u32x4_t y = {0, 0, 0, 0};
  if (find_slot(p.cache, p.slots[token], p.status, row, head)) {
    const uint32_t word = (side ? p.cache.v_codes : p.cache.k_codes)[row * (D / 8) + l];
    const uint32_t pair = (side ? p.cache.v_scales : p.cache.k_scales)[row * (D / GS) + l / (GS / 8)];
    const float s = bf16_lo(pair), b = bf16_hi(pair);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      y[i] = pack_half2<DT>(fmaf(s, (float)((word >> (8 * i)) & 15u), b),
                            fmaf(s, (float)((word >> (8 * i + 4)) & 15u), b));
  }
  *reinterpret_cast<u32x4_t*>(out + (int64_t)token * (side ? p.v_stride : p.k_stride) +
                              (int64_t)head * D + 8 * l) = y;
}

unsigned blocks(int T, const Cache& c) {
  return (unsigned)(((int64_t)T * 2 * c.kv_heads * (c.head_dim / 8) + 255) / 256);
}

template <int D, int GS, int DT>
hipError_t append(const AppendParams& p, hipStream_t stream) {
  const dim3 grid(blocks(p.T, p.cache));
  hipLaunchKernelGGL((kv_append_kernel<D, GS, DT>), grid, dim3(256), 0, stream, p);
  launch_log(grid, dim3(256), 0, "kv_append_kernel<%d, %d, %d>", D, GS, DT);
  return hipGetLastError();
}

template <int D, int GS, int DT>
hipError_t read(const ReadParams& p, hipStream_t stream) {
  const dim3 grid(blocks(p.T, p.cache));
  hipLaunchKernelGGL((kv_read_kernel<D, GS, DT>), grid, dim3(256), 0, stream, p);
  launch_log(grid, dim3(256), 0, "kv_read_kernel<%d, %d, %d>", D, GS, DT);
  return hipGetLastError();
}

// f(head_dim, group, dtype as constants).
template <typename F>
hipError_t with_sizes(const Cache& c, int dtype, F f) {
  auto types = [&](auto d, auto g) {
    return dtype == 0 ? f(d, g, std::integral_constant<int, 0>{}) : f(d, g, std::integral_constant<int, 1>{});
  };
  auto groups = [&](auto d) {
    if (c.group == 32) return types(d, std::integral_constant<int, 32>{});
    if (c.group == 64) return types(d, std::integral_constant<int, 64>{});
    if constexpr (decltype(d)::value >= 128) return types(d, std::integral_constant<int, 128>{});
    return hipErrorInvalidValue;
  };
  return c.head_dim == 64    ? groups(std::integral_constant<int, 64>{})
         : c.head_dim == 128 ? groups(std::integral_constant<int, 128>{})
                             : groups(std::integral_constant<int, 256>{});
}

}  // namespace

hipError_t launch_kv_append(const AppendParams& p, int dtype, hipStream_t stream) {
  return with_sizes(p.cache, dtype, [&](auto d, auto g, auto t) {
    return append<decltype(d)::value, decltype(g)::value, decltype(t)::value>(p, stream);
  });
}

hipError_t launch_kv_read(const ReadParams& p, int dtype, hipStream_t stream) {
  return with_sizes(p.cache, dtype, [&](auto d, auto g, auto t) {
    return read<decltype(d)::value, decltype(g)::value, decltype(t)::value>(p, stream);
  });
}

}  // namespace attn
}  // namespace bitmm
