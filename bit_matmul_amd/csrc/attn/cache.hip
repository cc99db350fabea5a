// Writing and reading the 4-bit paged cache. A lane holds eight consecutive dims of a key head and
// the same of the value head: 16 bytes of activations and one word of codes each. A group of dims
// sits on 4, 8 or 16 neighbouring lanes, so its minimum and maximum are DPP reductions within a row
// of lanes, and the first lane of the group writes the (scale, bias) pair.
//   bias = bf16(min), scale = bf16((max - min) / 15), code = round((x - bias) / scale) to even,
// clamped to 0 .. 15. The quotient decides which of two codes is nearer, so it is a division where
// it comes near the border of two, and the product with a reciprocal elsewhere.
//
// What bounds them: HBM, in requests as short as a slot's codes (head_dim / 2 bytes) and pairs.
// 8192 tokens of 8 heads of 128 dims, scattered over pages: append 43 MB in 17 us, 2.5 TB/s, where
// the loads also wait for the slot; read 43 MB in 12 us, 3.6 TB/s. One thread for both sides' pieces
// keeps two loads in flight and finds the slot once.
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

// Each thread's place: dims 8 l .. 8 l + 7 of head `head` of token `token`.
template <int D>
__device__ __forceinline__ bool place(int T, int kv_heads, int& token, int& head, int& l) {
  constexpr int L = D / 8;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  l = (int)(id % L);
  const uint32_t unit = (uint32_t)(id / L);
  token = (int)(unit / (uint32_t)kv_heads);
  head = (int)(unit - (uint32_t)token * (uint32_t)kv_heads);
  return token < T;
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

template <int D, int GS, int DT>
__global__ __launch_bounds__(256) void kv_append_kernel(AppendParams p) {
  int token, head, l;
  if (!place<D>(p.T, p.cache.kv_heads, token, head, l)) return;
  int64_t row = 0;
  if (!find_slot(p.cache, p.slots[token], p.status, row, head)) return;  // a head's lanes go together
  const u32x4_t k = load_u128(p.k + (int64_t)token * p.k_stride + (int64_t)head * D + 8 * l);
  const u32x4_t v = load_u128(p.v + (int64_t)token * p.v_stride + (int64_t)head * D + 8 * l);
  uint32_t k_pair, v_pair;
  const uint32_t k_word = quantise<GS, DT>(k, k_pair), v_word = quantise<GS, DT>(v, v_pair);
  p.cache.k_codes[row * (D / 8) + l] = k_word;
  p.cache.v_codes[row * (D / 8) + l] = v_word;
  if (l % (GS / 8) == 0) {
    p.cache.k_scales[row * (D / GS) + l / (GS / 8)] = k_pair;
    p.cache.v_scales[row * (D / GS) + l / (GS / 8)] = v_pair;
  }
}

template <int DT>
__device__ __forceinline__ u32x4_t expand_word(uint32_t word, uint32_t pair) {
  const float s = bf16_lo(pair), b = bf16_hi(pair);
  u32x4_t y;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    y[i] = pack_half2<DT>(fmaf(s, (float)((word >> (8 * i)) & 15u), b),
                          fmaf(s, (float)((word >> (8 * i + 4)) & 15u), b));
  return y;
}

template <int D, int GS, int DT>
__global__ __launch_bounds__(256) void kv_read_kernel(ReadParams p) {
  int token, head, l;
  if (!place<D>(p.T, p.cache.kv_heads, token, head, l)) return;
  int64_t row = 0;
  u32x4_t k = {0, 0, 0, 0}, v = k;
  if (find_slot(p.cache, p.slots[token], p.status, row, head)) {
    const int64_t word = row * (D / 8) + l, pair = row * (D / GS) + l / (GS / 8);
    uint32_t kw = 0, kp = 0, vw = 0, vp = 0;
    if (p.k_out) {
      kw = p.cache.k_codes[word];
      kp = p.cache.k_scales[pair];
    }
    if (p.v_out) {
      vw = p.cache.v_codes[word];
      vp = p.cache.v_scales[pair];
    }
    k = expand_word<DT>(kw, kp);
    v = expand_word<DT>(vw, vp);
  }
  const int64_t at = (int64_t)head * D + 8 * l;
  if (p.k_out) *reinterpret_cast<u32x4_t*>(p.k_out + (int64_t)token * p.k_stride + at) = k;
  if (p.v_out) *reinterpret_cast<u32x4_t*>(p.v_out + (int64_t)token * p.v_stride + at) = v;
}

unsigned blocks(int T, const Cache& c) {
  return (unsigned)(((int64_t)T * c.kv_heads * (c.head_dim / 8) + 255) / 256);
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
