// Attention of a few query rows over a long 4-bit cache (decoding), and the join of partial
// results.
//
// A workgroup takes 16 query rows of one sequence and kv head (the query heads that share
// it, times the sequence's new tokens) and a range of the tokens, in steps of 32 that go
// round its four waves. Each wave keeps a running maximum and sum of its own (one pass over
// the cache) and the four join through LDS at the end. Scores are formed transposed, S^T =
// K Q^T, and so are outputs, O^T = V^T P^T: in the matrix cores' layouts (16x16x32, lane
// (n, g) = (lane % 16, lane / 16)) a lane then holds one query row throughout. Its
// probabilities, tokens 4 g + i of each half step, are the second product's operand as they
// stand, its maximum, sum and scale factors are plain registers, and nothing passes between
// lanes but the maximum. Codes go from HBM to registers and are expanded there:
//   keys    lane (n, g) loads dims [g D/4, (g + 1) D/4) of token n of each half step;
//   values  lane (n, g) loads dims [n D/16, (n + 1) D/16) of its eight tokens, so that
//           nibble j of the eight words is the operand of output dims n D/16 + j.
#include "attention.hpp"

#include <algorithm>

namespace bitmm {
namespace attn {
namespace {

constexpr int kRows = 16;   // query rows of a workgroup
constexpr int kStep = 32;   // tokens of a wave's step
constexpr int kWaves = 4;

template <int D, int GS>
struct StepData {
  static constexpr int KW = D / 32;                          // code words of a key piece
  static constexpr int KP = (D / 4 + GS - 1) / GS;           // groups it lies in
  static constexpr int VW = D >= 128 ? D / 128 : 1;          // words of a value piece (64: half a word)
  uint32_t k[2][KW];
  uint32_t kp[2][KP];
  uint32_t v[8][VW];
  uint32_t vp[8];
  bool ok[2];  // the half step's page is in the cache and holds live tokens
  int base;
};

template <int D, int GS>
__device__ __forceinline__ void load_step(const AttentionParams& p, const int32_t* table, int head,
                                          int kv, int base, int n, int g, StepData<D, GS>& s) {
  using S = StepData<D, GS>;
  s.base = base;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int tb = base + 16 * u;
    int page = tb < kv ? table[tb >> p.cache.page_shift] : 0;
    const bool inside = page >= 0 && page < p.cache.num_pages;
    if (!inside && p.status && threadIdx.x % 64 == 0) *p.status = 1;
    s.ok[u] = tb < kv && inside;
    page = inside ? page : 0;
    const int64_t row = (((int64_t)page * p.cache.kv_heads + head) << p.cache.page_shift) +
                        (tb & ((1 << p.cache.page_shift) - 1));
    const uint32_t* kc = p.cache.k_codes + (row + n) * (D / 8) + g * S::KW;
    if constexpr (S::KW == 2) {
      const u32x2_t w = *reinterpret_cast<const u32x2_t*>(kc);
      s.k[u][0] = w[0];
      s.k[u][1] = w[1];
    } else {
#pragma unroll
      for (int j = 0; j < S::KW; j += 4) {
        const u32x4_t w = load_u128(kc + j);
#pragma unroll
        for (int e = 0; e < 4; ++e) s.k[u][j + e] = w[e];
      }
    }
#pragma unroll
    for (int e = 0; e < S::KP; ++e)
      s.kp[u][e] = p.cache.k_scales[(row + n) * (D / GS) + g * (D / 4) / GS + e];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t vr = row + 4 * g + i;
      if constexpr (D == 64) {
        s.v[4 * u + i][0] = reinterpret_cast<const uint16_t*>(p.cache.v_codes)[vr * 16 + n];
      } else if constexpr (D == 128) {
        s.v[4 * u + i][0] = p.cache.v_codes[vr * 16 + n];
      } else {
        const u32x2_t w = *reinterpret_cast<const u32x2_t*>(p.cache.v_codes + vr * 32 + 2 * n);
        s.v[4 * u + i][0] = w[0];
        s.v[4 * u + i][1] = w[1];
      }
      s.vp[4 * u + i] = p.cache.v_scales[vr * (D / GS) + n * (D / 16) / GS];
    }
  }
}

template <int D, int GS, int DT>
__global__ __launch_bounds__(256) void attention_rows_kernel(AttentionParams p) {
  using S = StepData<D, GS>;
  constexpr int J = D / 16;  // output tiles
  __shared__ float o_lds[kWaves][J * 4][64];
  __shared__ float ml_lds[kWaves][2][16];

  int id = blockIdx.x;
  const int rt = id % p.row_tiles;
  id /= p.row_tiles;
  const int split = id % p.splits;
  id /= p.splits;
  const int head = id % p.cache.kv_heads;
  const int b = id / p.cache.kv_heads;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;

  const Extent ex = extent_of(p, b);
  const int r0 = rt * kRows;
  if (r0 >= ex.rows) return;
  const int rows = min(kRows, ex.rows - r0);
  const int lo_pos = ex.first + r0 / p.share;
  const int hi_pos = ex.first + (r0 + rows - 1) / p.share;
  const Steps<kStep> steps(lo_pos, hi_pos, p.window, p.sinks);
  const int i0 = (int)((int64_t)steps.count * split / p.splits);
  const int i1 = (int)((int64_t)steps.count * (split + 1) / p.splits);
  const int32_t* table = p.page_table + (int64_t)b * p.pages_per_seq;

  // This lane's query row, as binary16 with its largest magnitude in [1, 2): a bf16 query
  // keeps every bit that way. The order of a word's eight dims is the codes' (0 4 1 5 ...).
  const int r = min(r0 + n, ex.rows - 1);
  const int qi = r / p.share;
  const int q_head = head * p.share + r % p.share;
  const int pos = ex.first + qi;
  const uint16_t* qrow = p.q + (int64_t)(ex.q0 + qi) * p.q_stride + (int64_t)q_head * D + g * (D / 4);
  f16x8_t q[S::KW];
  float c;  // scores to base-2 logarithms, but for the keys' unit
  {
    u32x4_t raw[S::KW];
    float big = 0.f;
#pragma unroll
    for (int j = 0; j < S::KW; ++j) {
      raw[j] = load_u128(qrow + 8 * j);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x, y;
        unpack_half2<DT>(raw[j][e], x, y);
        big = fmaxf(big, fmaxf(fabsf(x), fabsf(y)));
      }
    }
    big = across32(across16(big, Max()), Max());
    const int e2 = big > 0.f && big < __uint_as_float(0x7F800000u) ? __builtin_amdgcn_frexp_expf(big) - 1 : 0;
    c = ldexpf(p.scale * kLog2e, e2);
#pragma unroll
    for (int j = 0; j < S::KW; ++j) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) unpack_half2<DT>(raw[j][e], x[2 * e], x[2 * e + 1]);
#pragma unroll
      for (int e = 0; e < 8; ++e) q[j][e] = (_Float16)ldexpf(x[(e & 1) * 4 + e / 2], -e2);
    }
  }

  f32x4_t o[J];
#pragma unroll
  for (int j = 0; j < J; ++j) o[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  float m = neg_inf(), l = 0.f;
  Unit uk = {0, 1.f, -1.f}, uv = {0, 1.f, -1.f};

  S next;
  if (i0 + wave < i1) load_step<D, GS>(p, table, head, ex.kv, steps.base(i0 + wave), n, g, next);
  for (int i = i0 + wave; i < i1; i += kWaves) {
    S s = next;
    if (i + kWaves < i1) load_step<D, GS>(p, table, head, ex.kv, steps.base(i + kWaves), n, g, next);

    // Slots that hold no live token may hold anything.
    const bool whole = s.ok[0] && s.ok[1] && s.base + kStep <= ex.kv;
    if (!whole) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (!s.ok[u] || s.base + 16 * u + n >= ex.kv)
#pragma unroll
          for (int e = 0; e < S::KP; ++e) s.kp[u][e] = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (!s.ok[u] || s.base + 16 * u + 4 * g + t >= ex.kv) s.vp[4 * u + t] = 0;
      }
    }
    uint32_t bad = 0;  // tokens of the step with a scale or bias that is not finite
    float ksize = 0.f, vsize = 0.f;
    auto sizes = [&] {
      ksize = vsize = 0.f;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < S::KP; ++e) ksize += pair_size(s.kp[u][e]);
#pragma unroll
      for (int t = 0; t < 8; ++t) vsize += pair_size(s.vp[t]);
    };
    sizes();
    if (__any(!(ksize * uk.down <= uk.limit) || !(vsize * uv.down <= uv.limit))) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        bool odd = false;
#pragma unroll
        for (int e = 0; e < S::KP; ++e)
          if (!pair_finite(s.kp[u][e])) {
            s.kp[u][e] = 0;
            odd = true;
          }
        const uint64_t who = __ballot(odd);
        bad |= (uint32_t)((who | who >> 16 | who >> 32 | who >> 48) & 0xFFFFu) << (16 * u);
      }
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const bool odd = !pair_finite(s.vp[t]);
        if (odd) s.vp[t] = 0;
        const uint64_t who = __ballot(odd);
#pragma unroll
        for (int gg = 0; gg < 4; ++gg)
          if ((who >> (16 * gg)) & 0xFFFFu) bad |= 1u << (16 * (t / 4) + 4 * gg + t % 4);
      }
      sizes();
      widen(uk, reduce_lanes<64>(ksize, Max()));
      const int before = uv.e;
      widen(uv, reduce_lanes<64>(vsize, Max()));
      if (uv.e != before) {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][e] = ldexpf(o[j][e], before - uv.e);
      }
    }

    // Scores.
    f32x4_t x[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      x[u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      f16x2_t ks[S::KP], kb[S::KP];
#pragma unroll
      for (int e = 0; e < S::KP; ++e) {
        const float sc = bf16_lo(s.kp[u][e]) * uk.down;
        ks[e] = splat_f16(sc);
        kb[e] = splat_f16(fmaf(8.f, sc, bf16_hi(s.kp[u][e]) * uk.down));
      }
#pragma unroll
      for (int j = 0; j < S::KW; ++j) {
        const int e = j * 8 / GS;
        const uint32_t w = s.k[u][j], w8 = w >> 8;
        const u32x4_t a = {as_u32(__builtin_elementwise_fma(codes_low(w), ks[e], kb[e])),
                           as_u32(__builtin_elementwise_fma(codes_high(w), ks[e], kb[e])),
                           as_u32(__builtin_elementwise_fma(codes_low(w8), ks[e], kb[e])),
                           as_u32(__builtin_elementwise_fma(codes_high(w8), ks[e], kb[e]))};
        x[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), q[j], x[u], 0, 0, 0);
      }
    }
    const float ck = ldexpf(c, uk.e);
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int t = 0; t < 4; ++t) x[u][t] *= ck;
    if (!whole || bad || !all_visible(s.base, kStep, lo_pos, hi_pos, p.window)) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int at = 16 * u + 4 * g + t;
          const bool see = s.ok[u] && s.base + at < ex.kv && visible(s.base + at, pos, p.window, p.sinks);
          if (!see)
            x[u][t] = neg_inf();
          else if (bad >> at & 1)
            x[u][t] = quiet_nan();
        }
    }

    // Running maximum, kept until a score passes it by 2^8: probabilities up to 256 are as
    // good as those up to 1.
    float top = fmaxf(fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[0][2], x[0][3])),
                      fmaxf(fmaxf(x[1][0], x[1][1]), fmaxf(x[1][2], x[1][3])));
    top = across32(across16(top, Max()), Max());
    if (__any(top > m + 8.f)) {
      const float to = fmaxf(m, top);
      const float alpha = m == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(m - to);
      if (to > neg_inf()) m = to;
      l *= alpha;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] *= alpha;
    }
    const float off = m == neg_inf() ? 0.f : m;
    f16x8_t pr;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float e = __builtin_amdgcn_exp2f(x[u][t] - off);
        l += e;
        pr[4 * u + t] = (_Float16)e;
      }

    // Outputs.
    f16x2_t vs[4], vb[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float s0 = bf16_lo(s.vp[2 * t]) * uv.down, s1 = bf16_lo(s.vp[2 * t + 1]) * uv.down;
      const float b0 = fmaf(8.f, s0, bf16_hi(s.vp[2 * t]) * uv.down);
      const float b1 = fmaf(8.f, s1, bf16_hi(s.vp[2 * t + 1]) * uv.down);
      vs[t] = f16x2_t{(_Float16)s0, (_Float16)s1};
      vb[t] = f16x2_t{(_Float16)b0, (_Float16)b1};
    }
#pragma unroll
    for (int j = 0; j < J; j += 2) {
      u32x4_t lo, hi;
      const uint32_t sel = 0x0c000c00u | (uint32_t)((j / 2) % 4) * 0x00010001u | 0x00040000u;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t w = perm_b32(s.v[2 * t + 1][j / 8], s.v[2 * t][j / 8], sel);
        lo[t] = as_u32(__builtin_elementwise_fma(codes_low(w), vs[t], vb[t]));
        hi[t] = as_u32(__builtin_elementwise_fma(codes_high(w), vs[t], vb[t]));
      }
      o[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, lo), pr, o[j], 0, 0, 0);
      o[j + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, hi), pr, o[j + 1], 0, 0, 0);
    }
  }

  // The four waves' results joined: each brings its own to the common maximum, and wave w
  // stores dims (4 g + w) D/16 .. of its lanes' rows.
  l = across32(across16(l, Add()), Add());
  if (g == 0) {
    ml_lds[wave][0][n] = m;
    ml_lds[wave][1][n] = l;
  }
  __syncthreads();
  float mt = neg_inf(), lt = 0.f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) mt = fmaxf(mt, ml_lds[w][0][n]);
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const float mw = ml_lds[w][0][n];
    // A sum that is NaN has a maximum of -infinity if it met nothing else.
    lt += ml_lds[w][1][n] * (mw == mt ? 1.f : __builtin_amdgcn_exp2f(mw - mt));
  }
  const float mine = ldexpf(m == mt ? 1.f : __builtin_amdgcn_exp2f(m - mt), uv.e);
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) o_lds[wave][4 * j + e][lane] = o[j][e] * mine;
  __syncthreads();
  if (r0 + n >= ex.rows) return;
  float y[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    y[j] = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) y[j] += o_lds[w][4 * j + wave][lane];
  }
  const int dim0 = (4 * g + wave) * J;
  const int64_t row = (int64_t)(ex.q0 + qi) * p.q_heads + q_head;
  if (p.splits > 1) {
    const int64_t at = (int64_t)split * p.T * p.q_heads + row;
    if (g == 0 && wave == 0) {
      p.part_ml[2 * at] = mt;
      p.part_ml[2 * at + 1] = lt;
    }
#pragma unroll
    for (int j = 0; j < J; j += 4)
      *reinterpret_cast<f32x4_t*>(p.part_o + at * D + dim0 + j) = f32x4_t{y[j], y[j + 1], y[j + 2], y[j + 3]};
    return;
  }
  const float inv = lt == 0.f ? 0.f : 1.f / lt;
  if (p.lse && g == 0 && wave == 0) p.lse[row] = kLn2 * (mt + __builtin_amdgcn_logf(lt));
  const int64_t at = (int64_t)(ex.q0 + qi) * p.out_stride + (int64_t)q_head * D + dim0;
  if (p.otype == kOutF32) {
#pragma unroll
    for (int j = 0; j < J; j += 4)
      *reinterpret_cast<f32x4_t*>(static_cast<float*>(p.out) + at + j) =
          f32x4_t{y[j] * inv, y[j + 1] * inv, y[j + 2] * inv, y[j + 3] * inv};
  } else {
#pragma unroll
    for (int j = 0; j < J; j += 4) {
      const u32x2_t w = p.otype == kOutBf16 ? u32x2_t{pack_half2<0>(y[j] * inv, y[j + 1] * inv),
                                                      pack_half2<0>(y[j + 2] * inv, y[j + 3] * inv)}
                                            : u32x2_t{pack_half2<1>(y[j] * inv, y[j + 1] * inv),
                                                      pack_half2<1>(y[j + 2] * inv, y[j + 3] * inv)};
      *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(p.out) + at + j) = w;
    }
  }
}

// Joins the partial results of the splits: each thread four dims of one query row, the
// splits in order.
__global__ __launch_bounds__(256) void attention_join_kernel(AttentionParams p) {
  const int D = p.cache.head_dim;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int d = (int)(id % (D / 4)) * 4;
  const int64_t unit = id / (D / 4);
  const int q_head = (int)(unit % p.q_heads);
  const int64_t rest = unit / p.q_heads;
  const int i = (int)(rest % p.max_q);
  const int64_t b = rest / p.max_q;
  if (b >= p.B) return;
  const Extent ex = extent_of(p, (int)b);
  if (i * p.share >= ex.rows) return;
  const int64_t row = (int64_t)(ex.q0 + i) * p.q_heads + q_head;
  const int64_t all = (int64_t)p.T * p.q_heads;
  float mt = neg_inf();
  for (int s = 0; s < p.splits; ++s) mt = fmaxf(mt, p.part_ml[2 * (s * all + row)]);
  float lt = 0.f;
  f32x4_t y = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < p.splits; ++s) {
    const int64_t at = s * all + row;
    const float m = p.part_ml[2 * at], l = p.part_ml[2 * at + 1];
    if (l == 0.f) continue;
    const float w = m == mt ? 1.f : __builtin_amdgcn_exp2f(m - mt);
    const f32x4_t o = *reinterpret_cast<const f32x4_t*>(p.part_o + at * D + d);
    lt += l * w;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] += o[e] * w;
  }
  const float inv = lt == 0.f ? 0.f : 1.f / lt;
  if (p.lse && d == 0) p.lse[row] = kLn2 * (mt + __builtin_amdgcn_logf(lt));
  const int64_t at = (int64_t)(ex.q0 + i) * p.out_stride + (int64_t)q_head * D + d;
  if (p.otype == kOutF32)
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(p.out) + at) =
        f32x4_t{y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv};
  else
    *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(p.out) + at) =
        p.otype == kOutBf16
            ? u32x2_t{pack_half2<0>(y[0] * inv, y[1] * inv), pack_half2<0>(y[2] * inv, y[3] * inv)}
            : u32x2_t{pack_half2<1>(y[0] * inv, y[1] * inv), pack_half2<1>(y[2] * inv, y[3] * inv)};
}

template <int D, int GS>
hipError_t launch_rows(const AttentionParams& p, int dtype, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)p.B * p.cache.kv_heads * p.row_tiles * p.splits));
  if (dtype == 0)
    hipLaunchKernelGGL((attention_rows_kernel<D, GS, 0>), grid, dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((attention_rows_kernel<D, GS, 1>), grid, dim3(256), 0, stream, p);
  launch_log(grid, dim3(256), (size_t)kWaves * (D * 64 + 128), "attention_rows_kernel<%d, %d, %d>", D, GS, dtype);
  return hipGetLastError();
}

template <int D>
hipError_t launch_groups(const AttentionParams& p, int dtype, hipStream_t stream) {
  if (p.cache.group == 32) return launch_rows<D, 32>(p, dtype, stream);
  if (p.cache.group == 64) return launch_rows<D, 64>(p, dtype, stream);
  if constexpr (D >= 128) return launch_rows<D, 128>(p, dtype, stream);
  return hipErrorInvalidValue;
}

}  // namespace

AttentionPlan plan_attention(int64_t B, int64_t max_q, int64_t max_kv, int64_t q_heads,
                             int64_t kv_heads, int64_t head_dim, int64_t window, int64_t sinks) {
  AttentionPlan plan;
  const int64_t rows = max_q * (q_heads / kv_heads);
  const int64_t span = window > 0 ? std::min(max_kv, window + sinks + max_q) : max_kv;
  if (rows > 64) {  // tiles of 32 rows a wave
    plan.waves = head_dim == 256 || B * kv_heads * ((rows + 255) / 256) < 256 ? 4 : 8;
    plan.row_tiles = (int)((rows + 32 * plan.waves - 1) / (32 * plan.waves));
    const int64_t groups = B * kv_heads * plan.row_tiles;
    const int64_t most = std::max<int64_t>(1, span / 512);
    plan.splits = (int)std::min<int64_t>(std::min((256 + groups - 1) / groups, most), 128);
    return plan;
  }
  plan.waves = 0;
  plan.row_tiles = (int)((rows + kRows - 1) / kRows);
  // Splits until there are four workgroups a CU, with at least four steps a wave.
  const int64_t groups = B * kv_heads * plan.row_tiles;
  const int64_t steps = (span + kStep - 1) / kStep;
  const int64_t most = std::max<int64_t>(1, steps / (4 * kWaves));
  const int64_t want = (4 * 256 + groups - 1) / std::max<int64_t>(1, groups);
  plan.splits = (int)std::min<int64_t>(std::min(want, most), 128);
  return plan;
}

hipError_t launch_kv_attention(AttentionParams p, const AttentionPlan& plan, int dtype,
                               hipStream_t stream) {
  p.row_tiles = plan.row_tiles;
  p.splits = plan.splits;
  hipError_t err = plan.waves > 0           ? launch_attention_tiles(p, plan.waves, dtype, stream)
                   : p.cache.head_dim == 64 ? launch_groups<64>(p, dtype, stream)
                   : p.cache.head_dim == 128 ? launch_groups<128>(p, dtype, stream)
                                             : launch_groups<256>(p, dtype, stream);
  if (err != hipSuccess || p.splits == 1) return err;
  const int64_t threads = (int64_t)p.B * p.max_q * p.q_heads * (p.cache.head_dim / 4);
  const dim3 grid((unsigned)((threads + 255) / 256));
  hipLaunchKernelGGL(attention_join_kernel, grid, dim3(256), 0, stream, p);
  launch_log(grid, dim3(256), 0, "attention_join_kernel");
  return hipGetLastError();
}

}  // namespace attn
}  // namespace bitmm
