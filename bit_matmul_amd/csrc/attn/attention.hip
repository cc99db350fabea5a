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

#include <stdlib.h>

#include <algorithm>

namespace bitmm {
namespace attn {
namespace {

constexpr int kRows = 16;   // query rows of a workgroup
constexpr int kStep = 32;   // tokens of a wave's step

// Where a step's two halves of 16 tokens lie: rows of the cache, the same in every lane.
struct StepPlace {
  int64_t row[2];
  bool ok[2];  // the half step's page is in the cache and holds live tokens
};

// Pages of the two halves of a step (0 where no token is live).
struct StepPages {
  int page[2];
};
__device__ __forceinline__ StepPages step_pages(const AttentionParams& p, const int32_t* table, int kv,
                                                int base) {
  StepPages s;
#pragma unroll
  for (int u = 0; u < 2; ++u) s.page[u] = base + 16 * u < kv ? table[(base + 16 * u) >> p.cache.page_shift] : 0;
  return s;
}
__device__ __forceinline__ StepPlace step_place(const AttentionParams& p, int head, int kv, int base,
                                                const StepPages& pages) {
  StepPlace s;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int tb = base + 16 * u;
    const int page = __builtin_amdgcn_readfirstlane(pages.page[u]);
    const bool inside = page >= 0 && page < p.cache.num_pages;
    if (!inside && p.status && (threadIdx.x & 63) == 0) *p.status = 1;
    s.ok[u] = tb < kv && inside;
    s.row[u] = (((int64_t)(inside ? page : 0) * p.cache.kv_heads + head) << p.cache.page_shift) +
               (tb & ((1 << p.cache.page_shift) - 1));
  }
  return s;
}

// Loads go through descriptors whose bases are those rows: scalar registers hold what moves from
// step to step, a lane's offset stays what it is, and no 64-bit address is formed in a lane.
// They span the 16 rows, which lie within one page.

// Pairs of a side of a step: those of a half are 16 NG neighbouring words, and pair 64 e + lane
// of the step is token (64 e + lane) / NG, group (64 e + lane) % NG.
template <int NG, int PL>
__device__ __forceinline__ void load_pairs(const uint32_t* scales, const StepPlace& s, int lane, uint32_t (&to)[PL]) {
  constexpr int BYTES = 64 * NG;  // of a half step's pairs
  const __amdgpu_buffer_rsrc_t half[2] = {make_rsrc(scales + s.row[0] * NG, BYTES), make_rsrc(scales + s.row[1] * NG, BYTES)};
#pragma unroll
  for (int e = 0; e < PL; ++e) {
    if constexpr (NG >= 4) {
      to[e] = __builtin_amdgcn_raw_buffer_load_b32(half[e / (NG / 4)], 4 * lane, 256 * (e % (NG / 4)), 0);
    } else {
      // Both halves in one wave: each lane's offset is inside one of the two and past the other,
      // where a load gives zero.
      const uint32_t at = 4 * lane;
      to[e] = __builtin_amdgcn_raw_buffer_load_b32(half[0], at, 0, 0) |
              __builtin_amdgcn_raw_buffer_load_b32(half[1], at - BYTES, 0, 0);
    }
  }
}

template <int D, int GS, int KW>
__device__ __forceinline__ void load_keys(const Cache& c, const StepPlace& s, int lane, uint32_t (&k)[2][KW]) {
  const uint32_t at = (uint32_t)((lane & 15) * (D / 2) + (lane >> 4) * (GS / 8));
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const __amdgpu_buffer_rsrc_t from = make_rsrc(c.k_codes + s.row[u] * (D / 8), 8 * D);
#pragma unroll
    for (int y = 0; y < D / GS; ++y) {
      if constexpr (GS == 32) {
        k[u][y] = __builtin_amdgcn_raw_buffer_load_b32(from, at + y * (GS / 2), 0, 0);
      } else if constexpr (GS == 64) {
        const u32x2_t w = __builtin_amdgcn_raw_buffer_load_b64(from, at + y * (GS / 2), 0, 0);
        k[u][2 * y] = w[0];
        k[u][2 * y + 1] = w[1];
      } else {
        const u32x4_t w = __builtin_amdgcn_raw_buffer_load_b128(from, at + y * (GS / 2), 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) k[u][4 * y + e] = w[e];
      }
    }
  }
}
template <int D, int VW>
__device__ __forceinline__ void load_values(const Cache& c, const StepPlace& s, int lane, uint32_t (&v)[8][VW]) {
  const uint32_t at = (uint32_t)(4 * (lane >> 4) * (D / 2) + (lane & 15) * (D / 32));
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const __amdgpu_buffer_rsrc_t from = make_rsrc(c.v_codes + s.row[u] * (D / 8), 8 * D);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (D == 64) {
        v[4 * u + i][0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(from, at + i * (D / 2), 0, 0);
      } else if constexpr (D == 128) {
        v[4 * u + i][0] = __builtin_amdgcn_raw_buffer_load_b32(from, at + i * (D / 2), 0, 0);
      } else {
        const u32x2_t w = __builtin_amdgcn_raw_buffer_load_b64(from, at + i * (D / 2), 0, 0);
        v[4 * u + i][0] = w[0];
        v[4 * u + i][1] = w[1];
      }
    }
  }
}

// A pair as binary16 in units of 2^e: (scale, bias + 8 scale), for codes less eight.
__device__ __forceinline__ uint32_t pair_f16(uint32_t pair, float down) {
  const float s = bf16_lo(pair) * down;
  return pack_half2<1>(s, fmaf(8.f, s, bf16_hi(pair) * down));
}

template <int D, int GS, int DT, int WAVES>
__global__ __launch_bounds__(64 * WAVES, D == 256 ? 2 : 4) void attention_rows_kernel(AttentionParams p) {
  constexpr int NG = D / GS;                         // groups of a head
  constexpr int J = D / 16;                          // output tiles
  constexpr int KW = D / 32, WG = GS / 32;           // a lane's key words, and those of a group
  constexpr int VW = D >= 128 ? D / 128 : 1;         // words of a value piece (64: half a word)
  constexpr int PL = NG > 2 ? NG / 2 : 1;            // pairs of a lane
  // Pairs of each wave's step, [group][token], of the keys and of the values; the joined outputs
  // afterwards.
  constexpr int PAIR_BYTES = WAVES * 2 * 32 * NG * 4, JOIN_BYTES = WAVES * J * 4 * 64 * 4;
  __shared__ __attribute__((aligned(16))) char lds[PAIR_BYTES > JOIN_BYTES ? PAIR_BYTES : JOIN_BYTES];
  __shared__ float ml_lds[WAVES][2][16];
  float(*o_lds)[J * 4][64] = reinterpret_cast<float(*)[J * 4][64]>(lds);

  int id = blockIdx.x;
  const int rt = id % p.row_tiles;
  id /= p.row_tiles;
  const int split = id % p.splits;
  id /= p.splits;
  const int head = id % p.cache.kv_heads;
  const int b = id / p.cache.kv_heads;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  uint32_t* k_pairs = reinterpret_cast<uint32_t*>(lds) + wave * 64 * NG;
  uint32_t* v_pairs = k_pairs + 32 * NG;

  const Extent ex = extent_of(p, b);
  const int r0 = rt * kRows;
  if (r0 >= ex.rows) return;
  const int rows = min(kRows, ex.rows - r0);
  const int lo_pos = ex.first + r0 / p.share;
  const int hi_pos = ex.first + (r0 + rows - 1) / p.share;
  const Steps<kStep> steps(lo_pos, hi_pos, p.window, p.sinks);
  const Part part = part_of(steps.count, split, p.splits);
  const int i0 = part.first, i1 = part.last;
  const int32_t* table = p.page_table + (int64_t)b * p.pages_per_seq;

  uint32_t k[2][KW], v[8][VW], kp[PL], vp[PL];
  StepPages pages = {};
  StepPlace place = {};
  const int first = i0 + wave;
  if (first < i1) {
    pages = step_pages(p, table, ex.kv, steps.base(first));
    place = step_place(p, head, ex.kv, steps.base(first), pages);
    if (first + WAVES < i1) pages = step_pages(p, table, ex.kv, steps.base(first + WAVES));
    load_keys<D, GS>(p.cache, place, lane, k);
    load_pairs<NG, PL>(p.cache.k_scales, place, lane, kp);
    load_values<D>(p.cache, place, lane, v);
    load_pairs<NG, PL>(p.cache.v_scales, place, lane, vp);
  }

  // This lane's query row as binary16, its largest magnitude in [2^7, 2^8): a bf16 query keeps
  // every bit that way. A word's codes come out in the order 0 4 1 5 2 6 3 7, the odd ones
  // times 16, which the query takes back.
  const RowOf row_of(p, head, min(r0 + n, ex.rows - 1));
  const int pos = ex.first + row_of.i;
  const uint16_t* qrow = p.q + (int64_t)(ex.q0 + row_of.i) * p.q_stride + (int64_t)row_of.head * D + g * (GS / 4);
  f16x8_t q[KW];
  float c;            // scores to base-2 logarithms, but for the keys' unit
  float q_sum[NG];    // sum of the query over each group
  float centre[NG];   // takes the codes' offsets (1024 + 8, and (1024 + 128) / 16) off a group's sum
  {
    u32x4_t raw[KW];
    float big = 0.f;
#pragma unroll
    for (int j = 0; j < KW; ++j) {
      raw[j] = load_u128(qrow + j / WG * GS + 8 * (j % WG));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x, y;
        unpack_half2<DT>(raw[j][e], x, y);
        big = fmaxf(big, fmaxf(fabsf(x), fabsf(y)));
      }
    }
    big = across32(across16(big, Max()), Max());
    const int e2 = big > 0.f && big < __uint_as_float(0x7F800000u) ? __builtin_amdgcn_frexp_expf(big) - 8 : 0;
    c = ldexpf(p.scale * kLog2e, e2);
#pragma unroll
    for (int y = 0; y < NG; ++y) {
      float even = 0.f, odd = 0.f;
#pragma unroll
      for (int j = y * WG; j < (y + 1) * WG; ++j) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) unpack_half2<DT>(raw[j][e], x[2 * e], x[2 * e + 1]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool high = e & 2;
          q[j][e] = (_Float16)ldexpf(x[(e & 1) * 4 + e / 2], high ? -e2 - 4 : -e2);
          (high ? odd : even) += (float)q[j][e];
        }
      }
      even = across32(across16(even, Add()), Add());
      odd = across32(across16(odd, Add()), Add());
      q_sum[y] = even + 16.f * odd;
      centre[y] = -fmaf(1032.f, even, 1152.f * odd);
    }
  }

  f32x4_t o[J];
#pragma unroll
  for (int j = 0; j < J; ++j) o[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  float m = neg_inf(), l = 0.f;
  Unit uk = {0, 1.f, -1.f}, uv = {0, 1.f, -1.f};
  // 1024 twice in binary16, in a register, so that mask and OR are one instruction. (No inline
  // assembly next to the matrix cores: the compiler keeps the distance that their operands and
  // results need only for instructions that it knows.)
  uint32_t k1024 = 0x64006400u;
  asm("" : "+v"(k1024));

  for (int i = first; i < i1; i += WAVES) {
    const int base = steps.base(i);
    const bool ok0 = place.ok[0], ok1 = place.ok[1], more = i + WAVES < i1;
    if (more) {
      place = step_place(p, head, ex.kv, steps.base(i + WAVES), pages);
      if (i + 2 * WAVES < i1) pages = step_pages(p, table, ex.kv, steps.base(i + 2 * WAVES));
    }

    // Slots that hold no live token may hold anything.
    const bool whole = ok0 && ok1 && base + kStep <= ex.kv;
    uint32_t bad = 0;  // tokens of the step with a scale or bias that is not finite
    if (!whole) {
      const int at = opaque(lane);
#pragma unroll
      for (int e = 0; e < PL; ++e) {
        const int token = (64 * e + at) / NG;
        const bool ok = (token < 16 ? ok0 : ok1) && base + token < ex.kv && token < 32;
        kp[e] = ok ? kp[e] : 0;
        vp[e] = ok ? vp[e] : 0;
      }
    }
    float ksize = 0.f, vsize = 0.f;
    auto sizes = [&] {
      ksize = vsize = 0.f;
#pragma unroll
      for (int e = 0; e < PL; ++e) {
        ksize += pair_size(kp[e]);
        vsize += pair_size(vp[e]);
      }
    };
    sizes();
    if (__any(!(ksize * uk.down <= uk.limit) || !(vsize * uv.down <= uv.limit))) {
      const int at = opaque(lane);
#pragma unroll
      for (int e = 0; e < PL; ++e) {
        const bool odd_k = !pair_finite(kp[e]), odd_v = !pair_finite(vp[e]);
        if (odd_k) kp[e] = 0;
        if (odd_v) vp[e] = 0;
        if (odd_k || odd_v) bad |= 1u << ((64 * e + at) / NG % 32);
      }
      bad = __float_as_uint(reduce_lanes<64>(__uint_as_float(bad), Or()));
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
    // The wave's own part of LDS: its operations are in order.
#pragma unroll
    for (int e = 0; e < PL; ++e) {
      const int f = 64 * e + lane;
      if (NG >= 2 || lane < 32) {
        k_pairs[f % NG * 32 + f / NG] = pair_f16(kp[e], uk.down);
        v_pairs[f % NG * 32 + f / NG] = pair_f16(vp[e], uv.down);
      }
    }
    __builtin_amdgcn_wave_barrier();

    // Scores: the products with the bare codes less eight, group by group, times the scales.
    f32x4_t x[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      x[u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int y = 0; y < NG; ++y) {
        float at = centre[y];
        asm volatile("" : "+v"(at));  // made four of here, not kept as four
        f32x4_t sum = {at, at, at, at};
#pragma unroll
        for (int j = y * WG; j < (y + 1) * WG; ++j) {
          const uint32_t w = k[u][j], w8 = w >> 8;
          const u32x4_t a = {(w & 0x000F000Fu) | k1024, (w & 0x00F000F0u) | k1024, (w8 & 0x000F000Fu) | k1024,
                             (w8 & 0x00F000F0u) | k1024};
          sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), q[j], sum, 0, 0, 0);
        }
        const u32x4_t pairs = *reinterpret_cast<const u32x4_t*>(k_pairs + 32 * y + 16 * u + 4 * g);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const f16x2_t sb = as_f16x2(pairs[t]);
          x[u][t] = fmaf(sum[t], (float)sb[0], fmaf(q_sum[y], (float)sb[1], x[u][t]));
        }
        // Done here: moved past the loads below, the sums and pairs of all groups would stay.
        asm volatile("" : "+v"(x[u]));
      }
    }
    if (more) {
      load_keys<D, GS>(p.cache, place, lane, k);
      load_pairs<NG, PL>(p.cache.k_scales, place, lane, kp);
    }
    const float ck = ldexpf(c, uk.e);
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int t = 0; t < 4; ++t) x[u][t] *= ck;
    if (!whole || bad || !all_visible(base, kStep, lo_pos, hi_pos, p.window)) {
      const int g4 = 4 * opaque(g);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int at = 16 * u + g4 + t;
          const bool see = (u ? ok1 : ok0) & (base + at < ex.kv) & visible(base + at, pos, p.window, p.sinks);
          const float y = bad >> at & 1 ? quiet_nan() : x[u][t];
          x[u][t] = see ? y : neg_inf();
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
    u32x4_t pr;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int t = 0; t < 4; t += 2) {
        const float e0 = __builtin_amdgcn_exp2f(x[u][t] - off), e1 = __builtin_amdgcn_exp2f(x[u][t + 1] - off);
        l += e0 + e1;
        pr[2 * u + t / 2] = pack_half2<1>(e0, e1);
      }
    const f16x8_t prob = __builtin_bit_cast(f16x8_t, pr);

    // Outputs.
    f16x2_t vs[4], vb[4];
    const uint32_t* v_read = v_pairs + n * (D / 16) / GS * 32 + 4 * g;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const u32x4_t w = *reinterpret_cast<const u32x4_t*>(v_read + 16 * u);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        vs[2 * u + t] = as_f16x2(perm_b32(w[2 * t + 1], w[2 * t], 0x05040100u));
        vb[2 * u + t] = as_f16x2(perm_b32(w[2 * t + 1], w[2 * t], 0x07060302u));
      }
    }
#pragma unroll
    for (int j = 0; j < J; j += 2) {
      u32x4_t lo, hi;
      const uint32_t sel = 0x0c000c00u | (uint32_t)((j / 2) % 4) * 0x00010001u | 0x00040000u;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t w = perm_b32(v[2 * t + 1][j / 8], v[2 * t][j / 8], sel);
        lo[t] = as_u32(__builtin_elementwise_fma(codes_low(w), vs[t], vb[t]));
        hi[t] = as_u32(__builtin_elementwise_fma(codes_high(w), vs[t], vb[t]));
      }
      o[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, lo), prob, o[j], 0, 0, 0);
      o[j + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, hi), prob, o[j + 1], 0, 0, 0);
    }
    if (more) {
      load_values<D>(p.cache, place, lane, v);
      load_pairs<NG, PL>(p.cache.v_scales, place, lane, vp);
    }
    __builtin_amdgcn_wave_barrier();
  }

  // The waves' results joined: each brings its own to the common maximum, and wave w stores
  // every WAVES / 4-th part of dims (4 g + w % 4) D/16 .. of its lanes' rows.
  l = across32(across16(l, Add()), Add());
  if (g == 0) {
    ml_lds[wave][0][n] = m;
    ml_lds[wave][1][n] = l;
  }
  __syncthreads();
  float mt = neg_inf(), lt = 0.f;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) mt = fmaxf(mt, ml_lds[w][0][n]);
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
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
  constexpr int PARTS = WAVES / 4 < J / 4 ? WAVES / 4 : J / 4;  // of a lane's J dims, four or more each
  constexpr int JP = J / PARTS;
  if (wave >= 4 * PARTS) return;
  const int i4 = wave & 3, j0 = (wave >> 2) * JP;
  float y[JP];
#pragma unroll
  for (int j = 0; j < JP; ++j) {
    y[j] = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) y[j] += o_lds[w][4 * (j0 + j) + i4][lane];
  }
  const int dim0 = (4 * g + i4) * J + j0;
  const bool speaker = g == 0 && wave == 0;
  const RowOf out_row(p, head, opaque(r0 + n));
  const int64_t row = (int64_t)(ex.q0 + out_row.i) * p.q_heads + out_row.head;
  if (p.splits > 1) {
    const int64_t at = (int64_t)split * p.T * p.q_heads + row;
    if (speaker) {
      p.part_ml[2 * at] = mt;
      p.part_ml[2 * at + 1] = lt;
    }
#pragma unroll
    for (int j = 0; j < JP; j += 4)
      *reinterpret_cast<f32x4_t*>(p.part_o + at * D + dim0 + j) = f32x4_t{y[j], y[j + 1], y[j + 2], y[j + 3]};
    return;
  }
  const float inv = lt == 0.f ? 0.f : 1.f / lt;
  if (p.lse && speaker) p.lse[row] = kLn2 * (mt + __builtin_amdgcn_logf(lt));
  const int64_t at = (int64_t)(ex.q0 + out_row.i) * p.out_stride + (int64_t)out_row.head * D + dim0;
#pragma unroll
  for (int j = 0; j < JP; j += 4) store4(p, at + j, y[j] * inv, y[j + 1] * inv, y[j + 2] * inv, y[j + 3] * inv);
}

// Joins the partial results of the splits. A workgroup takes one query row: 256 / (D / 4)
// groups of threads go round its splits, four dims a thread, and are added up in LDS.
template <int D>
__global__ __launch_bounds__(256) void attention_join_kernel(AttentionParams p) {
  constexpr int TPR = D / 4, GROUPS = 256 / TPR;
  __shared__ f32x4_t sums[GROUPS][TPR];
  __shared__ float part_l[GROUPS];
  const int64_t unit = blockIdx.x;
  const int q_head = (int)(unit % p.q_heads);
  const int64_t rest = unit / p.q_heads;
  const int i = (int)(rest % p.max_q);
  const Extent ex = extent_of(p, (int)(rest / p.max_q));
  if (i * p.share >= ex.rows) return;
  const int64_t row = (int64_t)(ex.q0 + i) * p.q_heads + q_head;
  const int64_t all = (int64_t)p.T * p.q_heads;
  const int lane = threadIdx.x & 63;
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  // At most 128 splits: two a lane.
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  float2 a = make_float2(neg_inf(), 0.f), b = a;
  if (lane < p.splits) a = ml[lane * all + row];
  if (lane + 64 < p.splits) b = ml[(lane + 64) * all + row];
  const float mt = reduce_lanes<64>(fmaxf(a.x, b.x), Max());
  f32x4_t y = {0.f, 0.f, 0.f, 0.f};
  float lt = 0.f;
#pragma unroll 4
  for (int s = grp; s < p.splits; s += GROUPS) {
    const int64_t at = s * all + row;
    const float2 part = ml[at];
    const f32x4_t o = *reinterpret_cast<const f32x4_t*>(p.part_o + at * D + 4 * t);
    if (part.y == 0.f) continue;  // saw nothing: the outputs were not written
    const float w = part.x == mt ? 1.f : __builtin_amdgcn_exp2f(part.x - mt);
    lt += part.y * w;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] += o[e] * w;
  }
  sums[grp][t] = y;
  if (t == 0) part_l[grp] = lt;
  __syncthreads();
  if (grp != 0) return;
  lt = 0.f;
  y = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < GROUPS; ++w) {
    lt += part_l[w];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] += sums[w][t][e];
  }
  const float inv = lt == 0.f ? 0.f : 1.f / lt;
  if (p.lse && t == 0) p.lse[row] = kLn2 * (mt + __builtin_amdgcn_logf(lt));
  store4(p, (int64_t)(ex.q0 + i) * p.out_stride + (int64_t)q_head * D + 4 * t, y[0] * inv, y[1] * inv, y[2] * inv,
         y[3] * inv);
}

template <int D, int GS, int WAVES>
hipError_t launch_rows(const AttentionParams& p, int dtype, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)p.B * p.cache.kv_heads * p.row_tiles * p.splits)), block(64 * WAVES);
  if (dtype == 0)
    hipLaunchKernelGGL((attention_rows_kernel<D, GS, 0, WAVES>), grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL((attention_rows_kernel<D, GS, 1, WAVES>), grid, block, 0, stream, p);
  launch_log(grid, block, (size_t)WAVES * (D * 64 + 128), "attention_rows_kernel<%d, %d, %d, %d>", D, GS, dtype, WAVES);
  return hipGetLastError();
}

template <int D, int GS>
hipError_t launch_waves(const AttentionParams& p, int waves, int dtype, hipStream_t stream) {
  return waves == 4 ? launch_rows<D, GS, 4>(p, dtype, stream) : launch_rows<D, GS, 8>(p, dtype, stream);
}

template <int D>
hipError_t launch_groups(const AttentionParams& p, int waves, int dtype, hipStream_t stream) {
  if (p.cache.group == 32) return launch_waves<D, 32>(p, waves, dtype, stream);
  if (p.cache.group == 64) return launch_waves<D, 64>(p, waves, dtype, stream);
  if constexpr (D >= 128) return launch_waves<D, 128>(p, waves, dtype, stream);
  return hipErrorInvalidValue;
}

}  // namespace

AttentionPlan plan_attention(int64_t B, int64_t max_q, int64_t max_kv, int64_t q_heads,
                             int64_t kv_heads, int64_t head_dim, int64_t window, int64_t sinks) {
  AttentionPlan plan;
  const int64_t rows = max_q * (q_heads / kv_heads);
  const int64_t span = window > 0 ? std::min(max_kv, window + sinks + max_q) : max_kv;
  plan.tiles = rows > 64;
  if (plan.tiles) {  // tiles of 32 rows a wave
    plan.waves = head_dim == 256 || B * kv_heads * ((rows + 255) / 256) < 256 ? 4 : 8;
    plan.row_tiles = (int)((rows + 32 * plan.waves - 1) / (32 * plan.waves));
    const int64_t groups = B * kv_heads * plan.row_tiles;
    const int64_t most = std::max<int64_t>(1, span / 512);
    plan.splits = (int)std::min<int64_t>(std::min((256 + groups - 1) / groups, most), 128);
    return plan;
  }
  plan.waves = 4;
  plan.row_tiles = (int)((rows + kRows - 1) / kRows);
  // Splits until there are four workgroups a CU, with at least four steps a wave.
  const int64_t groups = B * kv_heads * plan.row_tiles;
  const int64_t steps = (span + kStep - 1) / kStep;
  const int64_t most = std::max<int64_t>(1, steps / (4 * plan.waves));
  const int64_t want = (4 * 256 + groups - 1) / std::max<int64_t>(1, groups);
  plan.splits = (int)std::min<int64_t>(std::min(want, most), 128);
  if (const char* e = getenv("BX_WAVES")) plan.waves = atoi(e);
  if (const char* e = getenv("BX_SPLITS")) plan.splits = std::max(1, atoi(e));
  return plan;
}

hipError_t launch_kv_attention(AttentionParams p, const AttentionPlan& plan, int dtype,
                               hipStream_t stream) {
  p.row_tiles = plan.row_tiles;
  p.splits = plan.splits;
  const int D = p.cache.head_dim;
  hipError_t err = plan.tiles  ? launch_attention_tiles(p, plan.waves, dtype, stream)
                   : D == 64   ? launch_groups<64>(p, plan.waves, dtype, stream)
                   : D == 128  ? launch_groups<128>(p, plan.waves, dtype, stream)
                               : launch_groups<256>(p, plan.waves, dtype, stream);
  if (err != hipSuccess || p.splits == 1) return err;
  const dim3 grid((unsigned)((int64_t)p.B * p.max_q * p.q_heads)), block(256);
  if (D == 64)
    hipLaunchKernelGGL(attention_join_kernel<64>, grid, block, 0, stream, p);
  else if (D == 128)
    hipLaunchKernelGGL(attention_join_kernel<128>, grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL(attention_join_kernel<256>, grid, block, 0, stream, p);
  launch_log(grid, block, 256 * 16 + 256 / (D / 4) * 4, "attention_join_kernel<%d>", D);
  return hipGetLastError();
}

}  // namespace attn
}  // namespace bitmm
