// Attention of a few query rows over a long 4-bit cache (decoding), and the join of partial
// results.
//
// Mathematics. With key j = s_g c + b_g in group g of the head's dims (c the code of a dim),
//   q . k_j = sum_g s_g (sum q c - 8 sum q) + (b_g + 8 s_g) sum q
// over each group's dims, so bare codes (as 1024 + c: mask and OR) go through the matrix cores, a
// product a group whose sum starts from what takes 1024 + 8 off again, and two f32 operations a
// group give the score. Softmax in one pass: a running reference m and sum l of exp2(x - m), outputs
// scaled when m moves. Values are expanded to binary16, s (c - 8) + (b + 8 s), two at a time.
//
// Rounded to binary16 (11 bits, against the cache's 4): s and b + 8 s of each pair, values,
// probabilities. Queries are not, but for parts of a binary16 row 2^-14 and less of its largest.
// Sums, maxima and scores are f32.
//
// Layout. A workgroup takes 16 query rows of one sequence and kv head (the query heads that share
// it, times the sequence's new tokens) and a range of the tokens, in steps of 32 that go round its
// waves; each wave keeps m, l and outputs of its own, joined through LDS at the end. Scores and
// outputs are formed transposed, S^T = K Q^T and O^T = V^T P^T: in the matrix cores' layouts
// (16x16x32, lane (n, g) = (lane % 16, lane / 16)) a lane then holds one query row throughout. Its
// probabilities are the second product's operand as they stand, its maximum, sum and factors are
// plain registers, and nothing passes between lanes but the maximum. Row n of the first product is
// token 4 (n % 4) + n / 4 of a half step, so that lane (n, g) has the scores of tokens g, 4 + g,
// 8 + g and 12 + g.
//
// Codes are copied from HBM straight to LDS, a step ahead, in a ring of two steps of the wave's own
// (no barrier; 140 us with codes loaded to registers against 127), and their pairs through
// registers. Where they lie is held in scalar registers: 16 tokens of a half step share a page.
//
// What bounds it: with a long cache, HBM and the vector units together. Four sequences of 131072
// tokens, 40 heads over 8 of 128 dims, groups of 64: 604 MB in 121 us, 5.0 TB/s, with vector
// instructions issued in 64 % of the cycles; 6 us more for the join. Expanding keys and values to
// binary16 with their scales, as the kernel for many rows does, took 217 us. With short or windowed
// spans, latency: vector instructions in 50 % (32 ragged sequences) and 46 % (windows of 4096 at 256
// dims) of the cycles, waves waiting in 39 % and 37 % of theirs.
#pragma once

#include <algorithm>

#include "attention.hpp"

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
// `outside` collects whether a page was outside the cache that holds tokens which a row sees.
template <typename F>
__device__ __forceinline__ StepPlace step_place(const Cache& c, int head_row, int kv, int base,
                                                const StepPages& pages, F seen, bool& outside) {
  StepPlace s;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int tb = base + 16 * u;
    const int page = __builtin_amdgcn_readfirstlane(pages.page[u]);
    const bool inside = (uint32_t)page < (uint32_t)c.num_pages;
    outside = outside || (!inside && seen(tb, tb + 15));
    s.ok[u] = tb < kv && inside;
    s.row[u] = (int64_t)(inside ? page : 0) * (c.kv_heads << c.page_shift) + (head_row + (tb & ((1 << c.page_shift) - 1)));
  }
  return s;
}

// Copies and loads go through descriptors whose bases are those rows: scalar registers hold what
// moves from step to step and no 64-bit address is formed in a lane. They span the 16 rows,
// which lie within one page.

// Pairs of a side of a step: those of a half are 16 NG neighbouring words, and pair 64 e + lane
// of the step is token (64 e + lane) / NG, group (64 e + lane) % NG.
template <int NG, int PL>
__device__ __forceinline__ void load_pairs(const uint32_t* scales, const StepPlace& s, int lane, uint32_t (&to)[PL]) {
  constexpr int BYTES = 64 * NG;  // of a half step's pairs
  if constexpr (NG >= 4) {
    const __amdgpu_buffer_rsrc_t half[2] = {make_rsrc(scales + s.row[0] * NG, BYTES), make_rsrc(scales + s.row[1] * NG, BYTES)};
#pragma unroll
    for (int e = 0; e < PL; ++e)
      to[e] = __builtin_amdgcn_raw_buffer_load_b32(half[e / (NG / 4)], 4 * lane, 256 * (e % (NG / 4)), 0);
  } else {
    // Both halves in one wave, mostly as neighbours; a load past its descriptor's span gives 0.
    const bool joined = s.row[1] == s.row[0] + 16;
    to[0] = __builtin_amdgcn_raw_buffer_load_b32(make_rsrc(scales + s.row[0] * NG, joined ? 2 * BYTES : BYTES), 4 * lane, 0, 0);
    if (!joined) to[0] |= __builtin_amdgcn_raw_buffer_load_b32(make_rsrc(scales + s.row[1] * NG, BYTES), 4 * lane - BYTES, 0, 0);
  }
}

// Codes in LDS: rows of D / 2 bytes one after the other, and within a row the 16-byte piece w at
// w ^ swizzle(row), so that the pieces which the rows of a product's operand are read at lie on
// distinct banks. For heads of 256 dims, where straight rows meet on two places (decode of 64
// sequences over windows of 4096 tokens, in groups of 32: 50 us against 47); narrower rows meet
// little, and the extra arithmetic costs 1.5 %.
template <int D>
__device__ __forceinline__ constexpr int swizzle(int row) {
  return D == 256 ? (row >> 1) & 7 : 0;
}

// Copies the codes of a side of a step to LDS.
template <int D>
__device__ __forceinline__ void copy_codes(const uint32_t* codes, const StepPlace& s, int lane, char* to) {
  constexpr int HALF = 8 * D, PIECES = D / 32;  // bytes of 16 rows, pieces of a row
  // Source of the 16 bytes that land at place `at` of a half.
  auto source = [](int at) {
    const int row = at / PIECES;
    return 16 * (row * PIECES + ((at % PIECES) ^ swizzle<D>(row)));
  };
  if constexpr (D == 64) {  // one instruction's lanes hold both halves
    const int from = source(lane & 31);
    if (lane < 32)
      dma<16>(make_rsrc(codes + s.row[0] * (D / 8), HALF), from, to);
    else
      dma<16>(make_rsrc(codes + s.row[1] * (D / 8), HALF), from, to);
  } else {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const __amdgpu_buffer_rsrc_t from = make_rsrc(codes + s.row[u] * (D / 8), HALF);
#pragma unroll
      for (int e = 0; e < HALF / 1024; ++e) dma<16>(from, source(64 * e + lane), to + u * HALF + 1024 * e);
    }
  }
}

// A pair as binary16 in units of 2^e: (scale, bias + 8 scale), for codes less eight.
__device__ __forceinline__ uint32_t pair_f16(uint32_t pair, float down) {
  const float s = bf16_lo(pair) * down;
  return pack_half2<1>(s, fmaf(8.f, s, bf16_hi(pair) * down));
}

// The largest of a token's NG pairs, which lie side by side, in all their lanes.
template <int NG>
__device__ __forceinline__ float token_size(float v) {
  if constexpr (NG == 2) return fmaxf(v, dpp<0xB1>(v));
  if constexpr (NG >= 4) return reduce_lanes<NG>(v, Max());
  return v;
}
template <int PL>
__device__ __forceinline__ float largest(const float (&size)[PL]) {
  float m = size[0];
#pragma unroll
  for (int e = 1; e < PL; ++e) m = fmaxf(m, size[e]);
  return reduce_lanes<64>(m, Max());
}
// Whether most of the tokens that have a size do not fit.
template <typename U, int PL>
__device__ __forceinline__ bool mostly_apart(const U& u, const float (&size)[PL]) {
  int out = 0, all = 0;
#pragma unroll
  for (int e = 0; e < PL; ++e) {
    out += __builtin_popcountll(__ballot(!u.fits(size[e])));
    all += __builtin_popcountll(__ballot(size[e] > 0.f));
  }
  return 2 * out > all;
}

// LDS of a workgroup. Each wave's own: codes of two steps (keys, then values), and the pairs of one as binary16,
// [group][place] of the keys and of the values, where token t of a half is at 4 (t % 4) + t / 4, and the
// exponents of its tokens' keys and values over the units, where some have units of their own.
// The joined outputs afterwards.
template <int D, int GS, int WAVES>
struct RowsLds {
  static constexpr int SIDE = 16 * D;  // bytes of a step's keys or values
  static constexpr int WAVE_BYTES = 4 * SIDE + 2 * 32 * (D / GS) * 4 + 2 * 32 * 4, JOIN_BYTES = D / 16 * 4 * 64 * 4;
  __attribute__((aligned(16))) char bytes[WAVES * (WAVE_BYTES > JOIN_BYTES ? WAVE_BYTES : JOIN_BYTES)];
  float ml[WAVES][2][16];
};

// One result on top of another's: outputs of units 2^unit, which may differ, the sum of lane group g alone where the
// other's is whole.
template <int J, typename F>
__device__ __forceinline__ void take_in(f32x4_t (&o)[J], float& m, float& l, int& unit, float m2, float l2, F outputs) {
  const float top = fmaxf(m, m2);
  const float mine = m == top ? 1.f : __builtin_amdgcn_exp2f(m - top), other = m2 == top ? 1.f : __builtin_amdgcn_exp2f(m2 - top);
  const float ours = ldexpf(mine, unit);
  unit = 0;  // theirs may be far from it
  m = top;
  l = l * mine + l2 * other;
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[j][e] = o[j][e] * ours + outputs(j, e) * other;
}

// A workgroup's rows: those of a row tile, and which part of how many of the tokens; `part` is its place in the
// partial results.
struct Rows {
  Work work;
  Extent ex;
  int part, r0, rows;  // no rows: nothing to do
};
template <int PASS>
__device__ __forceinline__ Rows rows_of(const AttentionParams& p, int tid, int workgroup) {
  Work work(p, workgroup);
  Extent ex;
  int part = work.split * p.B + work.b;
  if (PASS != kPrefix && p.balanced) {
    part = workgroup / p.cache.kv_heads;
    work.head = workgroup - part * p.cache.kv_heads;
    const Shares shares(p, tid & 63, workgroup == 0);
    const Share mine = shares.of_slot(part);
    work.b = max(mine.b, 0);
    work.split = part - mine.first;
    work.splits = mine.count;
    ex = shares.extent(work.b);
    if (mine.b < 0) ex.rows = 0;
  } else {
    ex = extent_in_pass<PASS>(p, work.b, tid == 0);
  }
  const int r0 = work.row_tile * kRows;
  return {work, ex, part, r0, min(kRows, ex.rows - r0)};
}

// The same rows over the tokens that their group shares, all of which they see.
__device__ __forceinline__ Rows shared_rows_of(const AttentionParams& prefix, const Rows& own, int group) {
  Rows rows = own;
  rows.work.b = group;
  rows.work.split = 0;
  rows.work.splits = 1;
  const int64_t room = prefix.pages_per_seq << prefix.cache.page_shift;
  rows.ex.kv = min(max(prefix.kv_lens[group], 0), (int)(room < prefix.max_kv ? room : prefix.max_kv));
  rows.ex.first = rows.ex.kv - 1;
  rows.ex.step = 0;
  return rows;
}

// What a wave gathers: outputs in units of 2^unit, the exponents' reference and the sum.
template <int D>
struct Gathered {
  f32x4_t o[D / 16];
  float m, l;
  int unit;
};

// A wave's share of the tokens. CAREFUL: with units that change and tokens that have their own. Without, those of
// the wave's first step have to do for all its tokens, and it returns false where they do not. SHARE: the wave takes
// turns with those that its Turn says, not with all of the workgroup.
struct Turn {
  int index, count;
};
template <int D, int GS, int DT, int WAVES, bool CAREFUL, bool SHARE = false>
__device__ __forceinline__ bool gather_rows(const AttentionParams& p, const Rows& mine, int tid, RowsLds<D, GS, WAVES>& mem,
                                            Gathered<D>& out, Turn turn = {}) {
  constexpr int NG = D / GS;                         // groups of a head
  constexpr int J = D / 16;                          // output tiles
  constexpr int KW = D / 32, WG = GS / 32;           // a lane's key words, and those of a group
  constexpr int VW = D >= 128 ? D / 128 : 1;         // words of a value piece (64: half a word)
  constexpr int PL = NG > 2 ? NG / 2 : 1;            // pairs of a lane
  constexpr int SIDE = RowsLds<D, GS, WAVES>::SIDE, WAVE_BYTES = RowsLds<D, GS, WAVES>::WAVE_BYTES;
  char* lds = mem.bytes;

  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4;
  char* ring = lds + wave * WAVE_BYTES;
  uint32_t* k_pairs = reinterpret_cast<uint32_t*>(ring + 4 * SIDE);
  uint32_t* v_pairs = k_pairs + 32 * NG;
  int(*apart)[32] = reinterpret_cast<int(*)[32]>(v_pairs + 32 * NG);

  const Work work = mine.work;
  const Extent ex = mine.ex;
  const int head = work.head, r0 = mine.r0, rows = mine.rows;
  const int lo_pos = position(ex, r0 / p.share);
  const int hi_pos = position(ex, (r0 + rows - 1) / p.share);
  const Steps<kStep> steps(lo_pos, hi_pos, p.window, p.sinks);
  const Part range = part_of(steps.count, work.split, work.splits);
  const int i0 = range.first, i1 = range.last;
  const int32_t* table = p.page_table + (int64_t)work.b * p.pages_per_seq;

  uint32_t kp[PL], vp[PL];  // pairs of the step being copied
  StepPages pages = {};
  StepPlace place = {};
  bool outside = false;
  auto seen = [&](int from, int to) { return any_sees(from, to, lo_pos, hi_pos, p.window, p.sinks); };
  const int head_row = head << p.cache.page_shift;
  const int first = i0 + (SHARE ? turn.index : wave), each = SHARE ? turn.count : WAVES;
  if constexpr (SHARE) {
    if (first >= i1) {  // nothing to do, nor to prepare for it
#pragma unroll
      for (int j = 0; j < J; ++j) out.o[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      out.m = neg_inf();
      out.l = 0.f;
      out.unit = 0;
      return true;
    }
  }
  auto copy = [&](int stage) {
    char* to = ring + stage * 2 * SIDE;
    copy_codes<D>(p.cache.k_codes, place, lane, to);
    copy_codes<D>(p.cache.v_codes, place, lane, to + SIDE);
    load_pairs<NG, PL>(p.cache.k_scales, place, lane, kp);
    load_pairs<NG, PL>(p.cache.v_scales, place, lane, vp);
  };
  if (first < i1) {
    pages = step_pages(p, table, ex.kv, steps.base(first));
    place = step_place(p.cache, head_row, ex.kv, steps.base(first), pages, seen, outside);
    if (first + each < i1) pages = step_pages(p, table, ex.kv, steps.base(first + each));
    copy(0);
  }

  // This lane's query row as binary16, its largest magnitude in [2^7, 2^8): a bf16 query keeps
  // every bit that way. A word's codes come out in the order 0 4 1 5 2 6 3 7, the odd ones
  // times 16, which the query takes back.
  const RowOf row_of(p, head, min(r0 + n, ex.rows - 1));
  const int pos = position(ex, row_of.i);
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
    // The factor stays positive, so that it can wait until after the maximum.
    c = p.scale == 0.f ? 1.f : ldexpf(fabsf(p.scale) * kLog2e, e2);
    const float sign = p.scale < 0.f ? -1.f : p.scale == 0.f ? 0.f : 1.f;
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
          q[j][e] = (_Float16)(sign * ldexpf(x[(e & 1) * 4 + e / 2], high ? -e2 - 4 : -e2));
          (high ? odd : even) += (float)q[j][e];
        }
      }
      even = across32(across16(even, Add()), Add());
      odd = across32(across16(odd, Add()), Add());
      q_sum[y] = even + 16.f * odd;
      centre[y] = -fmaf(1032.f, even, 1152.f * odd);
    }
  }

  f32x4_t(&o)[J] = out.o;
#pragma unroll
  for (int j = 0; j < J; ++j) o[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  float &m = out.m, &l = out.l;
  m = neg_inf();
  l = 0.f;
  RowsKeys uk;
  Values uv;
  Sizes k_sizes, v_sizes;
  // 1024 twice in binary16, in a register, so that mask and OR are one instruction. (No inline
  // assembly next to the matrix cores: the compiler keeps the distance that their operands and
  // results need only for instructions that it knows.)
  uint32_t k1024 = 0x64006400u;
  asm("" : "+v"(k1024));

  // Steps past it and up to lo_pos are visible to every row.
  const int window_edge = p.window > 0 ? hi_pos - p.window : -1;
  int stage = 0;
  for (int i = first; i < i1; i += each) {
    const int base = steps.base(i);
    const bool ok0 = place.ok[0], ok1 = place.ok[1];
    const char* kc = ring + stage * 2 * SIDE;
    const char* vc = kc + SIDE;
    stage ^= 1;

    // This step's copies and pairs have landed; the next one's go to the other stage, whose codes
    // were all read before.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    // Slots that hold no live token may hold anything.
    const bool plain = ok0 && ok1 && base + kStep - 1 <= lo_pos && base > window_edge;
    uint32_t bad = 0;  // tokens of the step with a scale or bias that is not finite
    if (!plain) {
      const int at = opaque(lane);
#pragma unroll
      for (int e = 0; e < PL; ++e) {
        const int token = (64 * e + at) / NG;
        const bool ok = (token < 16 ? ok0 : ok1) && base + token < ex.kv && token < 32;
        kp[e] = ok ? kp[e] : 0;
        vp[e] = ok ? vp[e] : 0;
      }
    }
    bool spread = false;  // some of the step's tokens have units of their own
    if constexpr (!CAREFUL) {
#pragma unroll
      for (int e = 0; e < PL; ++e) {
        k_sizes.add(pair_size(kp[e]));
        v_sizes.add(pair_size(vp[e]));
      }
      if (i == first) {
        uk.take(reduce_lanes<64>(k_sizes.most(), Max()));
        uv.take(reduce_lanes<64>(v_sizes.most(), Max()));
      }
    } else {
      const int at = opaque(lane);
      float ks[PL], vs[PL];
#pragma unroll
      for (int e = 0; e < PL; ++e) {
        const bool odd_k = !pair_finite(kp[e]), odd_v = !pair_finite(vp[e]);
        if (odd_k) kp[e] = 0;
        if (odd_v) vp[e] = 0;
        if (odd_k || odd_v) bad |= 1u << ((64 * e + at) / NG % 32);
        ks[e] = token_size<NG>(pair_size(kp[e]));
        vs[e] = token_size<NG>(pair_size(vp[e]));
      }
      bad = __float_as_uint(reduce_lanes<64>(__uint_as_float(bad), Or()));
      if (mostly_apart(uk, ks)) uk.take(largest(ks));
      if (mostly_apart(uv, vs)) {
        const int before = uv.e;
        uv.take(largest(vs));
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][e] = ldexpf(o[j][e], before - uv.e);
      }
      bool rest = false;
#pragma unroll
      for (int e = 0; e < PL; ++e) rest = rest || !uk.fits(ks[e]) || !uv.fits(vs[e]);
      spread = __any(rest);
      if (spread) {
#pragma unroll
        for (int e = 0; e < PL; ++e) {
          const int kd = uk.apart(ks[e]), vd = uv.apart(vs[e]);
          kp[e] = pair_down(kp[e], kd);
          vp[e] = pair_down(vp[e], vd);
          const int f = 64 * e + at;
          if (f < 32 * NG) {
            apart[0][f / NG] = kd;
            apart[1][f / NG] = vd;
          }
        }
      }
    }
    // The wave's own part of LDS: its operations are in order.
#pragma unroll
    for (int e = 0; e < PL; ++e) {
      const int f = 64 * e + lane, t = f / NG;
      if (NG >= 2 || lane < 32) {
        const int to = f % NG * 32 + (t & 16) + 4 * (t & 3) + (t >> 2 & 3);
        k_pairs[to] = pair_f16(kp[e], uk.down());
        v_pairs[to] = pair_f16(vp[e], uv.down());
      }
    }
    __builtin_amdgcn_wave_barrier();
    if (i + each < i1) {
      place = step_place(p.cache, head_row, ex.kv, steps.base(i + each), pages, seen, outside);
      if (i + 2 * each < i1) pages = step_pages(p, table, ex.kv, steps.base(i + 2 * each));
      copy(stage);
    }

    // Scores: the products with the bare codes less eight, group by group, times the scales.
    f32x4_t x[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      x[u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      // Row n of the product is token 4 (n % 4) + n / 4 of the half, so that a lane's four scores
      // are tokens g, 4 + g, 8 + g, 12 + g, whose values the lanes then read in one piece.
      const int k_row = 4 * (n & 3) + (n >> 2), k_swizzle = 16 * swizzle<D>(k_row);
      const char* krow = kc + u * (8 * D) + k_row * (D / 2);
#pragma unroll
      for (int y = 0; y < NG; ++y) {
        uint32_t k[WG];
        if constexpr (WG == 1) {
          k[0] = *reinterpret_cast<const uint32_t*>(krow + ((y * (GS / 2) + g * (GS / 8)) ^ k_swizzle));
        } else if constexpr (WG == 2) {
          const u32x2_t w = *reinterpret_cast<const u32x2_t*>(krow + ((y * (GS / 2) + g * (GS / 8)) ^ k_swizzle));
          k[0] = w[0];
          k[1] = w[1];
        } else {
          const u32x4_t w = *reinterpret_cast<const u32x4_t*>(krow + ((y * (GS / 2) + g * (GS / 8)) ^ k_swizzle));
#pragma unroll
          for (int e = 0; e < 4; ++e) k[e] = w[e];
        }
        float at = centre[y];
        asm volatile("" : "+v"(at));  // made four of here, not kept as four
        f32x4_t sum = {at, at, at, at};
#pragma unroll
        for (int j = y * WG; j < (y + 1) * WG; ++j) {
          const uint32_t w = k[j - y * WG], w8 = w >> 8;
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
        // Done here: moved past the branch below, the sums and pairs of all groups would stay.
        if constexpr (NG >= 4) asm volatile("" : "+v"(x[u]));
      }
    }
    if constexpr (NG < 4) asm volatile("" : "+v"(x[0]), "+v"(x[1]));
    if (!plain || bad) {
      const int g0 = opaque(g);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int at = 16 * u + 4 * t + g0;
          const bool see = (u ? ok1 : ok0) & (base + at < ex.kv) & visible(base + at, pos, p.window, p.sinks);
          const float y = bad >> at & 1 ? quiet_nan() : x[u][t];
          x[u][t] = see ? y : neg_inf();
        }
    }

    const float ck0 = ldexpf(c, uk.e);
    float ck = ck0 < 1e-37f ? 1e-37f : ck0;  // masked scores times 0 would be NaN
    if (CAREFUL && spread) {  // to the exponents of what the values are multiplied by
      const int g0 = opaque(g);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int at = 16 * u + 4 * t + g0;
          x[u][t] = ldexpf(x[u][t] * ck, apart[0][at]) + (float)apart[1][at];
        }
      ck = 1.f;
    }

    // The reference m, kept while the step's largest probability is 2^-4 to 2^12; 2^4 where it is set.
    float top = fmaxf(fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[0][2], x[0][3])),
                      fmaxf(fmaxf(x[1][0], x[1][1]), fmaxf(x[1][2], x[1][3])));
    top = across32(across16(top, Max()), Max()) * ck;
    const float above = top - m;  // NaN where no score is seen yet
    const bool low = above < -4.f && top > neg_inf();
    if (__any(above > 12.f || low)) {
      float sofar = opaque(0.f);
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sofar = fmaxf(sofar, fabsf(o[j][e]));
      sofar = fmaxf(sofar * 0x1p-15f, l);
      const float room = room_below(across32(across16(sofar, Max()), Max()));
      const float to = above > 12.f ? top - 4.f : low ? fmaxf(top - 4.f, m - room) : m;
      const float alpha = m == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(m - to);
      m = to;
      l *= alpha;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] *= alpha;
    }
    const float off = m == neg_inf() ? 0.f : m;
    u32x4_t pr;
    float sum = 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int t = 0; t < 4; t += 2) {
        const float e0 = __builtin_amdgcn_exp2f(fmaf(x[u][t], ck, -off)),
                    e1 = __builtin_amdgcn_exp2f(fmaf(x[u][t + 1], ck, -off));
        sum += e0 + e1;
        pr[2 * u + t / 2] = pack_half2<1>(e0, e1);
      }
    if (CAREFUL && spread) {  // the sum is of the probabilities alone
      const int g0 = opaque(g);
      sum = 0.f;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int t = 0; t < 4; ++t) sum += __builtin_amdgcn_exp2f(x[u][t] - off - (float)apart[1][16 * u + 4 * t + g0]);
    }
    l += sum;
    const f16x8_t prob = __builtin_bit_cast(f16x8_t, pr);

    // Outputs.
    f16x2_t vs[4], vb[4];
    const uint32_t* v_read = v_pairs + n * (D / 16) / GS * 32 + 4 * g;
    uint32_t v[8][VW];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int row = 4 * (t % 4) + g;
      const char* at = vc + t / 4 * (8 * D) + row * (D / 2) + ((n * (D / 32)) ^ (16 * swizzle<D>(row)));
      if constexpr (D == 64) {
        v[t][0] = *reinterpret_cast<const uint16_t*>(at);
      } else if constexpr (D == 128) {
        v[t][0] = *reinterpret_cast<const uint32_t*>(at);
      } else {
        const u32x2_t w = *reinterpret_cast<const u32x2_t*>(at);
        v[t][0] = w[0];
        v[t][1] = w[1];
      }
    }
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
    __builtin_amdgcn_wave_barrier();
  }

  if (outside && p.status && lane == 0) *p.status = 1;

  out.unit = uv.e;
  return CAREFUL || !__any(!k_sizes.fit(uk) || !v_sizes.fit(uv));
}

template <int D, int GS, int DT, int WAVES, int PASS>
__global__ __launch_bounds__(64 * WAVES, D == 256 ? 2 : 4) void attention_rows_kernel(typename PassParams<PASS>::Type params) {
  const AttentionParams& p = params_of(params);
  constexpr int J = D / 16;
  __shared__ RowsLds<D, GS, WAVES> mem;
  const Rows own = rows_of<PASS>(p, threadIdx.x, blockIdx.x);
  if constexpr (PASS == kBoth) report_groups(params.prefix, threadIdx.x);
  if (own.rows <= 0) return;
  [[maybe_unused]] SharedRows shared;
  if constexpr (PASS == kOwn || PASS == kBoth) shared = SharedRows(params.prefix, own.work.b, threadIdx.x & 63);
  Gathered<D> got;
  if constexpr (PASS == kBoth) {
    // The first waves take the shared tokens, the last ones the sequence's own, as many as these are a part of all.
    Rows mine = own;
    const SharedParams& all_params = shared_params_again();  // in memory: one of its two is taken by the wave
    const AttentionParams* tokens = &all_params.own;
    Turn turn = {__builtin_amdgcn_readfirstlane(threadIdx.x >> 6), WAVES};
    if (shared.group >= 0) {
      const Rows before = shared_rows_of(params.prefix, own, shared.group);
      const int own_steps = (position(own.ex, (own.r0 + own.rows - 1) / p.share) + kStep) / kStep;
      const int shared_steps = (before.ex.kv + kStep - 1) / kStep, all = max(own_steps + shared_steps, 1);
      const int last = max(min((WAVES * own_steps + all / 2) / all, shared_steps > 0 ? WAVES - 1 : WAVES), own_steps > 0 ? 1 : 0);
      const bool late = turn.index >= WAVES - last;
      turn = late ? Turn{turn.index - (WAVES - last), last} : Turn{turn.index, WAVES - last};
      if (!late) {
        mine = before;
        tokens = &all_params.prefix;
      }
    }
    if (!gather_rows<D, GS, DT, WAVES, false, true>(*tokens, mine, threadIdx.x, mem, got, turn)) {
      const bool late = tokens == &all_params.own;
      const SharedParams& again = shared_params_again();
      const int same = opaque((int)threadIdx.x);
      gather_rows<D, GS, DT, WAVES, true, true>(late ? again.own : again.prefix, mine, same, mem, got, turn);
    }
  } else if (!gather_rows<D, GS, DT, WAVES, false>(p, own, threadIdx.x, mem, got)) {
    const AttentionParams& again = params_again();
    const int same = opaque((int)threadIdx.x);
    gather_rows<D, GS, DT, WAVES, true>(again, rows_of<PASS>(again, same, scalar_again(blockIdx.x)), same, mem, got);
  }
  f32x4_t(&o)[J] = got.o;
  float m = got.m, l = got.l;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const Work work = own.work;
  const Extent ex = own.ex;
  const int head = work.head, r0 = own.r0;

  auto partial = [&] { return PASS == kPrefix || (p.splits > 1 && (p.balanced || work.splits > 1)); };
  // Of the results over the shared tokens each wave takes in every WAVES-th part: their loads overlap, and the join
  // below is one for all (the parts one after the other behind it: 64 samples, ten parts 23 us against 20).
  [[maybe_unused]] int parts = 0;
  if constexpr (PASS == kBoth) parts = shared.parts(params.prefix, shared.row(params.prefix, ex.q0, min(r0 + n, ex.rows - 1)));
  if constexpr (PASS == kOwn) {
    if (!partial()) {
      const AttentionParams& prefix = params.prefix;
      const int64_t row = shared.row(prefix, ex.q0, min(r0 + n, ex.rows - 1));
      parts = shared.parts(prefix, row);
      for (int s = wave; __any(s < parts); s += WAVES) {
        if (s >= parts) continue;
        const int64_t at = prefix_row(prefix, s, shared.group, head, (int)row);
        const float2 ml = *reinterpret_cast<const float2*>(prefix.part_ml + 2 * at);
        const float* from = prefix.part_o + at * D + 4 * g * J;  // dim (4 g + e) J + j
        f32x4_t theirs[J];
#pragma unroll
        for (int i = 0; i < J; ++i) theirs[i] = *reinterpret_cast<const f32x4_t*>(from + 4 * i);
        if (ml.y == 0.f) continue;  // saw nothing
        // lanes of the other g hold zeros of the row's sum, which is added up below
        take_in(o, m, l, got.unit, ml.x, g == 0 ? ml.y : 0.f, [&](int j, int e) { return theirs[(e * J + j) / 4][j % 4]; });
      }
    }
  }

  // The waves' results joined: each brings its own to the common maximum, and wave w stores
  // every WAVES / 4-th part of dims (4 g + w % 4) D/16 .. of its lanes' rows.
  l = across32(across16(l, Add()), Add());
  if (g == 0) {
    mem.ml[wave][0][n] = m;
    mem.ml[wave][1][n] = l;
  }
  __syncthreads();
  float(*o_lds)[J * 4][64] = reinterpret_cast<float(*)[J * 4][64]>(mem.bytes);
  float mt = neg_inf(), lt = 0.f;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) mt = fmaxf(mt, mem.ml[w][0][n]);
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    const float mw = mem.ml[w][0][n];
    // A sum that is NaN has a maximum of -infinity if it met nothing else.
    lt += mem.ml[w][1][n] * (mw == mt ? 1.f : __builtin_amdgcn_exp2f(mw - mt));
  }
  const float mine = ldexpf(m == mt ? 1.f : __builtin_amdgcn_exp2f(m - mt), got.unit);
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
  const int row = opaque(r0 + n);
  if (partial()) {
    const int64_t at = partial_row<PASS>(p, work, own.part, row);
    if (speaker) {
      p.part_ml[2 * at] = mt;
      p.part_ml[2 * at + 1] = lt;
    }
#pragma unroll
    for (int j = 0; j < JP; j += 4)
      *reinterpret_cast<f32x4_t*>(p.part_o + at * D + dim0 + j) = f32x4_t{y[j], y[j + 1], y[j + 2], y[j + 3]};
    return;
  }
  if ((PASS == kOwn || PASS == kBoth) && parts < 0) {  // past the bound of its group's queries
    if (p.status) *p.status = 1;
    return;
  }
  const RowOf out_row(p, head, row);
  const float inv = lt == 0.f ? 0.f : 1.f / lt;
  if (p.lse && speaker) p.lse[(int64_t)(ex.q0 + out_row.i) * p.q_heads + out_row.head] = kLn2 * (mt + __builtin_amdgcn_logf(lt));
  const int64_t at = (int64_t)(ex.q0 + out_row.i) * p.out_stride + (int64_t)out_row.head * D + dim0;
#pragma unroll
  for (int j = 0; j < JP; j += 4) store4(p, at + j, y[j] * inv, y[j + 1] * inv, y[j + 2] * inv, y[j + 3] * inv);
}

template <int D, int GS, int WAVES, int PASS>
hipError_t launch_rows(const typename PassParams<PASS>::Type& p, unsigned workgroups, int dtype, hipStream_t stream) {
  const dim3 grid(workgroups), block(64 * WAVES);
  if (dtype == 0)
    hipLaunchKernelGGL((attention_rows_kernel<D, GS, 0, WAVES, PASS>), grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL((attention_rows_kernel<D, GS, 1, WAVES, PASS>), grid, block, 0, stream, p);
  static const char* const names[] = {"attention_rows_kernel<%d, %d, %d, %d>", "attention_rows_kernel<%d, %d, %d, %d, prefix>",
                                      "attention_rows_kernel<%d, %d, %d, %d, own>", "attention_rows_kernel<%d, %d, %d, %d, both>"};
  launch_log(grid, block, sizeof(RowsLds<D, GS, WAVES>), names[PASS], D, GS, dtype, WAVES);
  return hipGetLastError();
}

template <int D, int GS, int PASS>
hipError_t launch_waves(const typename PassParams<PASS>::Type& p, unsigned workgroups, int waves, int dtype, hipStream_t stream) {
  if constexpr (PASS == kBoth) return launch_rows<D, GS, 8, PASS>(p, workgroups, dtype, stream);
  return waves == 4 ? launch_rows<D, GS, 4, PASS>(p, workgroups, dtype, stream)
                    : launch_rows<D, GS, 8, PASS>(p, workgroups, dtype, stream);
}

template <int D, int PASS>
hipError_t launch_groups(const typename PassParams<PASS>::Type& p, int group, unsigned workgroups, int waves, int dtype,
                         hipStream_t stream) {
  if (group == 32) return launch_waves<D, 32, PASS>(p, workgroups, waves, dtype, stream);
  if (group == 64) return launch_waves<D, 64, PASS>(p, workgroups, waves, dtype, stream);
  if constexpr (D >= 128) return launch_waves<D, 128, PASS>(p, workgroups, waves, dtype, stream);
  return hipErrorInvalidValue;
}

// The kernel for few query rows.
template <int PASS>
hipError_t launch_attention_rows(const typename PassParams<PASS>::Type& p, const Cache& c, unsigned workgroups, int waves,
                                 int dtype, hipStream_t stream) {
  return c.head_dim == 64    ? launch_groups<64, PASS>(p, c.group, workgroups, waves, dtype, stream)
         : c.head_dim == 128 ? launch_groups<128, PASS>(p, c.group, workgroups, waves, dtype, stream)
                             : launch_groups<256, PASS>(p, c.group, workgroups, waves, dtype, stream);
}

}  // namespace
}  // namespace attn
}  // namespace bitmm
