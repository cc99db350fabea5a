// Attention of many query rows (prefill) over the 4-bit cache.
//
// Mathematics. Queries times scale * log2(e), keys and values are binary16 in LDS and registers,
// s (c - 8) + (b + 8 s) two codes at a time; the products' sums are f32 and start from -m, so that
// scores leave the matrix cores as the exponents of p = exp2(x - m). The sum of p is f32, taken
// before the rounding; p is rounded to binary16 for the product with the values. m follows the
// largest score only where a sum says that probabilities near the ends of binary16's range. Each
// of these roundings is 2^-12 of a value on the average where the cache keeps 4 bits: with bf16
// results the error is that of the result's own rounding. Binary16 results would be off by 4.5e-4 of
// their size against 2.1e-4 for their rounding alone. So with binary16 queries only values and
// probabilities are rounded (3.0e-4): keys are s (c - 8) alone, which is exact, and b + 8 s goes through
// one or two products more, in two parts, with the sums of the queries over each group; of the scores'
// factor the queries take the power of two, and the scores the rest. That takes 3 to 7 % longer (4096
// queries over 16384 tokens: 1.26 -> 1.32 ms). The factor on the keys instead, where f32 holds it, would
// round the scales: 8.0e-4.
//
// Layout. A workgroup of eight waves (four for heads of 256 dims) takes up to 256 query rows of one
// sequence and kv head (its new tokens times the query heads that share the kv head) and goes over
// the tokens in tiles of 128 (64 for 256 dims). A tile is expanded once a workgroup: each thread
// keeps the words of the tile after next in registers, turns them into binary16 in LDS for the next
// one (two buffers, one barrier a tile), and the waves multiply the present one, 64 tokens at a
// time. Scores and outputs are formed transposed (32x32x16, lane (c, h) = (lane % 32, lane / 32)
// holds query row c): a lane's sixteen scores of 32 tokens are the next product's operand as they
// stand.
//   keys    LDS rows of head_dim values; the 16-byte piece w of row r sits at w ^ swz(r), so
//           the sixteen rows that a quarter of a wave reads at once hit distinct banks.
//   values  LDS rows likewise, read by transposing reads (ds_read_b64_tr_b16): within 16 lanes,
//           lane m points at row m / 4, values 4 (m % 4) .. +3, and lane i receives value i of
//           the four rows.
// The eight dims of a word stay in the order in which its codes come out, 0 4 1 5 2 6 3 7, in
// keys and queries alike; outputs are put in order when they are stored.
//
// What bounds it: the two waves of a SIMD between matrix cores and vector units. 4096 queries at
// the end of 16384 tokens, 40 heads over 8 of 128 dims: 1.2 ms, 35 us of it for the join of the last
// round's split tiles, 1.0 PFLOP/s, with the matrix cores busy in 44 % of the cycles (1.0 ms with
// nothing but the products and their reads) and vector instructions issued in 45 %. LDS is busy in 39 % of
// them, 29 % of that with bank conflicts. Measured slower:
// the next scores formed beside the softmax of the last (1.9 ms), waves in two sets that take turns
// behind barriers (2.1 ms), 64 tokens between barriers and a maximum looked for each time (1.53 ms).
#include "attention.hpp"

namespace bitmm {
namespace attn {
namespace {

typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4_t lds_i16x4;

// What workgroups tell their waves about the tiles, beside keys and values.
struct TileNotes {
  struct Tile {
    uint64_t bad[2];   // tokens with a scale or bias that is not finite
    uint64_t gone[2];  // tokens on pages outside the cache
    // How many keys and values (in the upper half) do not fit the units, and the largest size (f32 bits) in
    // their waves and the smallest that is not zero (its bits inverted).
    uint32_t apart, most[2], least[2];
  } tile[4];           // by tile % 4
  static constexpr int WORDS = sizeof(Tile) / 4;
  uint32_t undone;     // the first tile's units do not fit all tokens
  float2 first[8];     // the largest sizes of the first tile's keys and values, by wave
  int2 apart[2][128];  // exponents of a token's keys and values over the units, by tile % 2, where some have any
};

template <int D, int GS, int NW, int H>
struct TileLoad {
  static constexpr int THREADS = 64 * NW;
  static constexpr int TPT = THREADS / (64 * H);         // threads of a token
  static constexpr int W = D / 8 / TPT;                  // words of a thread, of keys and values each
  static constexpr int PAIRS = (W * 8 + GS - 1) / GS;
  uint32_t k[W], v[W], kp[PAIRS], vp[PAIRS];
};

// The next N LDS reads, or matrix products, in the order that the scheduler is asked for.
template <int N>
__device__ __forceinline__ void sched_reads() {
  __builtin_amdgcn_sched_group_barrier(0x100, N, 0);
}
template <int N>
__device__ __forceinline__ void sched_products() {
  __builtin_amdgcn_sched_group_barrier(0x008, N, 0);
}

__device__ __forceinline__ void wait_lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// LDS of a workgroup: two tiles of keys and values, and for binary16 results two of the keys' biases: four places
// a group, in products' steps of 16.
template <int D, int NW>
constexpr int kTileBytes = NW * 64 * D * 2;
template <int D, int GS, int DT>
constexpr int kBiasSteps = DT == 1 ? (4 * D / GS + 15) / 16 : 0;
template <int D, int GS, int DT, int NW>
constexpr int kBiasBytes = NW * 32 * 32 * kBiasSteps<D, GS, DT>;

// A workgroup's rows.
template <int RW>
struct Rows {
  Work work;
  Extent ex;
  int r0, rows;
  __device__ __forceinline__ Rows(const AttentionParams& p, int tid, int workgroup)
      : work(p, workgroup), ex(extent_of(p, work.b, tid == 0)), r0(work.row_tile * 32 * RW), rows(min(32 * RW, ex.rows - r0)) {}
};

__device__ __forceinline__ float larger(float a, float b) {
  return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
}

// What a wave gathers: outputs in units of 2^unit, the exponents' reference and the sum.
template <int D>
struct Gathered {
  f32x16_t o[D / 32];
  float m, l;
  int unit;
};

// RW: waves that take rows of their own. Eight waves are eight row waves, or two for each of four: the one takes
// the first 64 tokens of each tile, the other the rest, and they join at the end.
// CAREFUL: with units that change and tokens that have their own. Without, the first tile's units have to do for
// all, and it returns false where they do not.
template <int D, int GS, int DT, int NW, int RW, bool CAREFUL>
__device__ __forceinline__ bool gather_tiles(const AttentionParams& p, const Rows<RW>& mine, int tid, char* lds, TileNotes& notes,
                                             Gathered<D>& out) {
  // A tile is one or two halves of 64 tokens, as LDS allows: with two, waves run freely between
  // barriers for twice as long.
  constexpr int H = NW / 4, TILE = 64 * H;
  constexpr bool PAIRED = RW < NW;
  using L = TileLoad<D, GS, NW, H>;
  constexpr int ROW = D * 2;                  // bytes of an LDS row
  constexpr int SIDE = TILE * ROW;           // bytes of a tile's keys or values
  constexpr int DB = D / 32;                  // blocks of output dims
  constexpr int V_AHEAD = 4;                  // value operands read before the first product
  static_assert(4 * SIDE == kTileBytes<D, NW>, "tiles");
  // Binary16 results have bits enough to show the rounding of keys and of scaled queries.
  constexpr bool EXACT = DT == 1;
  constexpr int BS = kBiasSteps<D, GS, DT>, BIAS_ROW = 32 * BS;  // steps and bytes of a token's biases
  static_assert(2 * TILE * BIAS_ROW == kBiasBytes<D, GS, DT, NW>, "biases");
  static_assert(!PAIRED || H == 2, "halves");

  const Work work = mine.work;
  const Extent ex = mine.ex;
  const int head = work.head, b = work.b, r0 = mine.r0, rows = mine.rows;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 31, h = lane >> 5;
  const Steps<TILE> steps(position(ex, r0 / p.share), position(ex, (r0 + rows - 1) / p.share), p.window, p.sinks);
  const Part part = part_of(steps.count, work.split, work.splits);
  const int i0 = part.first, i1 = part.last;
  const int32_t* table = p.page_table + (int64_t)b * p.pages_per_seq;
  if (tid < 4 * TileNotes::WORDS) reinterpret_cast<uint32_t*>(notes.tile)[tid] = 0;
  if (tid == 0) notes.undone = 0;
  if constexpr (EXACT)  // also those that no group has
    for (int at = 16 * tid; at < 2 * TILE * BIAS_ROW; at += 16 * L::THREADS)
      *reinterpret_cast<u32x4_t*>(lds + 4 * SIDE + at) = u32x4_t{0, 0, 0, 0};

  // This wave's rows, and this lane's.
  const int wr = r0 + 32 * (wave % RW);
  const bool wave_live = wr < ex.rows;
  const int lo_pos = position(ex, min(wr, ex.rows - 1) / p.share);
  const int hi_pos = position(ex, min(wr + 31, ex.rows - 1) / p.share);
  const int pos = position(ex, min(wr + c, ex.rows - 1) / p.share);

  // The row as binary16 and times the scores' factor, for keys in units of 2^k_unit, so that the
  // products are base-2 logarithms as they stand. Where that would pass binary16's range (scores
  // of 10^5 and more) the row is taken 2^-r fold, and its scores 2^r fold (`wide`). So it is where it
  // would near the other end (scores below 2^-4, but for tokens of a larger unit of their own). EXACT: times
  // the factor's power of two alone, the rest of which is in `wide`.
  f16x8_t q[D / 16];
  [[maybe_unused]] f16x8_t q_sums[EXACT ? BS : 1];
  float wide = 1.f;
  bool any_wide = EXACT;
  const float factor = p.scale * kLog2e;
  auto load_query = [&] {  // as it is
    const RowOf row(p, head, opaque(min(wr + c, ex.rows - 1)));
    const uint16_t* qrow = p.q + (int64_t)(ex.q0 + row.i) * p.q_stride + (int64_t)row.head * D;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) q[s] = __builtin_bit_cast(f16x8_t, load_u128(qrow + 16 * s + 8 * h));
  };
  auto convert_query = [&](int k_unit) {
    float big = 0.f;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      const u32x4_t raw = __builtin_bit_cast(u32x4_t, q[s]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x, y;
        unpack_half2<DT>(raw[e], x, y);
        big = fmaxf(big, fmaxf(fabsf(x), fabsf(y)));
      }
    }
    big = across32(big, Max());
    int r = 0;
    if (big > 0.f && big < __uint_as_float(0x7F800000u) && factor != 0.f) {
      const int end = __builtin_amdgcn_frexp_expf(big) + __builtin_amdgcn_frexp_expf(factor) + k_unit;
      r = end > 15 ? end - 15 : end < -7 ? max(end, -80) : 0;
    }
    int unit = k_unit - r;
    wide = ldexpf(1.f, r);
    if constexpr (EXACT) {
      unit = factor != 0.f ? unit + __builtin_amdgcn_frexp_expf(factor) : -300;
      wide *= factor != 0.f ? __builtin_amdgcn_frexp_mantf(factor) : 1.f;
    } else {
      any_wide = __any(r != 0);
    }
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      const u32x4_t raw = __builtin_bit_cast(u32x4_t, q[s]);
      float x[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) unpack_half2<DT>(raw[e], x[2 * e], x[2 * e + 1]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y = x[(e & 1) * 4 + e / 2];
        q[s][e] = (_Float16)ldexpf(EXACT ? y : y * factor, unit);
      }
    }
    if constexpr (EXACT) {
      constexpr int NG = D / GS, STEPS = GS / 16;
      float sum[4 * BS];  // of the groups, over their dims' number
#pragma unroll
      for (int y = 0; y < 4 * BS; ++y) {
        sum[y] = 0.f;
        if (y < NG) {
#pragma unroll
          for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[y] += (float)q[y * STEPS + s][e];
          sum[y] = across32(sum[y], Add()) * (1.f / GS);
        }
      }
#pragma unroll
      for (int t = 0; t < BS; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float y = h ? sum[4 * t + 2 + e] : sum[4 * t + e];
          const _Float16 hi = (_Float16)y, lo = (_Float16)(y - (float)hi);
          q_sums[t][4 * e] = q_sums[t][4 * e + 1] = hi;
          q_sums[t][4 * e + 2] = q_sums[t][4 * e + 3] = lo;
        }
    }
  };
  load_query();

  // ---- the tile's words: token tid / TPT, words (tid % TPT) W .. --------------------------
  const int lt = tid / L::TPT, lw = (tid % L::TPT) * L::W;
  auto page_of = [&](int i) {
    const int t = steps.base(i) + lt;
    return i < i1 && t < ex.kv ? table[t >> p.cache.page_shift] : 0;
  };
  auto load = [&](int i, int page, L& t) {
    const int at = steps.base(i) + lt;
    const bool inside = (uint32_t)page < (uint32_t)p.cache.num_pages;
    const bool live = i < i1 && at < ex.kv && inside;
    const int64_t row = (int64_t)((uint64_t)(uint32_t)(inside ? page : 0) * (uint32_t)(p.cache.kv_heads << p.cache.page_shift)) +
                        ((head << p.cache.page_shift) + (at & ((1 << p.cache.page_shift) - 1)));
    const uint32_t* kc = p.cache.k_codes + row * (D / 8) + lw;
    const uint32_t* vc = p.cache.v_codes + row * (D / 8) + lw;
    if constexpr (L::W == 1) {
      t.k[0] = kc[0];
      t.v[0] = vc[0];
    } else if constexpr (L::W == 2) {
      const u32x2_t a = *reinterpret_cast<const u32x2_t*>(kc), w = *reinterpret_cast<const u32x2_t*>(vc);
      t.k[0] = a[0];
      t.k[1] = a[1];
      t.v[0] = w[0];
      t.v[1] = w[1];
    } else {
#pragma unroll
      for (int e = 0; e < L::W; e += 4) {
        const u32x4_t a = load_u128(kc + e), w = load_u128(vc + e);
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          t.k[e + f] = a[f];
          t.v[e + f] = w[f];
        }
      }
    }
#pragma unroll
    for (int e = 0; e < L::PAIRS; ++e) {
      t.kp[e] = p.cache.k_scales[row * (D / GS) + lw * 8 / GS + e];
      t.vp[e] = p.cache.v_scales[row * (D / GS) + lw * 8 / GS + e];
    }
    if (!live) {
#pragma unroll
      for (int e = 0; e < L::PAIRS; ++e) t.kp[e] = t.vp[e] = 0;
      if (i < i1 && at < ex.kv) {
        atomicOr(reinterpret_cast<unsigned long long*>(&notes.tile[i & 3].gone[lt >> 6]), 1ull << (lt & 63));
        if (p.status && any_sees(at, at, position(ex, r0 / p.share), position(ex, (r0 + rows - 1) / p.share), p.window, p.sinks))
          *p.status = 1;
      }
    }
  };

  TileKeys uk;  // of the tile being written
  Values uv;
  // The size of a thread's token. As bits, where what is not finite is larger than all else.
  static_assert(L::TPT == 4, "token_size");
  auto token_size = [](const uint32_t* pairs) {
    float m = pair_size(pairs[0]);
#pragma unroll
    for (int e = 1; e < L::PAIRS; ++e) m = larger(m, pair_size(pairs[e]));
    return reduce_lanes<4>(m, larger);
  };
  // Tokens that are not finite are marked and emptied.
  auto empty_odd = [&](int i, L& t) {
    bool odd = false;
#pragma unroll
    for (int e = 0; e < L::PAIRS; ++e) {
      odd = odd || !pair_finite(t.kp[e]) || !pair_finite(t.vp[e]);
      if (!pair_finite(t.kp[e])) t.kp[e] = 0;
      if (!pair_finite(t.vp[e])) t.vp[e] = 0;
    }
    if (odd) atomicOr(reinterpret_cast<unsigned long long*>(&notes.tile[i & 3].bad[lt >> 6]), 1ull << (lt & 63));
  };
  // What the workgroup is told of a tile's keys (side 0) or values: not negative, so their bits are in order.
  auto tell = [&](int i, int side, const auto& u, float size) {
    TileNotes::Tile& note = notes.tile[i & 3];
    const uint32_t apart = __builtin_popcountll(__ballot(!u.fits(size))) / 4;
    const float most = reduce_lanes<64>(size, Max()), least = reduce_lanes<64>(size > 0.f ? size : 3e38f, Min());
    if (lane == 0) {
      atomicAdd(&note.apart, apart << (16 * side));
      atomicMax(&note.most[side], __float_as_uint(most));
      atomicMax(&note.least[side], ~__float_as_uint(least));
    }
  };
  // Whether the tile's tokens fit the units, told to the workgroup if not.
  auto measure = [&](int i, L& t) {
    if (__any(!uk.fits(token_size(t.kp)) || !uv.fits(token_size(t.vp)))) {
      empty_odd(i, t);
      tell(i, 0, uk, token_size(t.kp));
      tell(i, 1, uv, token_size(t.vp));
    }
  };
  Sizes k_sizes, v_sizes;  // not CAREFUL: of all tokens, looked at in the end
  auto collect = [&](const L& t) {
    k_sizes.add(token_size(t.kp));
    v_sizes.add(token_size(t.vp));
  };
  auto expand_side = [&](const uint32_t* words, const uint32_t* pairs, float down, char* row, int swz) {
#pragma unroll
    for (int e = 0; e < L::PAIRS; ++e) {
      const float s = bf16_lo(pairs[e]) * down;
      const f16x2_t s2 = splat_f16(s), b2 = splat_f16(fmaf(8.f, s, bf16_hi(pairs[e]) * down));
      constexpr int PER = L::W / L::PAIRS;
#pragma unroll
      for (int f = e * PER; f < (e + 1) * PER; ++f) {
        const uint32_t w = words[f], w8 = w >> 8;
        const u32x4_t a = {as_u32(__builtin_elementwise_fma(codes_low(w), s2, b2)),
                           as_u32(__builtin_elementwise_fma(codes_high(w), s2, b2)),
                           as_u32(__builtin_elementwise_fma(codes_low(w8), s2, b2)),
                           as_u32(__builtin_elementwise_fma(codes_high(w8), s2, b2))};
        *reinterpret_cast<u32x4_t*>(row + (((lw + f) ^ swz) << 4)) = a;
      }
    }
  };
  auto key_swz = [](int row) { return D == 64 ? (row >> 1) & 7 : row & 15; };
  auto value_swz = [](int row) { return D == 64 ? 4 * ((row >> 1) & 1) : 4 * (row & 3); };
  // EXACT: a scale's 8 bits times a code less eight are within binary16's 11. What is left of a key is the same for
  // all dims of a group, b + 8 s: times their number and as two parts, twice, for the queries' sums over it.
  [[maybe_unused]] char* biases = lds + 4 * SIDE;
  [[maybe_unused]] auto expand_keys = [&](const L& t, char* row, char* bias_row) {
#pragma unroll
    for (int e = 0; e < L::PAIRS; ++e) {
      const float s = bf16_lo(t.kp[e]) * uk.down(), b = fmaf(8.f, s, bf16_hi(t.kp[e]) * uk.down()) * GS;
      const f16x2_t s2 = splat_f16(s);
      constexpr int PER = L::W / L::PAIRS;
#pragma unroll
      for (int f = e * PER; f < (e + 1) * PER; ++f) {
        const uint32_t w = t.k[f], w8 = w >> 8;
        const u32x4_t a = {as_u32(codes_low(w) * s2), as_u32(codes_high(w) * s2), as_u32(codes_low(w8) * s2),
                           as_u32(codes_high(w8) * s2)};
        *reinterpret_cast<u32x4_t*>(row + (((lw + f) ^ key_swz(lt)) << 4)) = a;
      }
      if ((lw + e * PER) * 8 % GS == 0) {
        const _Float16 hi = (_Float16)b;
        const uint32_t parts = as_u32(f16x2_t{hi, (_Float16)(b - (float)hi)});
        *reinterpret_cast<u32x2_t*>(bias_row + (lw + e * PER) * 8 / GS * 8) = u32x2_t{parts, parts};
      }
    }
  };
  auto expand = [&](int i, const L& t) {
    char* base = lds + (i & 1) * 2 * SIDE;
    if constexpr (EXACT)
      expand_keys(t, base + lt * ROW, biases + ((i & 1) * TILE + lt) * BIAS_ROW);
    else
      expand_side(t.k, t.kp, uk.down(), base + lt * ROW, key_swz(lt));
    expand_side(t.v, t.vp, uv.down(), base + SIDE + lt * ROW, value_swz(lt));
  };
  // CAREFUL: where tokens of a tile were found not to fit the units: others for most of them, and units of
  // their own for the rest. Returns whether there may be such a rest.
  auto settle = [&](int i, uint32_t apart, L& t) {
    const int tokens = max(min(TILE, ex.kv - steps.base(i)), 0);
    auto rest = [&](int side, int count, auto& u) {
      if (2 * count <= tokens) return count > 0;
      const TileNotes::Tile& note = notes.tile[i & 3];
      const bool first = !u.set;  // then all that have a size have told it
      u.take(__uint_as_float(note.most[side]));
      return !first || !u.fits(__uint_as_float(note.most[side])) || !u.fits(__uint_as_float(~note.least[side]));
    };
    const bool keys = rest(0, apart & 0xFFFF, uk), values = rest(1, apart >> 16, uv);
    if (!__builtin_amdgcn_readfirstlane(keys || values)) return false;
    const int kd = uk.apart(token_size(t.kp)), vd = uv.apart(token_size(t.vp));
#pragma unroll
    for (int e = 0; e < L::PAIRS; ++e) {
      t.kp[e] = pair_down(t.kp[e], kd);
      t.vp[e] = pair_down(t.vp[e], vd);
    }
    if (tid % 4 == 0) notes.apart[i & 1][lt] = make_int2(kd, vd);
    return true;
  };
  auto tokens_apart = [&](int i) { return (uint32_t)__builtin_amdgcn_readfirstlane(notes.tile[i & 3].apart); };

  f32x16_t(&o)[DB] = out.o;
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[d][e] = 0.f;
  float &m = out.m, &l = out.l;
  m = neg_inf();
  l = 0.f;
  f32x16_t start;  // what a score's sum starts from: -m, over `wide`
#pragma unroll
  for (int e = 0; e < 16; ++e) start[e] = 0.f;
  int& o_unit = out.unit;  // exponent of the outputs' unit
  o_unit = 0;

  // Read offsets. Keys: row c of a block of 32 tokens, pieces 2 s + h. Values: see above.
  const int krow = c * ROW, kswz = key_swz(c);
  const int tm = lane & 15, tg = (lane >> 4) & 1;
  const int vrow = (4 * h + (tm >> 2)) * ROW;
  const int vpiece = 2 * tg + ((tm & 3) >> 1), vswz = value_swz(tm >> 2), vhalf = 8 * (tm & 1);

  L t;
  bool spread = false;  // some tokens of the tile being multiplied may have units of their own
  int page = 0;
  if (i0 < i1) {
    const int page0 = page_of(i0), page1 = page_of(i0 + 1);
    page = page_of(i0 + 2);
    __syncthreads();  // the notes are clear
    load(i0, page0, t);
    if constexpr (CAREFUL) {
      empty_odd(i0, t);
      tell(i0, 0, uk, token_size(t.kp));
      tell(i0, 1, uv, token_size(t.vp));
      __syncthreads();
      if (const uint32_t apart = tokens_apart(i0)) spread = settle(i0, apart, t);
    } else {
      collect(t);
      const float key = reduce_lanes<64>(k_sizes.most(), Max()), value = reduce_lanes<64>(v_sizes.most(), Max());
      if (lane == 0) notes.first[wave] = make_float2(key, value);
      __syncthreads();
      float2 all = notes.first[0];
#pragma unroll
      for (int w = 1; w < NW; ++w) {
        all.x = fmaxf(all.x, notes.first[w].x);
        all.y = fmaxf(all.y, notes.first[w].y);
      }
      uk.take(all.x);
      uv.take(all.y);
    }
    expand(i0, t);
    load(i0 + 1, page1, t);
    if constexpr (CAREFUL)
      measure(i0 + 1, t);
    else
      collect(t);
  }
  int k_unit = uk.e, v_unit = uv.e;  // of the tile being multiplied
  int q_unit = k_unit;
  if constexpr (!CAREFUL) o_unit = v_unit;
  convert_query(q_unit);
  for (int i = i0; i < i1; ++i) {
    wait_lds_barrier();
    if (tid < TileNotes::WORDS) reinterpret_cast<uint32_t*>(&notes.tile[(i + 3) & 3])[tid] = 0;
    [[maybe_unused]] bool spread_next = false;
    if constexpr (CAREFUL)
      if (const uint32_t apart = tokens_apart(i + 1)) spread_next = settle(i + 1, apart, t);
    [[maybe_unused]] const int k_next = uk.e, v_next = uv.e;
    expand(i + 1, t);
    load(i + 2, page, t);
    page = page_of(i + 3);

#pragma unroll 1
    for (int half = PAIRED ? wave / RW : 0; half < (PAIRED ? wave / RW + 1 : H); ++half) {
      const int base = steps.base(i) + 64 * half;
      if (!wave_live || base > hi_pos) break;
      // Before the window of all the wave's rows, and past the first tokens (chunks of 1024 tokens
      // with a window of 512: 39.6 -> 36.8 us).
      if (p.window > 0 && base + 63 <= lo_pos - p.window && base >= p.sinks) continue;
      const char* kb = lds + (i & 1) * 2 * SIDE + half * 64 * ROW;
      const char* vb = kb + SIDE;
      const uint64_t bad = CAREFUL ? notes.tile[i & 3].bad[half] : 0, gone = notes.tile[i & 3].gone[half];
      if (CAREFUL && k_unit != q_unit) {
        q_unit = k_unit;
        load_query();
        convert_query(q_unit);
#pragma unroll
        for (int e = 0; e < 16; ++e) start[e] = m == neg_inf() ? 0.f : -m / wide;
      }
      // Between the products a wave goes first: its SIMD's other wave then has products to fill the
      // time with (1.31 -> 1.27 ms at 4096 queries over 16384 tokens).
      __builtin_amdgcn_s_setprio(0);
      f32x16_t x[2];
      constexpr int PRODUCTS = 2 * (D / 16);
      auto key = [&](int s, int tb) {
        return __builtin_bit_cast(f16x8_t, *reinterpret_cast<const u32x4_t*>(kb + tb * 32 * ROW + krow +
                                                                           (((2 * s + h) ^ kswz) << 4)));
      };
      auto score = [&](int s, int tb, f16x8_t k) {
        x[tb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, q[s], s ? x[tb] : CAREFUL ? f32x16_t{} : start, 0, 0, 0);
      };
      if constexpr (D == 64) {
        // All keys of the half before the first product: the order below leaves each read to be
        // waited for where there are so few (4 % of a chunk's time).
        f16x8_t k[PRODUCTS];
#pragma unroll
        for (int n = 0; n < PRODUCTS; ++n) k[n] = key(n / 2, n % 2);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < PRODUCTS; ++n) score(n / 2, n % 2, k[n]);
      } else {
        // Order of the scheduler's making: AHEAD reads, then a read with each product.
        constexpr int AHEAD = 6;
#pragma unroll
        for (int n = 0; n < PRODUCTS; ++n) score(n / 2, n % 2, key(n / 2, n % 2));
        sched_reads<AHEAD>();
        static_for<0, PRODUCTS - AHEAD>([](auto) {
          sched_products<1>();
          sched_reads<1>();
        });
        sched_products<AHEAD>();
      }
      if constexpr (EXACT) {
        const char* rows_at = biases + ((i & 1) * TILE + half * 64 + c) * BIAS_ROW + 16 * h;
#pragma unroll
        for (int t = 0; t < BS; ++t)
#pragma unroll
          for (int tb = 0; tb < 2; ++tb)
            x[tb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                __builtin_bit_cast(f16x8_t, *reinterpret_cast<const u32x4_t*>(rows_at + tb * 32 * BIAS_ROW + 32 * t)), q_sums[t],
                x[tb], 0, 0, 0);
      }
      __builtin_amdgcn_s_setprio(1);
      if constexpr (CAREFUL) {
        // The scores stand alone: beside -m the small ones of small keys would be rounded. They become the
        // exponents of what the values are multiplied by.
        const int2* apart = notes.apart[i & 1] + 64 * half + 4 * opaque(h);
        const float was = m == neg_inf() ? 0.f : m;
#pragma unroll
        for (int tb = 0; tb < 2; ++tb)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int2 d = spread ? apart[32 * tb + 8 * (e >> 2) + (e & 3)] : make_int2(0, 0);
            x[tb][e] = ldexpf(x[tb][e] * wide, d.x) - was + (float)d.y;
          }
      } else if (any_wide) {
#pragma unroll
        for (int tb = 0; tb < 2; ++tb)
#pragma unroll
          for (int e = 0; e < 16; ++e) x[tb][e] *= wide;
      }
      // Score e of block tb is token 32 tb + 8 (e / 4) + 4 h + e % 4 of the half.
      auto mask = [&](auto keep) {
#pragma unroll
        for (int tb = 0; tb < 2; ++tb)
#pragma unroll
          for (int e = 0; e < 16; ++e) x[tb][e] = keep(32 * tb + 8 * (e >> 2) + (e & 3)) ? x[tb][e] : neg_inf();
      };
      if (base + 63 > lo_pos) {
        const int last = opaque(pos) - base - 4 * h;
        mask([&](int at) { return at <= last; });
      }
      if (p.window > 0 && base <= hi_pos - p.window) {
        const int before = opaque(pos) - p.window - base - 4 * h, sinks = p.sinks - base - 4 * h;
        if (base < p.sinks)
          mask([&](int at) { return (at > before) | (at < sinks); });
        else
          mask([&](int at) { return at > before; });
      }
      if (bad || gone) {
        const int h4 = 4 * opaque(h);
#pragma unroll
        for (int tb = 0; tb < 2; ++tb)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int at = 32 * tb + 8 * (e >> 2) + h4 + (e & 3);
            const bool see = x[tb][e] != neg_inf() && !(gone >> at & 1);
            x[tb][e] = !see ? neg_inf() : bad >> at & 1 ? quiet_nan() : x[tb][e];
          }
      }
      if (CAREFUL && v_unit != o_unit) {
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int e = 0; e < 16; ++e) o[d][e] = ldexpf(o[d][e], o_unit - v_unit);
        o_unit = v_unit;
      }
      u32x4_t pr[4];
      float sum = 0.f;
      auto exponentials = [&] {
        float odd = 0.f;
        sum = 0.f;
#pragma unroll
        for (int tb = 0; tb < 2; ++tb)
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float p0 = __builtin_amdgcn_exp2f(x[tb][e]), p1 = __builtin_amdgcn_exp2f(x[tb][e + 1]);
            sum += p0;
            odd += p1;
            pr[2 * tb + (e >> 3)][(e & 7) / 2] = pack_half2<1>(p0, p1);
          }
        sum += odd;
      };
      exponentials();
      // The reference m of the exponents is set so that the largest probability is 2^4, and need not follow
      // scores as long as a half's probabilities neither near binary16's upper end nor become all small: a
      // sum from 2^-9 to 2^15.9 says so (32 of them round to 2^-25 at worst, 2^-11 of that together; none at
      // all are masked ones). Only past it is a maximum looked for.
      if (spread | __any(!(sum <= 61440.f) || (sum < 0x1p-9f && sum > 0.f) || m == neg_inf())) {
        float top = neg_inf();
#pragma unroll
        for (int tb = 0; tb < 2; ++tb)
#pragma unroll
          for (int e = 0; e < 16; ++e) top = fmaxf(top, x[tb][e]);
        top = across32(top, Max());
        const bool seen = top > neg_inf();
        float up = 0.f, alpha = 1.f;
        if (m == neg_inf()) {
          up = seen ? top - 4.f : 0.f;
          m = seen ? up : m;
        } else {
          float sofar = l;
          if constexpr (CAREFUL) {  // else none of the values is beyond 2^15 units
            float most = opaque(0.f);
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
              for (int e = 0; e < 16; ++e) most = fmaxf(most, fabsf(o[d][e]));
            sofar = fmaxf(sofar, most * 0x1p-15f);
          }
          const float room = room_below(across32(sofar, Max()));
          up = top > 4.f ? top - 4.f : seen && top < -4.f ? fmaxf(top - 4.f, -room) : 0.f;
          alpha = __builtin_amdgcn_exp2f(-up);
          m += up;
        }
        if (__any(up != 0.f)) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            if constexpr (!CAREFUL) start[e] = m == neg_inf() ? 0.f : -m / wide;
            x[0][e] -= up;
            x[1][e] -= up;
          }
          l *= alpha;
#pragma unroll
          for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[d][e] *= alpha;
          exponentials();
        }
        if (spread) {  // the sum is of the probabilities alone
          const int2* apart = notes.apart[i & 1] + 64 * half + 4 * opaque(h);
          sum = 0.f;
#pragma unroll
          for (int tb = 0; tb < 2; ++tb)
#pragma unroll
            for (int e = 0; e < 16; ++e)
              sum += __builtin_amdgcn_exp2f(x[tb][e] - (float)apart[32 * tb + 8 * (e >> 2) + (e & 3)].y);
        }
      }
      l += sum;
      __builtin_amdgcn_s_setprio(0);
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int d = 0; d < DB; ++d) {
          const char* at = vb + vrow + (((4 * d + vpiece) ^ vswz) << 4) + vhalf;
          const u32x2_t lo = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(at + 16 * s * ROW)));
          const u32x2_t hi = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(at + (16 * s + 8) * ROW)));
          const u32x4_t a = {lo[0], lo[1], hi[0], hi[1]};
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, pr[s]), o[d], 0, 0, 0);
        }
      sched_reads<2 * V_AHEAD>();
      static_for<0, 4 * DB - V_AHEAD>([](auto) {
        sched_products<1>();
        sched_reads<2>();
      });
      sched_products<V_AHEAD>();
    }
    if constexpr (CAREFUL) {
      measure(i + 2, t);
      k_unit = k_next;
      v_unit = v_next;
      spread = spread_next;
    } else {
      collect(t);
    }
  }
  if constexpr (!CAREFUL) {
    if (__any(!k_sizes.fit(uk) || !v_sizes.fit(uv)) && lane == 0) notes.undone = 1;
    __syncthreads();
    return !__builtin_amdgcn_readfirstlane(notes.undone);
  }
  return true;
}

template <int D, int GS, int DT, int NW, int RW>
__global__ __launch_bounds__(64 * NW, NW / 4) void attention_tiles_kernel(AttentionParams p) {
  constexpr bool PAIRED = RW < NW;
  constexpr int ROW = D * 2, DB = D / 32;
  __shared__ __attribute__((aligned(16))) char lds[kTileBytes<D, NW> + kBiasBytes<D, GS, DT, NW>];
  __shared__ TileNotes notes;
  static_assert(RW * 32 * ROW <= kTileBytes<D, NW> && (!PAIRED || RW * (D / 2 * 256 + 512) <= kTileBytes<D, NW>), "epilogue");
  // The row tiles of a sequence and kv head on one XCD: its codes meet in one L2.
  const int tid = threadIdx.x, workgroup = xcd_remap(blockIdx.x, gridDim.x);
  const Rows<RW> own(p, tid, workgroup);
  if (own.rows <= 0) return;
  Gathered<D> got;
  if (!gather_tiles<D, GS, DT, NW, RW, false>(p, own, tid, lds, notes, got)) {
    __syncthreads();
    const AttentionParams& again = params_again();
    const int same = opaque(tid);
    gather_tiles<D, GS, DT, NW, RW, true>(again, Rows<RW>(again, same, scalar_again(workgroup)), same, lds, notes, got);
  }
  f32x16_t(&o)[DB] = got.o;
  float m = got.m, l = got.l;
  int o_unit = got.unit;
  const Work work = own.work;
  const Extent ex = own.ex;
  const int head = work.head, b = work.b;
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 31, h = lane >> 5;
  const int wr = own.r0 + 32 * (wave % RW);
  auto key_swz = [](int row) { return D == 64 ? (row >> 1) & 7 : row & 15; };

  l = across32(l, Add());
  if constexpr (PAIRED) {
    // [wave of the pair's rows][register][lane], then references and sums.
    float* part = reinterpret_cast<float*>(lds) + (wave % RW) * (D / 2 * 64 + 128) + lane;
    __syncthreads();
    if (wave >= RW) {
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) part[(16 * d + e) * 64] = ldexpf(o[d][e], o_unit);
      part[D / 2 * 64] = m;
      part[D / 2 * 64 + 64] = l;
    }
    __syncthreads();
    if (wave < RW) {
      const float m2 = part[D / 2 * 64], l2 = part[D / 2 * 64 + 64], mt = fmaxf(m, m2);
      const float f = m == mt ? 1.f : __builtin_amdgcn_exp2f(m - mt), f2 = m2 == mt ? 1.f : __builtin_amdgcn_exp2f(m2 - mt);
      const float own = ldexpf(f, o_unit);
      m = mt;
      l = l * f + l2 * f2;
      o_unit = 0;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] = o[d][e] * own + part[(16 * d + e) * 64] * f2;
    }
  }
  const RowOf mine_row(p, head, opaque(min(wr + c, ex.rows - 1)));
  const bool live = wr + c < ex.rows && wave < RW;
  const float out_scale = work.splits > 1 ? ldexpf(1.f, o_unit) : (l == 0.f ? 0.f : ldexpf(1.f / l, o_unit));
  // Dims of a lane's registers: block d, eight dims e / 4, of which (0, 4, 1, 5) for h = 0 and
  // (2, 6, 3, 7) for h = 1, so that registers (0, 2) and (1, 3) are neighbouring dims.
  if (work.splits > 1) {
    if (!live) return;
    const int64_t at = part_row(p, work.split * p.B + b, head, wr + c);
    if (h == 0) {
      p.part_ml[2 * at] = m;
      p.part_ml[2 * at + 1] = l;
    }
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        float* to = p.part_o + at * D + 32 * d + 2 * e + 2 * h;
        *reinterpret_cast<float2*>(to) = make_float2(o[d][e] * out_scale, o[d][e + 2] * out_scale);
        *reinterpret_cast<float2*>(to + 4) = make_float2(o[d][e + 1] * out_scale, o[d][e + 3] * out_scale);
      }
    return;
  }
  if (p.lse && live && h == 0) p.lse[(int64_t)(ex.q0 + mine_row.i) * p.q_heads + mine_row.head] = kLn2 * (m + __builtin_amdgcn_logf(l));
  if (p.otype == kOutF32) {
    if (!live) return;
    float* to0 = static_cast<float*>(p.out) + (int64_t)(ex.q0 + mine_row.i) * p.out_stride + (int64_t)mine_row.head * D;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        float* to = to0 + 32 * d + 2 * e + 2 * h;
        *reinterpret_cast<float2*>(to) = make_float2(o[d][e] * out_scale, o[d][e + 2] * out_scale);
        *reinterpret_cast<float2*>(to + 4) = make_float2(o[d][e + 1] * out_scale, o[d][e + 3] * out_scale);
      }
    return;
  }
  // 16-bit outputs go through LDS, so that a row is stored in 16-byte pieces. The wave's own
  // region: no barrier but the one that ends the tiles.
  __syncthreads();
  if (wave >= RW) return;
  char* mine = lds + wave * 32 * ROW;
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      const int dim = 32 * d + 2 * e + 2 * h;
      const float y0 = o[d][e] * out_scale, y1 = o[d][e + 2] * out_scale;
      const float y2 = o[d][e + 1] * out_scale, y3 = o[d][e + 3] * out_scale;
      const uint32_t a = p.otype == kOutBf16 ? pack_half2<0>(y0, y1) : pack_half2<1>(y0, y1);
      const uint32_t w = p.otype == kOutBf16 ? pack_half2<0>(y2, y3) : pack_half2<1>(y2, y3);
      char* to = mine + c * ROW + (((dim >> 3) ^ key_swz(c)) << 4);
      *reinterpret_cast<uint32_t*>(to + 4 * h) = a;
      *reinterpret_cast<uint32_t*>(to + 8 + 4 * h) = w;
    }
  constexpr int PIECES = D / 8;  // of a row
#pragma unroll
  for (int e = 0; e < 32 * PIECES / 64; ++e) {
    const int at = e * 64 + lane, rr = at / PIECES, piece = at % PIECES;
    const u32x4_t y = *reinterpret_cast<const u32x4_t*>(mine + rr * ROW + ((piece ^ key_swz(rr)) << 4));
    if (wr + rr < ex.rows) {
      const int i = (wr + rr) / p.share, qh = head * p.share + (wr + rr) % p.share;
      *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p.out) + (int64_t)(ex.q0 + i) * p.out_stride +
                                  (int64_t)qh * D + 8 * piece) = y;
    }
  }
}

template <int D, int GS, int NW, int RW>
hipError_t launch_tiles(const AttentionParams& p, unsigned workgroups, int dtype, hipStream_t stream) {
  const dim3 grid(workgroups);
  if (dtype == 0)
    hipLaunchKernelGGL((attention_tiles_kernel<D, GS, 0, NW, RW>), grid, dim3(64 * NW), 0, stream, p);
  else
    hipLaunchKernelGGL((attention_tiles_kernel<D, GS, 1, NW, RW>), grid, dim3(64 * NW), 0, stream, p);
  launch_log(grid, dim3(64 * NW), (size_t)(NW * 64 * D * 2 + (dtype ? kBiasBytes<D, GS, 1, NW> : 0) + sizeof(TileNotes)),
             "attention_tiles_kernel<%d, %d, %d, %d, %d>", D, GS, dtype, NW, RW);
  return hipGetLastError();
}

template <int D, int NW, int RW>
hipError_t launch_groups(const AttentionParams& p, unsigned workgroups, int dtype, hipStream_t stream) {
  if (p.cache.group == 32) return launch_tiles<D, 32, NW, RW>(p, workgroups, dtype, stream);
  if (p.cache.group == 64) return launch_tiles<D, 64, NW, RW>(p, workgroups, dtype, stream);
  if constexpr (D >= 128) return launch_tiles<D, 128, NW, RW>(p, workgroups, dtype, stream);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_attention_tiles(const AttentionParams& p, int rows_each, unsigned workgroups, int dtype,
                                  hipStream_t stream) {
  if (p.cache.head_dim == 256) return launch_groups<256, 4, 4>(p, workgroups, dtype, stream);
  if (p.cache.head_dim == 128)
    return rows_each == 256 ? launch_groups<128, 8, 8>(p, workgroups, dtype, stream)
                            : launch_groups<128, 8, 4>(p, workgroups, dtype, stream);
  return rows_each == 256 ? launch_groups<64, 8, 8>(p, workgroups, dtype, stream)
                          : launch_groups<64, 8, 4>(p, workgroups, dtype, stream);
}

}  // namespace attn
}  // namespace bitmm
