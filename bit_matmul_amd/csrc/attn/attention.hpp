// Device parts shared by the attention kernels: a sequence's extent, the tokens that a tile
// of query rows has to go over, masks, and the binary16 form of the 4-bit codes.
//
// Units. Keys and values enter the matrix cores as binary16, whose eleven bits hold
// scale * code + bias with an eighth of the rounding of bf16, but whose range is narrow
// against a bf16 scale's. So each is taken in units of a power of two 2^E, chosen so that the first tokens'
// largest magnitude is near 2^9 of 2^15 (keys over many rows: 2^3 of 2^8). Scores are scaled back by a factor
// that multiplies them anyway, outputs when they are stored. The largest of a token has all its bits down to
// 2^-6 units. The sizes met are kept, a maximum and a minimum a lane, and looked at when all is done.
// Where a token was not within, all is done again, in a careful form that ordinary data does not meet and
// that has registers of its own: units move to where most tokens of a step or tile are, and any other token has
// a unit 2^d times theirs: its score is multiplied by 2^d, and the exponent of its probability takes d in,
// for the product with the values alone. So no row depends on the size of a token that it does not see.
// (As one form for both, a prompt's chunk took 5 to 15 % longer, for scalar registers alone.)
//
// Probabilities. What the second product takes is exp2(x - m) as binary16, which reaches from 2^16 down to
// 2^-14, or 2^-24 with fewer and fewer bits. m is a reference near the largest score of late, not the largest of
// all: where a token of long ago has most of the weight (the first one often has, with little to give) the rest
// would otherwise be rounded to nothing, each by itself, in an output that they alone make up. m rises when a
// probability nears 2^16, and falls when those of a step or half tile are all small, as long as the sum of what
// came before stays below 2^40 beside them: what they add to it is then past f32's 24 bits.
#pragma once

#include "attn.hpp"

namespace bitmm {
namespace attn {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xFF800000u); }
__device__ __forceinline__ float quiet_nan() { return __uint_as_float(0x7FC00000u); }

__device__ __forceinline__ f16x2_t as_f16x2(uint32_t w) { return __builtin_bit_cast(f16x2_t, w); }
__device__ __forceinline__ uint32_t as_u32(f16x2_t v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ f16x2_t splat_f16(float v) {
  const _Float16 h = (_Float16)v;
  return f16x2_t{h, h};
}

// Codes of bits [0, 4) of each half of w, less eight (exact): 1024 + c in binary16 is
// 0x6400 | c. And of bits [4, 8): 1024 + 16 c.
__device__ __forceinline__ f16x2_t codes_low(uint32_t w) {
  return as_f16x2(and_or_b32(w, 0x000F000Fu, 0x64006400u)) - splat_f16(1032.f);
}
__device__ __forceinline__ f16x2_t codes_high(uint32_t w) {
  return __builtin_elementwise_fma(as_f16x2(and_or_b32(w, 0x00F000F0u, 0x64006400u)),
                                   splat_f16(0.0625f), splat_f16(-72.f));
}

// What a sequence has, with lengths and offsets cut to what the host was told.
struct Extent {
  int q0;     // first query row
  int rows;   // query rows of one kv head: queries * share
  int first;  // position of the first query (may be negative)
  int kv;     // tokens
};

__device__ __forceinline__ Extent extent_of(const AttentionParams& p, int b, bool report) {
  Extent e;
  const int c0 = p.cu_q[b], c1 = p.cu_q[b + 1], len = p.kv_lens[b];
  const int64_t room = p.pages_per_seq << p.cache.page_shift;
  const int most = (int)(room < p.max_kv ? room : p.max_kv);
  const int q0 = min(max(c0, 0), p.T);
  const int q1 = min(max(c1, q0), p.T);
  const int n = q1 - q0;
  e.q0 = q0;
  e.kv = min(max(len, 0), most);
  e.rows = min(n, p.max_q) * p.share;
  e.first = e.kv - n;
  if (report && p.status && (q0 != c0 || q1 != c1 || n > p.max_q || e.kv != len)) *p.status = 1;
  return e;
}

// Position of the sequence's query i. Those before the first token see nothing, wherever they are: all at
// -1, so that a window's width can be taken off any position in 32 bits.
__device__ __forceinline__ int position(const Extent& e, int i) { return max(e.first + i, -1); }

// Row r of a sequence and kv head: query i of the sequence, one of the heads that share.
struct RowOf {
  int i, head;
  __device__ __forceinline__ RowOf(const AttentionParams& p, int kv_head, int r) {
    i = r / p.share;
    head = kv_head * p.share + r - i * p.share;
  }
};

// The tokens that rows at positions lo_pos .. hi_pos go over, in steps of STEP tokens that
// start at multiples of it: first those of the tokens that stay visible, then the window's.
template <int STEP>
struct Steps {
  int sink_steps;
  int start;  // first token of the window's steps
  int count;

  __device__ __forceinline__ Steps(int lo_pos, int hi_pos, int window, int sinks) {
    const int hi = hi_pos + 1;
    const int lo = window > 0 ? max(0, lo_pos - window + 1) : 0;
    start = lo / STEP * STEP;
    sink_steps = window > 0 ? (min(sinks, lo) + STEP - 1) / STEP : 0;
    if (sink_steps * STEP > start) {
      sink_steps = 0;
      start = 0;
    }
    count = hi > 0 ? sink_steps + (hi - start + STEP - 1) / STEP : 0;
  }
  __device__ __forceinline__ int base(int i) const {
    return i < sink_steps ? i * STEP : start + (i - sink_steps) * STEP;
  }
};

// A lane's value moved across; zero where none arrives.
template <int CTRL, int ROWS>
__device__ __forceinline__ int moved(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}

// The balanced form: B * splits slots of workgroups shared out among up to 64 sequences so that all
// have about as many steps. Lane b holds sequence b.
struct Share {
  int b, first, count;  // sequence (-1: none), its first slot and how many it has
};
struct Shares {
  Extent mine;
  int count, end;  // slots of lane b's sequence, and up to its end

  __device__ __forceinline__ Shares(const AttentionParams& p, int lane, bool report) {
    mine = lane < p.B ? extent_of(p, lane, report) : Extent{0, 0, 0, 0};
    int steps = 0;
    if (mine.rows > 0) {
      steps = Steps<32>(position(mine, 0), position(mine, (mine.rows - 1) / p.share), p.window, p.sinks).count;
    }
    const int slots = p.B * p.splits;
    auto sum = [](int v) {
      return (int)__float_as_uint(reduce_lanes<64>(__uint_as_float((uint32_t)v), AddInt()));
    };
    // A last share is half full on the average; all fit for certain if each may be nearly empty.
    // A sequence without steps still has its rows to write.
    const int total = __builtin_amdgcn_readfirstlane(sum(steps));
    auto shared_out = [&](int of) {
      const int share = max(1, (total + of - 1) / of);
      count = mine.rows > 0 ? max(1, (steps + share - 1) / share) : 0;
      return __builtin_amdgcn_readfirstlane(sum(count)) <= slots;
    };
    if (!shared_out(slots - p.B / 2)) shared_out(slots - p.B);
    end = count;
    end += moved<0x111, 0xF>(end);  // within 16 lanes, from 1, 2, 4 and 8 before
    end += moved<0x112, 0xF>(end);
    end += moved<0x114, 0xF>(end);
    end += moved<0x118, 0xF>(end);
    end += moved<0x142, 0xA>(end);  // the 16 lanes before, then the 32
    end += moved<0x143, 0xC>(end);
  }
  __device__ __forceinline__ Share of_sequence(int b) const {
    const int n = __builtin_amdgcn_readlane(count, b);
    return {b, __builtin_amdgcn_readlane(end, b) - n, n};
  }
  __device__ __forceinline__ Share of_slot(int slot) const {
    const int b = __builtin_popcountll(__ballot(end <= slot));
    return b < 64 ? of_sequence(b) : Share{-1, 0, 0};
  }
  __device__ __forceinline__ Extent extent(int b) const {
    return {__builtin_amdgcn_readlane(mine.q0, b), __builtin_amdgcn_readlane(mine.rows, b),
            __builtin_amdgcn_readlane(mine.first, b), __builtin_amdgcn_readlane(mine.kv, b)};
  }
};

// Without branches: it is asked for each score of a step at the edge of what is visible.
__device__ __forceinline__ bool visible(int token, int pos, int window, int sinks) {
  return (token <= pos) & ((window <= 0) | (token > pos - window) | (token < sinks));
}

// Whether a row at one of the positions lo_pos .. hi_pos sees one of the tokens from .. to.
__device__ __forceinline__ bool any_sees(int from, int to, int lo_pos, int hi_pos, int window, int sinks) {
  return from <= hi_pos && (window <= 0 || to > lo_pos - window || from < sinks);
}

// A kernel's parameters, and a scalar, to be read and worked with anew: what a rare second attempt shares with the
// first one would take up scalar registers throughout.
__device__ __forceinline__ const AttentionParams& params_again() {
  typedef __attribute__((address_space(4))) AttentionParams Params;
  const Params* p = (const Params*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const AttentionParams*)p;
}
__device__ __forceinline__ int scalar_again(unsigned v) { return __builtin_amdgcn_readfirstlane(opaque((int)v)); }

// A workgroup's work: a sequence and kv head, one of its row tiles, and which part of how many of
// the tokens.
struct Work {
  int b, head, row_tile, split, splits;
  __device__ __forceinline__ Work(const AttentionParams& p, int id) {
    const int whole = p.row_tiles - p.tail_tiles, each = whole + p.tail_tiles * p.splits;
    const int group = id / each, k = id - group * each;
    b = group / p.cache.kv_heads;
    head = group - b * p.cache.kv_heads;
    if (k < whole) {  // the last rows see most: they come first
      row_tile = p.row_tiles - 1 - k;
      split = 0;
      splits = 1;
    } else {
      const int t = (k - whole) / p.splits;
      row_tile = p.tail_tiles - 1 - t;
      split = k - whole - t * p.splits;
      splits = p.splits;
    }
  }
};

// Row r of a kv head in part `part` of the partial results: parts are a split of a sequence, split
// by split, or in the balanced form the slots of the sequences one after the other.
__device__ __forceinline__ int64_t part_row(const AttentionParams& p, int part, int head, int r) {
  return ((int64_t)part * p.cache.kv_heads + head) * p.tail_rows + r;
}

// The steps [first, last) of part `split` of `splits`: the first ones take one more where the
// count does not divide.
struct Part {
  int first, last;
};
__device__ __forceinline__ Part part_of(int count, int split, int splits) {
  const int each = count / splits, more = count - each * splits;
  Part s;
  s.first = split * each + min(split, more);
  s.last = s.first + each + (split < more ? 1 : 0);
  return s;
}

__device__ __forceinline__ bool pair_finite(uint32_t pair) {
  return (pair & 0x7F80u) != 0x7F80u && (pair & 0x7F800000u) != 0x7F800000u;
}
__device__ __forceinline__ float pair_size(uint32_t pair) {
  return fmaf(15.f, fabsf(bf16_lo(pair)), fabsf(bf16_hi(pair)));
}

// 15 s + |b| of the largest finite s and b is past f32.
__device__ __forceinline__ int size_exponent(float size) { return __builtin_amdgcn_frexp_expf(fminf(size, 3e38f)); }

// The unit 2^e of keys or values. NEAR: the exponent, in units, that a token's size is brought to; MOST: the one
// that it may reach; LOW, HIGH: the units' range. Keys' units may be any that keep their reciprocal finite. Outputs
// are held in the values' units as these change, so those stay where that leaves f32's range alone.
template <int NEAR, int MOST, int LOW, int HIGH>
struct Unit {
  int e = 0;  // in a scalar register, and all else made from it
  bool set = false;  // before tokens with a nonzero magnitude have come, those of zero alone fit
  __device__ __forceinline__ float down() const { return __uint_as_float((uint32_t)(127 - e) << 23); }
  // The sizes of tokens that it is good for, as bits.
  __device__ __forceinline__ uint32_t most() const { return set ? (uint32_t)(127 + min(e + MOST, 127)) << 23 : 0; }
  __device__ __forceinline__ uint32_t least() const { return set ? (uint32_t)(127 + max(e - 6, -126)) << 23 : 0; }
  __device__ __forceinline__ bool fits(float size) const {
    return size <= __uint_as_float(most()) && (size >= __uint_as_float(least()) || size == 0.f);
  }
  // Takes a unit for a size, the same in every lane.
  __device__ __forceinline__ void take(float size) {
    const float m = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(size)));
    e = __builtin_amdgcn_readfirstlane(min(max(size_exponent(m) - NEAR, LOW), HIGH));
    set = true;
  }
  // The exponent d of a token that does not fit, over the unit.
  __device__ __forceinline__ int apart(float size) const { return fits(size) ? 0 : size_exponent(size) - NEAR - e; }
};

// The largest and smallest of some sizes, that of zero apart, and whether a unit is good for all between.
// As bits: those of what is not finite are larger than all others, and zero, less one, is large.
struct Sizes {
  uint32_t high = 0, low = ~0u;
  __device__ __forceinline__ void add(float size) {
    high = max(high, __float_as_uint(size));
    low = min(low, __float_as_uint(size) - 1);
  }
  __device__ __forceinline__ float most() const { return __uint_as_float(high); }
  template <typename U>
  __device__ __forceinline__ bool fit(const U& u) const {
    return high <= u.most() && low >= u.least() - 1;
  }
};
using RowsKeys = Unit<9, 15, -120, 118>;
using TileKeys = Unit<3, 8, -120, 118>;
using Values = Unit<9, 15, -30, 30>;

// A pair in units 2^d times larger: exact, where it does not become too small to matter.
__device__ __forceinline__ uint32_t pair_down(uint32_t pair, int d) {
  return pack_bf16x2(ldexpf(bf16_lo(pair), -d), ldexpf(bf16_hi(pair), -d));
}

// How many bits the reference of a row's exponents may still fall, by the largest of its sum l so far and
// 2^-15 of its outputs, in all its lanes: until that is near 2^40.
__device__ __forceinline__ float room_below(float largest) {
  return (float)max(0, 40 - __builtin_amdgcn_frexp_expf(largest));
}

// Four neighbouring outputs at index `at` of p.out.
__device__ __forceinline__ void store4(const AttentionParams& p, int64_t at, float a, float b, float c, float d) {
  if (p.otype == kOutF32)
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(p.out) + at) = f32x4_t{a, b, c, d};
  else
    *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(p.out) + at) =
        p.otype == kOutBf16 ? u32x2_t{pack_half2<0>(a, b), pack_half2<0>(c, d)}
                            : u32x2_t{pack_half2<1>(a, b), pack_half2<1>(c, d)};
}

}  // namespace attn
}  // namespace bitmm
