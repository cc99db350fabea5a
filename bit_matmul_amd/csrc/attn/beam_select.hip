// Beam search's selection: of a group's beams x vocabulary candidates
//   total = score[beam] + x[beam, token] - log sum_t exp x[beam, t]
// the k largest, ties to the lowest (beam, token).
//
// One pass over the logits (beam_scan_kernel): a wave goes over a part of a row, sums its exponentials and keeps
// its k largest logits, whose order is that of the totals. A second kernel (beam_merge_kernel), one workgroup a
// group, joins the parts of each row, then the rows.
//
// Precision. Which of two beams' candidates comes first may hang on the last bits of their rows' sums, so
// exponentials and sums are f64: 2^z with z split into a whole and a fraction by an addition, and a polynomial of
// degree 7 in the fraction whose relative error is 4e-11 (fitted for the smallest largest one). So sums agree with
// exact ones to some 1e-11, and totals to that. Equal rows have equal sums: they are added up in the same order.
// Differences of logits are taken before anything is done with them: two f32 numbers' is exact in f64, or far from
// all that counts. (A reference's product with log2 e, rounded, is off by 2^-53 of it: for logits of 1e8 by more than the
// exponentials, and past 5e18 by whole powers of two.)
//
// The k largest. A wave's threshold is a lower bound of its part's k-th largest logit: the k-th largest of the
// lanes' largest ones at first, then the k-th of those found so far. Logits that pass it go to LDS as pairs
// (order-preserving key, token inverted), one 64-bit number each, so that the pair's order is the candidates';
// where they become many their ranks are counted and the first k stay.
//
// What bounds it: f64 arithmetic, 15 instructions a logit of 18, and latency. 256 rows of 131072 bf16
// logits, a fifth of them not read: 39 us for 54 MB (a copy's rate: 10) with vector instructions issued in 52 % of the
// cycles, so that neither they nor HBM are full: waves wait for a load one turn ahead in a third of theirs. Join 8: each
// of k picks waits for a load of its list. 24 % fewer instructions in the sums' loop, none of them f64, changed nothing, nor did a threshold
// that the waves of a row share, nor 1536 or 2048 workgroups for 1024 (44, 50 and 48 us). Four rows of 32000 f32
// logits: 7.1 and 5.0 us, two launches and their latencies.
#include "beam.hpp"

namespace bitmm {
namespace attn {
namespace {

constexpr int kWaves = 4;     // of a workgroup that scans
constexpr int kFound = 256;   // logits that a wave holds in LDS
constexpr int kVectors = 2;   // 16-byte pieces of a lane at a time

// A number's place in the order of floats (-0 and 0 alike), larger than 0 for all but NaN.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float float_of(uint32_t order) {
  return __uint_as_float(order & 0x80000000u ? order & 0x7FFFFFFFu : ~order);
}

struct MaxWord {  // of bit patterns as unsigned numbers
  __device__ float operator()(float a, float b) const { return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b))); }
};
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  return __builtin_amdgcn_readfirstlane(__float_as_uint(reduce_lanes<64>(__uint_as_float(v), MaxWord())));
}
// The largest of a wave's 64-bit numbers; `at`: the first lane that has it.
__device__ __forceinline__ uint64_t wave_max(uint64_t v, int& at) {
  const uint32_t hi = wave_max((uint32_t)(v >> 32));
  const bool first = (uint32_t)(v >> 32) == hi;
  const uint32_t lo = wave_max(first ? (uint32_t)v : 0u);
  at = __builtin_ctzll(__ballot(first && (uint32_t)v == lo));
  return (uint64_t)hi << 32 | lo;
}

__device__ __forceinline__ double add_lanes(double v) {
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  return v;
}

// 2^z for z from -1000 to 900.
__device__ __forceinline__ double exp2_f64(double z) {
  const double shifted = z + 0x1.8p52, f = z - (shifted - 0x1.8p52);
  // In vector registers: an instruction takes one scalar constant, and two would have the one moved each time.
  double y = 0x1.fe178300e5507p-17;
  asm("" : "+v"(y));
  y = fma(f, y, 0x1.446a1fe276ad3p-13);
  y = fma(y, f, 0x1.5d8a708963d9cp-10);
  y = fma(y, f, 0x1.3b29dc40cc7e3p-7);
  y = fma(y, f, 0x1.c6b08aaf2d76ap-5);
  y = fma(y, f, 0x1.ebfbe0a4be8e5p-3);
  y = fma(y, f, 0x1.62e42ff11629dp-1);
  y = fma(y, f, 0x1.ffffffffabbc9p-1);
  // the whole part is in the low bits of the shifted number
  return __hiloint2double(__double2hiint(y) + (__double2loint(shifted) << 20), __double2loint(y));
}

constexpr double kLog2eF64 = 1.4426950408889634074;
constexpr float kLowest = -3.402823466e38f;

// A load of 16 bytes from any even address.
typedef u32x4_t Unaligned __attribute__((aligned(2)));

// The values of a 16-byte piece.
template <int TYPE>
struct Piece {
  static constexpr int N = TYPE == kOutF32 ? 4 : 8;
  static constexpr int BYTES = 16 / N;
  static constexpr uint32_t NOTHING = TYPE == kOutF32 ? 0xFF800000u : TYPE == kOutBf16 ? 0xFF80FF80u : 0xFC00FC00u;
  static __device__ __forceinline__ void unpack(u32x4_t raw, float* to) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TYPE == kOutF32)
        to[i] = __uint_as_float(raw[i]);
      else
        unpack_half2<TYPE == kOutBf16 ? 0 : 1>(raw[i], to[2 * i], to[2 * i + 1]);
    }
  }
  static __device__ __forceinline__ float one(const char* at) {
    if constexpr (TYPE == kOutF32)
      return *reinterpret_cast<const float*>(at);
    else
      return half_to_f32<TYPE == kOutBf16 ? 0 : 1>(*reinterpret_cast<const uint16_t*>(at));
  }
};

// What a wave has found.
struct Found {
  uint64_t* list;  // its part of LDS
  int k, lane;
  int n = 0;
  float pass = kLowest;  // logits from here on are looked at: all but -infinity
  uint64_t last = 0;     // and kept if above this: the k-th of those found, once there are k

  // Brings the first k in order. Returns with the pass mark at the k-th, which later ones of a lower
  // token may still beat.
  __device__ __forceinline__ void shrink() {
    __builtin_amdgcn_wave_barrier();
    uint64_t mine[kFound / 64];
    int rank[kFound / 64];
#pragma unroll
    for (int i = 0; i < kFound / 64; ++i) {
      mine[i] = lane + 64 * i < n ? list[lane + 64 * i] : 0;
      rank[i] = 0;
    }
    if (n <= 64) {
      for (int j = 0; j < n; ++j) rank[0] += list[j] > mine[0];
    } else {
      for (int j = 0; j < n; ++j) {
        const uint64_t other = list[j];
#pragma unroll
        for (int i = 0; i < kFound / 64; ++i) rank[i] += other > mine[i];
      }
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < kFound / 64; ++i)
      if (lane + 64 * i < n && rank[i] < k) list[rank[i]] = mine[i];
    __builtin_amdgcn_wave_barrier();
    n = min(n, k);
    if (n == k) {
      const uint64_t kth = list[k - 1];
      const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)kth), hi = __builtin_amdgcn_readfirstlane((uint32_t)(kth >> 32));
      last = (uint64_t)hi << 32 | lo;
      pass = float_of(hi);
    }
  }
  __device__ __forceinline__ void add(uint64_t mask, float x, uint32_t token) {
    const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
    if (mask >> lane & 1) list[n + before] = (uint64_t)order_of(x) << 32 | ~token;
    n += __builtin_popcountll(mask);
  }
  // For tokens in any order and any number of them: there may be no room, and those found may hold a k-th that
  // equals a logit of a lower token.
  __device__ __forceinline__ void add_any(float x, uint32_t token) {
    const uint64_t pair = (uint64_t)order_of(x) << 32 | ~token;
    auto better = [&] { return __ballot(x >= pass && pair > last); };
    uint64_t mask = better();
    if (n + __builtin_popcountll(mask) > kFound) {
      shrink();
      mask = better();
    }
    if (mask) add(mask, x, token);
  }
  // The next tokens are higher than all that were found: of the k-th's equals none comes before it.
  __device__ __forceinline__ void higher_tokens_follow() {
    if (last) pass = float_of((uint32_t)(last >> 32) + 1);
  }
};

template <int TYPE>
__global__ __launch_bounds__(64 * kWaves) void beam_scan_kernel(SelectParams p) {
  using P = Piece<TYPE>;
  constexpr int N = P::N * kVectors;
  __shared__ uint64_t lists[kWaves][kFound];
  __shared__ double sums[kWaves];
  __shared__ float refs[kWaves];
  __shared__ int counts[kWaves];
  const int row = blockIdx.x / p.parts, part = blockIdx.x - row * p.parts;
  const float score = p.scores[row];
  if ((p.finished && p.finished[row]) || score == -INFINITY) return;  // its logits do not matter
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // The row in pieces of 16 bytes from its start on, wherever that lies: rows with the same logits are added up
  // in the same order, so that equal beams have equal totals.
  const char* base = static_cast<const char*>(p.logits) + (int64_t)row * p.row_stride * P::BYTES;
  const int pieces = p.vocab / P::N, tail = p.vocab - pieces * P::N;
  const Unaligned* body = reinterpret_cast<const Unaligned*>(base);
  const int id = part * kWaves + wave;
  const int first = (int)min((int64_t)id * p.each, (int64_t)pieces), end = (int)min((int64_t)(id + 1) * p.each, (int64_t)pieces);

  Found found;
  found.list = lists[wave];
  found.k = p.k;
  found.lane = lane;
  float ref = -INFINITY;     // exponentials are of x - ref
  double ref64 = 0., sum = 0.;
  int positive = 0;          // the largest bit patterns of all, as signed and as unsigned numbers: NaN and
  uint32_t negative = 0;     // infinity lie above all others of their sign, but -infinity above all negative ones

  auto load = [&](int at, u32x4_t* to) {
#pragma unroll
    for (int v = 0; v < kVectors; ++v) {
      const int i = at + 64 * v + lane;
      to[v] = i < end ? __builtin_nontemporal_load(body + i) : u32x4_t{P::NOTHING, P::NOTHING, P::NOTHING, P::NOTHING};
    }
  };
  auto take = [&](const float* x, int n) {
    float most = x[0];
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) {
        most = fmaxf(most, x[i]);
        positive = max(positive, (int)__float_as_uint(x[i]));
        negative = max(negative, __float_as_uint(x[i]));
      }
    if (__any(most > ref + 300.f)) {  // the first ones, and much larger ones
      const float top = fminf(reduce_lanes<64>(most, Max()), -kLowest);
      sum = ref == -INFINITY ? 0. : sum * exp2_f64(fmax((ref64 - (double)top) * kLog2eF64, -1000.));
      ref = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(top)));
      ref64 = (double)ref;
    }
    double a = 0., b = 0.;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) (i & 1 ? b : a) += exp2_f64(fmax(((double)x[i] - ref64) * kLog2eF64, -1000.));
    sum += a + b;
    return most;
  };

  u32x4_t raw[kVectors];
  if (first < end) load(first, raw);
  for (int at = first; at < end; at += 64 * kVectors) {
    float x[N];
#pragma unroll
    for (int v = 0; v < kVectors; ++v) P::unpack(raw[v], x + v * P::N);
    if (at + 64 * kVectors < end) load(at + 64 * kVectors, raw);
    const float most = take(x, N);
    if (at == first) {  // the k-th largest of the lanes' largest, by its upper 16 bits
      const uint32_t key = order_of(most);
      uint32_t t = 0;
#pragma unroll 1
      for (int bit = 31; bit >= 16; --bit)
        if (__builtin_popcountll(__ballot(key >= (t | 1u << bit))) >= p.k) t |= 1u << bit;
      found.pass = fmaxf(float_of(t), kLowest);  // of no number: NaN
    }
    if (__any(most >= found.pass)) {
      uint64_t mask[N];
      int more = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        mask[i] = __ballot(x[i] >= found.pass);
        more += __builtin_popcountll(mask[i]);
      }
      auto token = [&](int i) { return (uint32_t)((at + 64 * (i / P::N) + lane) * P::N + i % P::N); };
      if (found.n + more <= kFound) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (mask[i]) found.add(mask[i], x[i], token(i));
      } else {  // many alike: read again, one after the other
#pragma unroll 1
        for (int i = 0; i < N; ++i) {
          const bool live = at + 64 * (i / P::N) + lane < end;
          found.add_any(live ? P::one(base + (int64_t)token(i) * P::BYTES) : -INFINITY, token(i));
        }
      }
      if (found.n >= p.k + 24 || at == first) found.shrink();
      found.higher_tokens_follow();
    }
  }
  if (id == 0 && tail > 0) {
    const uint32_t token = p.vocab - tail + lane;
    const float x = lane < tail ? P::one(base + (int64_t)token * P::BYTES) : -INFINITY;
    take(&x, 1);
    found.add_any(x, token);
  }
  found.shrink();
  // exponentials of -infinity were 2^-1000: a row of nothing else sums to nothing
  sum = ref == -INFINITY ? 0. : sum;
  if (__any(positive >= 0x7F800000 || negative > 0xFF800000u)) sum = __longlong_as_double(0x7FF8000000000000ll);
  sum = add_lanes(sum);
  if (lane == 0) {
    sums[wave] = sum;
    refs[wave] = ref;
    counts[wave] = found.n;
  }
  __syncthreads();

  // The waves' lists as one: an entry's rank is its own place and how many of the others' come before it.
  uint64_t* out = p.part_top + (int64_t)blockIdx.x * p.k;
  int total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) total += counts[w];
  for (int i = lane; i < counts[wave]; i += 64) {
    const uint64_t pair = lists[wave][i];
    int rank = i;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w == wave) continue;
      int lo = 0, hi = counts[w];
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (lists[w][mid] > pair)
          lo = mid + 1;
        else
          hi = mid;
      }
      rank += lo;
    }
    if (rank < p.k) out[rank] = pair;
  }
  if ((int)threadIdx.x < p.k && (int)threadIdx.x >= total) out[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    float top = refs[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) top = fmaxf(top, refs[w]);
    double all = 0.;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      if (sums[w] != 0.) all += sums[w] * (refs[w] == top ? 1. : exp2_f64(fmax(((double)refs[w] - (double)top) * kLog2eF64, -1000.)));
    p.part_sum[2 * (int64_t)blockIdx.x] = top;
    p.part_sum[2 * (int64_t)blockIdx.x + 1] = all;
  }
}

// An f64's place in the order of numbers, larger than 0; not for NaN.
__device__ __forceinline__ uint64_t order_of(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v + 0.);
  return u >> 63 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ double double_of(uint64_t order) {
  return __longlong_as_double((long long)(order >> 63 ? order & ~(1ull << 63) : ~order));
}

__global__ __launch_bounds__(512) void beam_merge_kernel(SelectParams p) {
  extern __shared__ uint64_t totals[];  // [beams][k], then the tokens
  int* tokens = reinterpret_cast<int*>(totals + p.beams * p.k);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int64_t row0 = (int64_t)blockIdx.x * p.beams;
  for (int b = wave; b < p.beams; b += waves) {
    const int64_t row = row0 + b;
    const float score = p.scores[row];
    const bool done = p.finished && p.finished[row];
    uint64_t* mine = totals + b * p.k;
    if (lane < p.k) mine[lane] = 0;
    const bool odd = score != score || score == INFINITY;
    bool bad = odd;
    if (!odd && !done && score != -INFINITY) {
      // the parts' sums, each of exponentials of x - ref
      const double ref = lane < p.parts ? p.part_sum[2 * (row * p.parts + lane)] : -INFINITY;
      const double part = lane < p.parts ? p.part_sum[2 * (row * p.parts + lane) + 1] : 0.;
      const double top = (double)reduce_lanes<64>((float)ref, Max());
      const double sum = add_lanes(part == 0. ? 0. : part * exp2_f64(fmax((ref - top) * kLog2eF64, -1000.)));
      bad = sum != sum;
      const double log_sum = log(sum);
      if (!bad && sum > 0.) {
        // The parts' lists are in order: the largest of their first ones, k times.
        const uint64_t* list = p.part_top + (row * p.parts + min(lane, p.parts - 1)) * p.k;
        uint64_t now = lane < p.parts ? list[0] : 0, next = lane < p.parts && p.k > 1 ? list[1] : 0;
        int taken = 0;
        for (int i = 0; i < p.k; ++i) {
          int at;
          const uint64_t best = wave_max(now, at);
          if (best == 0) break;
          if (lane == at) {
            mine[i] = order_of((double)score + (((double)float_of((uint32_t)(best >> 32)) - top) - log_sum));
            tokens[b * p.k + i] = (int)~(uint32_t)best;
            ++taken;
            now = next;
            next = taken + 1 < p.k ? list[taken + 1] : 0;
          }
        }
      }
    } else if (!odd && done && score != -INFINITY && p.end_token >= 0 && p.end_token < p.vocab && lane == 0) {
      mine[0] = order_of((double)score);
      tokens[b * p.k] = p.end_token;
    }
    if (bad && p.status && lane == 0) *p.status = 1;
  }
  __syncthreads();
  if (wave != 0) return;
  // The same over the rows' lists, a lane each; equal totals go to the lowest lane.
  const bool done = lane < p.beams && p.finished && p.finished[row0 + lane];
  const uint64_t doners = __ballot(done);
  uint64_t now = lane < p.beams ? totals[lane * p.k] : 0, mine = 0;
  int taken = 0, parent = -1, token = -1;
  for (int i = 0; i < p.k; ++i) {
    int at;
    const uint64_t best = wave_max(now, at);
    if (best == 0) break;
    const int place = __builtin_amdgcn_readlane(taken, at);
    if (lane == i) {
      mine = best;
      parent = at;
      token = tokens[at * p.k + place];
    }
    if (lane == at) {
      ++taken;
      now = taken < p.k ? totals[lane * p.k + taken] : 0;
    }
  }
  if (lane >= p.k) return;
  const int64_t to = (int64_t)blockIdx.x * p.k + lane;
  p.scores_out[to] = mine ? (float)double_of(mine) : -INFINITY;
  p.parents[to] = parent;
  p.tokens[to] = token;
  if (p.finished_out) p.finished_out[to] = parent >= 0 && ((doners >> parent & 1) || token == p.end_token);
}

template <int TYPE>
hipError_t scan(const SelectParams& p, int64_t workgroups, hipStream_t stream) {
  const dim3 grid((unsigned)workgroups), block(64 * kWaves);
  hipLaunchKernelGGL(beam_scan_kernel<TYPE>, grid, block, 0, stream, p);
  launch_log(grid, block, kWaves * (kFound * 8 + 16), "beam_scan_kernel<%d>", TYPE);
  return hipGetLastError();
}

}  // namespace

SelectPlan plan_select(int64_t rows, int64_t vocab, bitmm_out type) {
  const int64_t pieces = (vocab * (type == BITMM_OUT_F32 ? 4 : 2) + 15) / 16, step = 64 * kVectors;
  const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(64, 1024 / std::max<int64_t>(rows, 1)));
  SelectPlan plan;
  const int64_t each = (pieces + parts * kWaves - 1) / (parts * kWaves);
  plan.each = (int)((each + step - 1) / step * step);
  plan.parts = (int)std::max<int64_t>(1, (pieces + (int64_t)plan.each * kWaves - 1) / ((int64_t)plan.each * kWaves));
  return plan;
}

hipError_t launch_beam_select(SelectParams p, const SelectPlan& plan, int64_t groups, bitmm_out type, hipStream_t stream) {
  p.parts = plan.parts;
  p.each = plan.each;
  const int64_t workgroups = groups * p.beams * plan.parts;
  const hipError_t err = type == BITMM_OUT_F32    ? scan<kOutF32>(p, workgroups, stream)
                         : type == BITMM_OUT_BF16 ? scan<kOutBf16>(p, workgroups, stream)
                                                  : scan<kOutF16>(p, workgroups, stream);
  if (err != hipSuccess) return err;
  const dim3 grid((unsigned)groups), block(64 * std::min(8, p.beams));
  const size_t lds = (size_t)p.beams * p.k * 12;
  hipLaunchKernelGGL(beam_merge_kernel, grid, block, lds, stream, p);
  launch_log(grid, block, lds, "beam_merge_kernel");
  return hipGetLastError();
}

}  // namespace attn
}  // namespace bitmm
