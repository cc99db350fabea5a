// Attention of groups of sequences that share their first tokens.
//
// The tokens that a group shares are gone over once for all its queries, as if these were one sequence's
// whose every query sees every token; then each sequence's own tokens as in attention.hip. With both passes'
// references m, sums l and outputs o (of exponents to the base 2, not normalised) a row is
//   sum_s o_s 2^(m_s - m) / sum_s l_s 2^(m_s - m),  m = max_s m_s
// over the parts s of both, added up in f32: by the second pass where it ends a row, else, where a row's own tokens
// are split, by attention_join_shared_kernel.
//
// What bounds it. Few beams: latency, one chain of it in one launch where tokens are few (12.2 us for four beams after
// 573 tokens, 9.6 of which attention of one sequence takes). Eight ragged groups of four beams after up to 4096: 21.6 us
// for the shared tokens, three steps a wave of the longest group behind a chain of loads (groups, rows, pages, codes); a
// short group has as many parts as a long one, and 20 rows are a tile of 16 and one of 4, which goes over all again. Then
// 11.1 for the own ones. 64 samples of 32768 tokens, 320 query rows a kv head: 82 to 84 us, of which 42 are products and
// softmax (matrix cores busy in 20 % of the cycles), 9 the tiles' expansion, 9 the parts' stores and 12 begin and end;
// some ten are not accounted for. Then 20.5 for the own tokens, ten parts of each row taken in. Two tiles of 16 rows to a
// wave, which would share its expanded values, were not kept (registers leave two waves a SIMD; with three they spill);
// nor did workgroups of four waves, two a CU, win for many rows (88 us against 87), nor fewer parts for a last tile
// with few rows (90 against 91).
#include "attention_rows.hpp"

namespace bitmm {
namespace attn {
namespace {

// Joins a row's parts of both passes, as attention_join_kernel does those of one.
template <int D>
__global__ __launch_bounds__(256) void attention_join_shared_kernel(SharedParams both) {
  constexpr int TPR = D / 4, GROUPS = 256 / TPR;
  __shared__ f32x4_t sums[GROUPS][TPR];
  __shared__ float part_l[GROUPS];
  const AttentionParams &p = both.own, &prefix = both.prefix;
  const int unit = blockIdx.x / p.tail_rows, r = blockIdx.x - unit * p.tail_rows;
  const int b = unit / p.cache.kv_heads, head = unit - b * p.cache.kv_heads;
  const int lane = threadIdx.x & 63;
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  // The row's parts: every `step`-th from `first` on.
  Extent ex;
  int first = b, step = p.B, parts = p.splits;
  if (p.balanced) {
    const Shares shares(p, lane, blockIdx.x == 0);
    const Share mine = shares.of_sequence(b);
    ex = shares.extent(b);
    first = mine.first;
    step = 1;
    parts = mine.count;
  } else {
    ex = extent_of(p, b, threadIdx.x == 0);
  }
  if (r >= ex.rows) return;
  const int64_t row = part_row(p, first, head, r), all = part_row(p, step, 0, 0);
  const SharedRows shared(prefix, b, lane);
  const int64_t shared_row = shared.row(prefix, ex.q0, r);
  const int shared_parts = shared.parts(prefix, shared_row);
  if (shared_parts < 0) {  // past the bound of its group's queries
    if (p.status && threadIdx.x == 0) *p.status = 1;
    return;
  }
  // A part's place among those of its pass.
  auto at = [&](int s) { return s < parts ? s * all + row : prefix_row(prefix, s - parts, shared.group, head, (int)shared_row); };
  const int count = parts + shared_parts;
  float mt = neg_inf();
  for (int s = lane; s < count; s += 64) mt = fmaxf(mt, (s < parts ? p : prefix).part_ml[2 * at(s)]);
  mt = reduce_lanes<64>(mt, Max());
  f32x4_t y = {0.f, 0.f, 0.f, 0.f};
  float lt = 0.f;
#pragma unroll 4
  for (int s = grp; s < count; s += GROUPS) {
    const AttentionParams& from = s < parts ? p : prefix;
    const float2 part = *reinterpret_cast<const float2*>(from.part_ml + 2 * at(s));
    const f32x4_t o = *reinterpret_cast<const f32x4_t*>(from.part_o + at(s) * D + 4 * t);
    if (part.y == 0.f) continue;  // saw nothing
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
  const RowOf out_row(p, head, r);
  if (p.lse && t == 0) p.lse[(int64_t)(ex.q0 + out_row.i) * p.q_heads + out_row.head] = kLn2 * (mt + __builtin_amdgcn_logf(lt));
  store4(p, (int64_t)(ex.q0 + out_row.i) * p.out_stride + (int64_t)out_row.head * D + 4 * t, y[0] * inv, y[1] * inv, y[2] * inv,
         y[3] * inv);
}

void take(AttentionParams& p, const AttentionPlan& plan) {
  p.row_tiles = plan.row_tiles;
  p.tail_tiles = plan.tail_tiles;
  p.tail_rows = plan.tail_rows;
  p.splits = plan.splits;
  p.balanced = plan.balanced;
}

template <int D>
void launch_join(const SharedParams& p, dim3 grid, hipStream_t stream) {
  hipLaunchKernelGGL(attention_join_shared_kernel<D>, grid, dim3(256), 0, stream, p);
  launch_log(grid, dim3(256), 256 * 16 + 256 / (D / 4) * 4, "attention_join_shared_kernel<%d>", D);
}

}  // namespace

SharedPlan plan_attention_shared(int64_t groups, int64_t B, int64_t max_group_q, int64_t max_prefix, int64_t max_q,
                                 int64_t max_kv, int64_t q_heads, int64_t kv_heads, int64_t head_dim) {
  SharedPlan plan = {};
  plan.own = plan_attention(B, max_q, max_kv, q_heads, kv_heads, head_dim, 0, 0);
  if (groups == 0 || max_group_q == 0) return plan;
  // Where all sequences' workgroups run at once, two a CU, and tokens are few, each goes over the shared ones by itself:
  // one launch, one chain of latencies. Calls in us, this against two launches, 40 heads over 8 of 128 dims: four beams
  // after 573 tokens 11.7 and 15.9, after 1200 17.4 and 18.4, after 1600 21.0 and 19.8; 32 beams after 600 13.6 and 21.3;
  // 16 groups of four after 600 19.6 and 24.8, after 1200 26.8 and 29.4, after 1600 32.7 and 32.1; 20 groups after 600
  // 26.9 and 25.7. 16 heads over 4 of 256 dims, one group after 900 22.2 and 21.7, after 1200 24.9 and 22.9.
  const int64_t row_tiles = (max_q * (q_heads / kv_heads) + kRows - 1) / kRows;
  plan.both = B * kv_heads * row_tiles <= 512 && max_prefix <= (head_dim == 256 ? 1024 : 1280) && max_kv <= 1024;
  if (plan.both) {
    plan.own = {};
    plan.own.row_tiles = (int)row_tiles;
    plan.own.splits = 1;
  } else {
    plan.prefix = plan_attention(groups, max_group_q, max_prefix, q_heads, kv_heads, head_dim, 0, 0);
    plan.prefix.balanced = false;
    if (!plan.prefix.tiles) {
      // Parts cost no launch here, and are joined by as many waves: four waves and two steps each, until the
      // workgroups fill the chip (four beams after 573 tokens: 18.4 us unsplit, 16 in eight parts).
      AttentionPlan& few = plan.prefix;
      few.waves = 4;
      const int64_t fill = (head_dim == 256 ? 2 : 4) * 256, tiles = groups * kv_heads * few.row_tiles;
      few.splits = (int)std::max<int64_t>(1, std::min<int64_t>({fill / tiles, (max_prefix + 63) / 64, 128}));
      few.tail_tiles = few.splits > 1 ? few.row_tiles : 0;
      few.tail_rows = few.splits > 1 ? (int)(max_group_q * (q_heads / kv_heads)) : 0;
    }
  }
  return plan;
}

hipError_t launch_kv_attention_shared(SharedParams p, const SharedPlan& plan, int dtype, hipStream_t stream) {
  take(p.prefix, plan.prefix);
  take(p.own, plan.own);
  const Cache& c = p.own.cache;
  if (plan.both)
    return launch_attention_rows<kBoth>(p, c, (unsigned)((int64_t)p.own.B * c.kv_heads * p.own.row_tiles), 8, dtype, stream);
  if (plan.prefix.row_tiles > 0) {
    const unsigned n = (unsigned)plan.prefix.workgroups((int64_t)p.prefix.B * c.kv_heads);
    const hipError_t err = plan.prefix.tiles ? launch_attention_tiles_prefix(p.prefix, plan.prefix.rows_each, n, dtype, stream)
                                             : launch_attention_rows<kPrefix>(p.prefix, c, n, plan.prefix.waves, dtype, stream);
    if (err != hipSuccess) return err;
  }
  const int64_t groups = (int64_t)p.own.B * c.kv_heads;
  const unsigned n = (unsigned)plan.own.workgroups(groups);
  const hipError_t err = plan.own.tiles ? launch_attention_tiles_own(p, plan.own.rows_each, n, dtype, stream)
                                        : launch_attention_rows<kOwn>(p, c, n, plan.own.waves, dtype, stream);
  if (err != hipSuccess || plan.own.splits == 1) return err;
  const dim3 grid((unsigned)(groups * plan.own.tail_rows));
  c.head_dim == 64 ? launch_join<64>(p, grid, stream) : c.head_dim == 128 ? launch_join<128>(p, grid, stream) : launch_join<256>(p, grid, stream);
  return hipGetLastError();
}

}  // namespace attn
}  // namespace bitmm
