// Attention over the 4-bit cache: how a call is cut up, and the join of partial results. The kernel for few
// query rows is in attention_rows.hpp, that for many in attention_tiles.hpp.
#include "attention_rows.hpp"

namespace bitmm {
namespace attn {
namespace {

// Joins the partial results of the splits. A workgroup takes one query row: 256 / (D / 4)
// groups of threads go round its splits, four dims a thread, and are added up in LDS.
template <int D>
__global__ __launch_bounds__(256) void attention_join_kernel(AttentionParams p) {
  constexpr int TPR = D / 4, GROUPS = 256 / TPR;
  __shared__ f32x4_t sums[GROUPS][TPR];
  __shared__ float part_l[GROUPS];
  const int group = blockIdx.x / p.tail_rows, r = blockIdx.x - group * p.tail_rows;
  const int b = group / p.cache.kv_heads, head = group - b * p.cache.kv_heads;
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
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  float mt = neg_inf();
  for (int s = lane; s < parts; s += 64) mt = fmaxf(mt, ml[s * all + row].x);
  mt = reduce_lanes<64>(mt, Max());
  f32x4_t y = {0.f, 0.f, 0.f, 0.f};
  float lt = 0.f;
#pragma unroll 4
  for (int s = grp; s < parts; s += GROUPS) {
    const int64_t at = s * all + row;
    const float2 part = ml[at];
    const f32x4_t o = *reinterpret_cast<const f32x4_t*>(p.part_o + at * D + 4 * t);
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

}  // namespace

AttentionPlan plan_attention(int64_t B, int64_t max_q, int64_t max_kv, int64_t q_heads,
                             int64_t kv_heads, int64_t head_dim, int64_t window, int64_t sinks) {
  constexpr int64_t CUS = 256;
  AttentionPlan plan;
  const int64_t rows = max_q * (q_heads / kv_heads), groups = B * kv_heads;
  const int64_t span = window > 0 ? std::min(max_kv, window + sinks + max_q) : max_kv;
  const int64_t tiles16 = (rows + kRows - 1) / kRows, steps = (span + kStep - 1) / kStep;
  // The kernel for few rows starts and ends sooner, and spreads over more CUs; tiles of many rows
  // read and expand the cache once for all of them. Up to 64 rows, or 64 steps for each CU, the
  // first, above that the second. Both sides, in us, for the last n of m tokens of one sequence, 40 heads
  // over 8 of 128 dims: 64 of 600 11 and 24, 300 of 600 19 and 24, 48 of 4096 28 and 31, 8 sequences' 12 of
  // 2048 31 and 31, 32 sequences' 4 of 2048 45 and 54; then 64 of 4096 33 and 33, 600 of 600 40 and 25, 160 of
  // 4096 63 and 47, 32 sequences' 16 of 2048 112 and 57. Where 49 to 64 rows of many sequences make four row
  // tiles, the rule takes the slower: 32 sequences' 12 of 2048 63 and 57.
  plan.tiles = rows > 64 && (double)groups * tiles16 * steps > 64 * CUS;
  plan.waves = 0;
  int64_t rows_each, fill, most;  // fill: workgroups at a time; most: parts of a tile's tokens
  if (plan.tiles) {
    // 256 rows a workgroup where that still gives every CU one, else half of them, with two waves
    // for each 32 rows (a prompt of 600 tokens, 40 heads over 8: 25 us against 30; always half, at 64 dims:
    // ragged windowed chunks 150 against 102).
    rows_each = head_dim == 256 || groups * ((rows + 255) / 256) < CUS ? 128 : 256;
    fill = CUS;
    // Over short spans the join costs more than the split saves (400 of 1600 tokens: 56 us against 43).
    most = span < 2048 ? 1 : span / 512;
  } else {
    // Few short sequences, as many workgroups as the chip holds at a time: eight waves each and no
    // joining launch (573 tokens, 8 kv heads: 9.5 us against 10.2 of four waves and the join; 160 of 600
    // tokens: 16 against 27). Otherwise four waves, and splits until the workgroups fill the chip once,
    // as many as registers and LDS let a CU hold: at twice as many the second half waits (decode
    // of 64 sequences, head dim 256: 60 us against 51). A wave has at least one step.
    plan.waves = groups * tiles16 <= (head_dim == 256 ? CUS : 2 * CUS) && steps <= 32 ? 8 : 4;
    rows_each = kRows;
    fill = plan.waves == 8 ? 1 : head_dim == 256 ? 2 * CUS : 4 * CUS;
    most = std::max<int64_t>(1, steps / plan.waves);
  }
  plan.rows_each = (int)rows_each;
  plan.row_tiles = (int)((rows + rows_each - 1) / rows_each);
  // Whole rounds of workgroups run as they are; the tiles left over for the last, partial round
  // are split so that they fill it (4096 of 16384 tokens: 1.34 -> 1.24 ms).
  const int64_t whole = std::min<int64_t>(plan.row_tiles, groups * plan.row_tiles / fill * fill / groups);
  plan.tail_tiles = (int)(plan.row_tiles - whole);
  plan.splits = plan.tail_tiles > 0 ? (int)std::min<int64_t>({fill / (groups * plan.tail_tiles), most, 128}) : 1;
  if (plan.splits <= 1) {
    plan.splits = 1;
    plan.tail_tiles = 0;
  }
  // One row tile of each of several sequences: the workgroups are shared out by what each has to
  // do, which the kernels find from the lengths, join included, for 1 us. 32 sequences of 512
  // tokens but one of 32768: 103 us as equal splits, 28 so; of 1024 to 4096: 38 against 34; all of
  // 4096: 41 against 42. A wave looks at 64 sequences, with step counts that add up in 31 bits.
  plan.balanced = !plan.tiles && plan.row_tiles == 1 && plan.splits > 1 && B > 1 && B <= 64 &&
                  B * (max_kv / kStep + 2) <= INT32_MAX;
  plan.tail_rows = (int)std::min<int64_t>(rows, plan.tail_tiles * rows_each);
  return plan;
}

hipError_t launch_kv_attention(AttentionParams p, const AttentionPlan& plan, int dtype,
                               hipStream_t stream) {
  p.row_tiles = plan.row_tiles;
  p.tail_tiles = plan.tail_tiles;
  p.tail_rows = plan.tail_rows;
  p.splits = plan.splits;
  p.balanced = plan.balanced;
  const int D = p.cache.head_dim;
  const int64_t groups = (int64_t)p.B * p.cache.kv_heads;
  const unsigned n = (unsigned)plan.workgroups(groups);
  hipError_t err = plan.tiles ? launch_attention_tiles(p, plan.rows_each, n, dtype, stream)
                              : launch_attention_rows<kAlone>(p, p.cache, n, plan.waves, dtype, stream);
  if (err != hipSuccess || plan.splits == 1) return err;
  const dim3 grid((unsigned)(groups * plan.tail_rows)), block(256);
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
