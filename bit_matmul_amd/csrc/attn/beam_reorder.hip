// Reordering of the cached states of beams after a selection. Rows of the page table follow their parents, so
// that full pages are shared by all that descend from them; of rows whose last page is partly filled and the same,
// the first of those with the most tokens on it keeps it, if it is of their pool, and the others get pages of their own
// with a copy of its tokens, in every layer. So a row that gets no room keeps what it has: nothing is stored where it,
// or a longer row, holds a token.
//
// Two kernels. beam_plan_kernel, a workgroup a group of beams: the new table and lengths, which pages of the group's
// pool no row holds (a bit each in LDS), the pages handed out, the slots of the next tokens and a list of copies.
// beam_copy_kernel, a workgroup a row, layer and side: the copies.
//
// What bounds it: latency. Four beams through 40 layers of 8 heads of 128 dims: 4.8 us for the plan, whose loads of
// parents, lengths and table wait for one another, 6.7 for the copies of 3 MB. 16 groups of eight beams through 24
// layers: 7.2 and 16.9 us for 52 MB, 3.1 TB/s (a copy 5.2). Source and target of a copy lie in one buffer, so the compiler
// lets no load pass the store before it, unrolled or not: a wave has one piece of 1 KB in flight, and waits in 82 % of its
// cycles.
#include "beam.hpp"

namespace bitmm {
namespace attn {
namespace {

constexpr int kPlanThreads = 256;
constexpr int kEntries = 4;  // table entries of a thread at a time

// A row's copy: `tokens` slots of page src to page dst; none where that is 0.
struct Copy {
  int src, dst, tokens, unused;
};

__global__ __launch_bounds__(kPlanThreads) void beam_plan_kernel(ReorderParams p) {
  extern __shared__ uint32_t held_pages[];  // a bit for each page of the group's pool
  __shared__ int parent[64], tokens[64], last_page[64], handed[64];
  const int tid = threadIdx.x, g = blockIdx.x, beams = p.beams;
  const int64_t row0 = (int64_t)g * beams;
  const int size = 1 << p.page_shift, base = p.first_page + g * p.pages_per_group;
  const int words = (p.pages_per_group + 31) / 32;
  bool wrong = false;
  if (tid < 64) {
    int from = -1, n = 0;
    if (tid < beams) {
      from = p.parents[row0 + tid];
      if (from < -1 || from >= beams) {
        wrong = true;
        from = -1;
      }
      if (from >= 0) {
        const int len = p.lens[row0 + from];
        const int64_t room = p.pages_per_seq << p.page_shift;
        n = (int)min((int64_t)max(len, 0), room);
        wrong = wrong || n != len;
      }
    }
    parent[tid] = from;
    tokens[tid] = n;
    last_page[tid] = -1;
  }
  for (int i = tid; i < words; i += kPlanThreads) held_pages[i] = 0;
  __syncthreads();

  // Columns of the table, as many at a time as the threads have entries for; a column's entries are all read
  // before any is written, since the new table may be the old one.
  int columns = 0;
  for (int j = 0; j < beams; ++j) columns = max(columns, (tokens[j] + size - 1) >> p.page_shift);
  if (p.table_out != p.table) columns = (int)p.pages_per_seq;
  const int at_once = kPlanThreads * kEntries / beams;
  for (int c0 = 0; c0 < columns; c0 += at_once) {
    int value[kEntries];
    int64_t to[kEntries];
#pragma unroll
    for (int e = 0; e < kEntries; ++e) {
      const int i = e * kPlanThreads + tid, j = i / at_once, c = c0 + i - j * at_once;
      to[e] = -1;
      if (j >= beams || c >= columns) continue;
      const bool held = c << p.page_shift < tokens[j];  // else the row's own entry, which nobody reads
      const int64_t from = held ? row0 + parent[j] : row0 + j;
      value[e] = p.table[from * p.pages_per_seq + c];
      if (held || p.table_out != p.table) to[e] = (row0 + j) * p.pages_per_seq + c;
      if (!held) continue;
      if (c == (tokens[j] - 1) >> p.page_shift && tokens[j] & (size - 1)) last_page[j] = value[e];
      const uint32_t in_pool = (uint32_t)(value[e] - base);
      if (in_pool < (uint32_t)p.pages_per_group) atomicOr(&held_pages[in_pool >> 5], 1u << (in_pool & 31));
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kEntries; ++e)
      if (to[e] >= 0) p.table_out[to[e]] = value[e];
  }
  __syncthreads();
  if (tid >= 64) return;

  // A lane a row. Rows that need a page: those without a partly filled one, and those whose is also that of a row with
  // more tokens on it (the other once got no room) or of an earlier one with as many, or is full in a longer row, or is
  // not the pool's: a prompt's pages are not written.
  const int n = tokens[tid], column = n >> p.page_shift, part = n & (size - 1), mine = last_page[tid];
  const bool live = parent[tid] >= 0;
  bool again = false;
  int longest = 0;
  for (int j = 0; j < beams; ++j) {
    const int there = tokens[j] & (size - 1);
    again = again || (there && last_page[j] == mine && (there > part || (there == part && j < tid)));
    longest = max(longest, tokens[j]);
  }
  const bool inside = (uint32_t)mine < (uint32_t)p.num_pages;
  again = again || (inside && (uint32_t)(mine - base) >= (uint32_t)p.pages_per_group);
  if (part && inside && longest >> p.page_shift > column)  // mostly the rows are as long as each other
    for (int j = 0; j < beams; ++j)
      if (!again && tokens[j] >> p.page_shift > column) again = p.table_out[(row0 + j) * p.pages_per_seq + column] == mine;
  const bool wants = live && (part == 0 || again) && column < p.pages_per_seq;
  const uint64_t all = __ballot(wants);
  const int want = __builtin_popcountll(all), place = __builtin_popcountll(all & ((1ull << tid) - 1));
  int found = 0;
  for (int w0 = 0; w0 < words && found < want; w0 += 64) {
    const int w = w0 + tid;
    uint32_t open = w < words ? ~held_pages[w] : 0;
    if (w == words - 1 && p.pages_per_group & 31) open &= (1u << (p.pages_per_group & 31)) - 1;
    const int count = __builtin_popcount(open);
    int before = count;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int other = __shfl_up(before, d);
      if (tid >= d) before += other;
    }
    const int sum = __shfl(before, 63);
    before += found - count;
    while (open && before < want) {
      handed[before++] = base + 32 * w + __builtin_ctz(open);
      open &= open - 1;
    }
    found += sum;
  }
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_s_waitcnt(0);
  if (tid < beams) {
    const int64_t row = row0 + tid;
    Copy copy = {0, 0, 0, 0};
    int page = -1;
    if (wants && place < found) {
      page = handed[place];
      if (part > 0 && inside) copy = {mine, page, part, 0};
      if (part > 0 && !inside) wrong = true;  // its tokens are lost already
      p.table_out[row * p.pages_per_seq + column] = page;
    } else if (live && part > 0 && !again && inside) {
      page = mine;
    }
    if (live && page < 0) wrong = true;
    p.lens_out[row] = n + (page >= 0);
    p.slots[row] = page >= 0 ? (int64_t)page * size + part : -1;
    reinterpret_cast<Copy*>(p.copies)[row] = copy;
  }
  if (wrong && p.status) *p.status = 1;
}

__global__ __launch_bounds__(256) void beam_copy_kernel(ReorderParams p, ReorderLayers layers) {
  const Copy copy = reinterpret_cast<const Copy*>(p.copies)[blockIdx.x];
  if (copy.tokens == 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t* codes = layers.at[blockIdx.y].side[blockIdx.z].codes;
  uint32_t* scales = layers.at[blockIdx.y].side[blockIdx.z].scales;
  const int pieces = copy.tokens * p.code_pieces, pairs = copy.tokens * p.groups_of_head;  // of a head
  for (int h = wave; h < p.kv_heads; h += 4) {
    const int64_t src = ((int64_t)copy.src * p.kv_heads + h) << p.page_shift, dst = ((int64_t)copy.dst * p.kv_heads + h) << p.page_shift;
    const u32x4_t* from = reinterpret_cast<const u32x4_t*>(codes) + src * p.code_pieces;
    u32x4_t* to = reinterpret_cast<u32x4_t*>(codes) + dst * p.code_pieces;
#pragma unroll 4
    for (int i = lane; i < pieces; i += 64) to[i] = from[i];
    const uint32_t* pairs_from = scales + src * p.groups_of_head;
    uint32_t* pairs_to = scales + dst * p.groups_of_head;
#pragma unroll 4
    for (int i = lane; i < pairs; i += 64) pairs_to[i] = pairs_from[i];
  }
}

}  // namespace

hipError_t launch_beam_reorder(const ReorderParams& p, const bitmm_kv_cache* caches, int64_t layers, int64_t groups,
                               hipStream_t stream) {
  const size_t lds = (size_t)(p.pages_per_group + 31) / 32 * 4;
  hipLaunchKernelGGL(beam_plan_kernel, dim3((unsigned)groups), dim3(kPlanThreads), lds, stream, p);
  launch_log(dim3((unsigned)groups), dim3(kPlanThreads), lds + 4 * 64 * 4, "beam_plan_kernel");
  hipError_t err = hipGetLastError();
  for (int64_t first = 0; err == hipSuccess && first < layers; first += ReorderLayers::MOST) {
    const int n = (int)std::min<int64_t>(ReorderLayers::MOST, layers - first);
    ReorderLayers some;
    for (int i = 0; i < n; ++i) {
      const bitmm_kv_cache& c = caches[first + i];
      some.at[i].side[0] = {static_cast<uint32_t*>(c.k_codes), static_cast<uint32_t*>(c.k_scales)};
      some.at[i].side[1] = {static_cast<uint32_t*>(c.v_codes), static_cast<uint32_t*>(c.v_scales)};
    }
    const dim3 grid((unsigned)(groups * p.beams), n, 2);
    hipLaunchKernelGGL(beam_copy_kernel, grid, dim3(256), 0, stream, p, some);
    launch_log(grid, dim3(256), 0, "beam_copy_kernel");
    err = hipGetLastError();
  }
  return err;
}

}  // namespace attn
}  // namespace bitmm
