// C ABI of include/bitmm_beam.h: argument validation and dispatch, as in attn_api.cpp.
#include "bitmm_beam.h"

#include "beam.hpp"
#include "checks.hpp"

using namespace bitmm::attn;

namespace {

// A launch's threads are counted in 32 bits, and a row takes 256 at least.
bool beam_rows_ok(int64_t groups, int64_t beams) {
  return groups >= 0 && beams >= 1 && beams <= 64 && groups <= (1 << 22) / beams;
}

bool select_sizes_ok(int64_t groups, int64_t beams, int64_t vocab, int64_t k) {
  return beam_rows_ok(groups, beams) && vocab >= 1 && vocab <= 1 << 30 && k >= 1 && k <= 64;
}

bool shared_sizes_ok(int64_t T, int64_t B, int64_t groups, int64_t max_group_q, int64_t max_prefix, int64_t max_q,
                     int64_t max_kv, int64_t q_heads, int64_t kv_heads) {
  return attention_sizes_ok(T, B, max_q, max_kv, q_heads, kv_heads, 0, 0) &&
         attention_sizes_ok(T, groups, max_group_q, max_prefix, q_heads, kv_heads, 0, 0);
}

// Rows of partial results: a first part of each over the shared tokens, the others of those that are split, and
// the parts of split rows over the own tokens.
struct PartRows {
  int64_t prefix, own;
};
PartRows part_rows(const SharedPlan& plan, int64_t B, int64_t groups, int64_t max_group_q, int64_t q_heads, int64_t kv_heads) {
  if (plan.both) return {0, 0};
  return {groups * kv_heads * (max_group_q * (q_heads / kv_heads) + (int64_t)std::max(plan.prefix.splits - 1, 0) * plan.prefix.tail_rows),
          plan.own.splits > 1 ? (int64_t)plan.own.splits * B * kv_heads * plan.own.tail_rows : 0};
}

}  // namespace

extern "C" {

bitmm_status bitmm_qk_norm_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                       const void* v, int64_t v_stride, const void* q_weight,
                                       const void* k_weight, const int32_t* positions,
                                       const float* inv_freq, void* q_out, int64_t q_out_stride,
                                       const int64_t* slots, const bitmm_kv_cache* cache, int64_t T,
                                       int64_t q_heads, int64_t rot_dim, int interleaved, float eps,
                                       float weight_offset, float rope_scale, bitmm_dtype dtype,
                                       uint32_t* status, void* stream) {
  try {
    bitmm::launch_log_begin();
    bitmm_status st = check_cache(cache);
    if (st != BITMM_OK) return st;
    if (!dtype_ok(dtype)) return BITMM_ERR_UNSUPPORTED;
    const int64_t D = cache->head_dim, kv_heads = cache->kv_heads;
    if (!fits_int(T) || !fits_int(q_heads)) return BITMM_ERR_SHAPE;
    if (rot_dim < 0 || rot_dim > D || rot_dim % 8 != 0) return BITMM_ERR_SHAPE;
    if (T > 1 << 24 || T * (q_heads + kv_heads) >= (int64_t)1 << 30) return BITMM_ERR_SHAPE;
    if (T == 0) return BITMM_OK;
    if (q_heads > 0) {
      if ((st = check_rows(q, q_stride, q_heads, D)) != BITMM_OK) return st;
      if ((st = check_rows(q_out, q_out_stride, q_heads, D)) != BITMM_OK) return st;
    }
    if ((st = check_rows(k, k_stride, kv_heads, D)) != BITMM_OK) return st;
    if ((st = check_rows(v, v_stride, kv_heads, D)) != BITMM_OK) return st;
    if (!slots || (rot_dim > 0 && (!positions || !inv_freq))) return BITMM_ERR_NULL;
    if (!aligned(q_weight, 2) || !aligned(k_weight, 2) || !aligned(positions, 4) || !aligned(inv_freq, 4) ||
        !aligned(slots, 8) || !aligned(status, 4))
      return BITMM_ERR_ALIGN;
    if ((st = device_check()) != BITMM_OK) return st;
    RopeAppendParams p = {};
    p.rope.q = static_cast<const uint16_t*>(q);
    p.rope.k = static_cast<const uint16_t*>(k);
    p.rope.q_weight = static_cast<const uint16_t*>(q_weight);
    p.rope.k_weight = static_cast<const uint16_t*>(k_weight);
    p.rope.positions = positions;
    p.rope.inv_freq = inv_freq;
    p.rope.q_out = static_cast<uint16_t*>(q_out);
    p.rope.q_stride = q_stride;
    p.rope.k_stride = k_stride;
    p.rope.q_out_stride = q_out_stride;
    p.rope.T = (int)T;
    p.rope.q_heads = (int)q_heads;
    p.rope.rot_dim = (int)rot_dim;
    p.rope.eps = eps;
    p.rope.weight_offset = weight_offset;
    p.rope.rope_scale = rope_scale;
    p.v = static_cast<const uint16_t*>(v);
    p.v_stride = v_stride;
    p.slots = slots;
    p.cache = view(cache);
    p.status = status;
    return launched(launch_qk_norm_rope_append(p, interleaved != 0, (int)dtype, static_cast<hipStream_t>(stream)));
  } catch (...) {
    return BITMM_ERR_LAUNCH;
  }
}

size_t bitmm_beam_select_workspace_bytes(int64_t groups, int64_t beams, int64_t vocab, int64_t k, bitmm_out logits_type) {
  if (!select_sizes_ok(groups, beams, vocab, k) || groups == 0) return 0;
  const SelectPlan plan = plan_select(groups * beams, vocab, logits_type);
  return (size_t)(groups * beams) * plan.parts * (16 + 8 * (size_t)k);
}

bitmm_status bitmm_beam_select(const void* logits, int64_t row_stride, const float* scores,
                               const uint8_t* finished, float* scores_out, int32_t* parents,
                               int32_t* tokens, uint8_t* finished_out, int64_t groups, int64_t beams,
                               int64_t vocab, int64_t k, int32_t end_token, bitmm_out logits_type,
                               void* workspace, size_t workspace_bytes, uint32_t* status, void* stream) {
  try {
    bitmm::launch_log_begin();
    if (logits_type != BITMM_OUT_BF16 && logits_type != BITMM_OUT_F32 && logits_type != BITMM_OUT_F16)
      return BITMM_ERR_UNSUPPORTED;
    if (!select_sizes_ok(groups, beams, vocab, k)) return BITMM_ERR_SHAPE;
    if (row_stride < vocab) return BITMM_ERR_SHAPE;
    if (groups == 0) return BITMM_OK;
    if (!logits || !scores || !scores_out || !parents || !tokens) return BITMM_ERR_NULL;
    if (!aligned(logits, logits_type == BITMM_OUT_F32 ? 4 : 2) || !aligned(scores, 4) || !aligned(scores_out, 4) ||
        !aligned(parents, 4) || !aligned(tokens, 4) || !aligned(status, 4) || !aligned(workspace, 16))
      return BITMM_ERR_ALIGN;
    if (!workspace || workspace_bytes < bitmm_beam_select_workspace_bytes(groups, beams, vocab, k, logits_type))
      return BITMM_ERR_WORKSPACE;
    bitmm_status st;
    if ((st = device_check()) != BITMM_OK) return st;
    const SelectPlan plan = plan_select(groups * beams, vocab, logits_type);
    SelectParams p = {};
    p.logits = logits;
    p.row_stride = row_stride;
    p.scores = scores;
    p.finished = finished;
    p.scores_out = scores_out;
    p.parents = parents;
    p.tokens = tokens;
    p.finished_out = finished_out;
    p.part_sum = static_cast<double*>(workspace);
    p.part_top = reinterpret_cast<uint64_t*>(p.part_sum + 2 * groups * beams * plan.parts);
    p.status = status;
    p.beams = (int)beams;
    p.vocab = (int)vocab;
    p.k = (int)k;
    p.end_token = end_token;
    return launched(launch_beam_select(p, plan, groups, logits_type, static_cast<hipStream_t>(stream)));
  } catch (...) {
    return BITMM_ERR_LAUNCH;
  }
}

size_t bitmm_kv_beam_reorder_workspace_bytes(int64_t groups, int64_t beams) {
  return beam_rows_ok(groups, beams) ? (size_t)(groups * beams) * 16 : 0;
}

bitmm_status bitmm_kv_beam_reorder(const bitmm_kv_cache* caches, int64_t layers, const int32_t* page_table,
                                   int32_t* page_table_out, int64_t pages_per_seq, const int32_t* lens,
                                   int32_t* lens_out, const int32_t* parents, int64_t* slots,
                                   int64_t groups, int64_t beams, int64_t first_page,
                                   int64_t pages_per_group, void* workspace, size_t workspace_bytes,
                                   uint32_t* status, void* stream) {
  try {
    bitmm::launch_log_begin();
    if (layers < 1 || layers > 4096) return BITMM_ERR_SHAPE;
    if (!caches) return BITMM_ERR_NULL;
    bitmm_status st;
    for (int64_t i = 0; i < layers; ++i) {
      if ((st = check_cache(caches + i)) != BITMM_OK) return st;
      const bitmm_kv_cache &a = caches[0], &b = caches[i];
      if (a.num_pages != b.num_pages || a.page_size != b.page_size || a.kv_heads != b.kv_heads || a.head_dim != b.head_dim ||
          a.group_size != b.group_size)
        return BITMM_ERR_SHAPE;
    }
    if (!beam_rows_ok(groups, beams)) return BITMM_ERR_SHAPE;
    if (pages_per_seq < 1 || pages_per_seq > (int64_t)1 << 22) return BITMM_ERR_SHAPE;
    if (first_page < 0 || pages_per_group < 0 || pages_per_group > 1 << 18 || first_page > caches->num_pages ||
        groups * pages_per_group > caches->num_pages - first_page)
      return BITMM_ERR_SHAPE;
    if (groups == 0) return BITMM_OK;
    if (!page_table || !page_table_out || !lens || !lens_out || !parents || !slots) return BITMM_ERR_NULL;
    if (!aligned(page_table, 4) || !aligned(page_table_out, 4) || !aligned(lens, 4) || !aligned(lens_out, 4) ||
        !aligned(parents, 4) || !aligned(slots, 8) || !aligned(status, 4) || !aligned(workspace, 16))
      return BITMM_ERR_ALIGN;
    if (!workspace || workspace_bytes < bitmm_kv_beam_reorder_workspace_bytes(groups, beams)) return BITMM_ERR_WORKSPACE;
    if ((st = device_check()) != BITMM_OK) return st;
    const Cache c = view(caches);
    ReorderParams p = {};
    p.table = page_table;
    p.table_out = page_table_out;
    p.lens = lens;
    p.lens_out = lens_out;
    p.parents = parents;
    p.slots = slots;
    p.copies = workspace;
    p.status = status;
    p.pages_per_seq = pages_per_seq;
    p.beams = (int)beams;
    p.page_shift = c.page_shift;
    p.num_pages = c.num_pages;
    p.first_page = (int)first_page;
    p.pages_per_group = (int)pages_per_group;
    p.kv_heads = c.kv_heads;
    p.code_pieces = c.head_dim / 32;
    p.groups_of_head = c.head_dim / c.group;
    return launched(launch_beam_reorder(p, caches, layers, groups, static_cast<hipStream_t>(stream)));
  } catch (...) {
    return BITMM_ERR_LAUNCH;
  }
}

size_t bitmm_kv_attention_shared_workspace_bytes(int64_t T, int64_t B, int64_t groups, int64_t max_group_q,
                                                 int64_t max_prefix, int64_t max_q, int64_t max_kv,
                                                 int64_t q_heads, int64_t kv_heads, int64_t head_dim) {
  if (!shared_sizes_ok(T, B, groups, max_group_q, max_prefix, max_q, max_kv, q_heads, kv_heads) || !head_dim_ok(head_dim)) return 0;
  if (T == 0 || B == 0 || max_q == 0) return 0;
  const SharedPlan plan = plan_attention_shared(groups, B, max_group_q, max_prefix, max_q, max_kv, q_heads, kv_heads, head_dim);
  const PartRows rows = part_rows(plan, B, groups, max_group_q, q_heads, kv_heads);
  return ((size_t)(rows.prefix + rows.own) * (size_t)(head_dim + 2) * 4 + 255) / 256 * 256;
}

bitmm_status bitmm_kv_attention_shared(const void* q, int64_t q_stride, const bitmm_kv_cache* cache,
                                       const int32_t* prefix_table, int64_t pages_per_prefix,
                                       const int32_t* prefix_lens, const int32_t* cu_groups,
                                       const int32_t* page_table, int64_t pages_per_seq,
                                       const int32_t* kv_lens, const int32_t* cu_q, void* out,
                                       int64_t out_stride, float* lse, int64_t T, int64_t B, int64_t groups,
                                       int64_t q_heads, int64_t max_group_q, int64_t max_prefix,
                                       int64_t max_q, int64_t max_kv, float scale, bitmm_dtype dtype,
                                       bitmm_out out_type, void* workspace, size_t workspace_bytes,
                                       uint32_t* status, void* stream) {
  try {
    bitmm::launch_log_begin();
    bitmm_status st = check_cache(cache);
    if (st != BITMM_OK) return st;
    if (!dtype_ok(dtype)) return BITMM_ERR_UNSUPPORTED;
    if (out_type != BITMM_OUT_BF16 && out_type != BITMM_OUT_F32 && out_type != BITMM_OUT_F16) return BITMM_ERR_UNSUPPORTED;
    const int64_t kv_heads = cache->kv_heads, D = cache->head_dim;
    if (!shared_sizes_ok(T, B, groups, max_group_q, max_prefix, max_q, max_kv, q_heads, kv_heads) || !fits_int(pages_per_prefix) ||
        !fits_int(pages_per_seq))
      return BITMM_ERR_SHAPE;
    if (q_heads / kv_heads > 64 || B > 65535 || groups > 65535) return BITMM_ERR_UNSUPPORTED;
    if (T == 0 || B == 0 || max_q == 0) return BITMM_OK;
    if ((st = check_rows(q, q_stride, q_heads, D)) != BITMM_OK) return st;
    if ((st = check_rows(out, out_stride, q_heads, D)) != BITMM_OK) return st;
    if ((pages_per_seq > 0 && !page_table) || !kv_lens || !cu_q) return BITMM_ERR_NULL;
    if (groups > 0 && ((pages_per_prefix > 0 && !prefix_table) || !prefix_lens || !cu_groups)) return BITMM_ERR_NULL;
    if (!aligned(prefix_table, 4) || !aligned(prefix_lens, 4) || !aligned(cu_groups, 4) || !aligned(page_table, 4) ||
        !aligned(kv_lens, 4) || !aligned(cu_q, 4) || !aligned(lse, 4) || !aligned(status, 4) || !aligned(workspace, 16))
      return BITMM_ERR_ALIGN;
    const SharedPlan plan = plan_attention_shared(groups, B, max_group_q, max_prefix, max_q, max_kv, q_heads, kv_heads, D);
    // A launch's threads are counted in 32 bits.
    const int64_t limit = ((int64_t)1 << 32) / 512 - 1;
    if (plan.prefix.workgroups(groups * kv_heads) > limit || plan.own.workgroups(B * kv_heads) > limit ||
        groups * kv_heads * max_group_q * (q_heads / kv_heads) > INT32_MAX || B * kv_heads * plan.own.tail_rows > limit)
      return BITMM_ERR_UNSUPPORTED;
    const size_t need = bitmm_kv_attention_shared_workspace_bytes(T, B, groups, max_group_q, max_prefix, max_q, max_kv, q_heads,
                                                                  kv_heads, D);
    if (need > 0 && (!workspace || workspace_bytes < need)) return BITMM_ERR_WORKSPACE;
    if ((st = device_check()) != BITMM_OK) return st;
    AttentionParams p = {};
    p.q = static_cast<const uint16_t*>(q);
    p.cache = view(cache);
    p.page_table = page_table;
    p.kv_lens = kv_lens;
    p.cu_q = cu_q;
    p.out = out;
    p.lse = lse;
    p.status = status;
    p.q_stride = q_stride;
    p.out_stride = out_stride;
    p.pages_per_seq = pages_per_seq;
    p.T = (int)T;
    p.B = (int)B;
    p.q_heads = (int)q_heads;
    p.share = (int)(q_heads / kv_heads);
    p.max_q = (int)max_q;
    p.max_kv = (int)max_kv;
    p.otype = out_type == BITMM_OUT_F32 ? bitmm::kOutF32 : (out_type == BITMM_OUT_F16 ? bitmm::kOutF16 : bitmm::kOutBf16);
    p.scale = scale;
    SharedParams both = {p, p};
    both.prefix.page_table = prefix_table;
    both.prefix.kv_lens = prefix_lens;
    both.prefix.pages_per_seq = pages_per_prefix;
    both.prefix.B = (int)groups;
    both.prefix.max_q = (int)max_group_q;
    both.prefix.max_kv = (int)max_prefix;
    both.prefix.cu_groups = cu_groups;
    both.prefix.sequences = (int)B;
    const PartRows rows = part_rows(plan, B, groups, max_group_q, q_heads, kv_heads);
    both.prefix.part_o = static_cast<float*>(workspace);
    both.own.part_o = both.prefix.part_o + rows.prefix * D;
    both.prefix.part_ml = both.own.part_o + rows.own * D;
    both.own.part_ml = both.prefix.part_ml + 2 * rows.prefix;
    return launched(launch_kv_attention_shared(both, plan, (int)dtype, static_cast<hipStream_t>(stream)));
  } catch (...) {
    return BITMM_ERR_LAUNCH;
  }
}

}  // extern "C"
