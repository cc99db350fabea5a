// Internal interface of the kernels behind include/bitmm_beam.h. Callers of the launch functions
// have validated every argument.
#pragma once

#include <algorithm>

#include "attn.hpp"
#include "bitmm_beam.h"

namespace bitmm {
namespace attn {

struct RopeAppendParams {
  RopeParams rope;  // its queries' side; of the keys' side k, k_stride and k_weight
  const uint16_t* v;
  int64_t v_stride;
  const int64_t* slots;
  Cache cache;
  uint32_t* status;
  int kv_waves;        // of a token's keys and values
  unsigned kv_blocks;  // workgroups of all keys and values: the grid's first
};
hipError_t launch_qk_norm_rope_append(const RopeAppendParams& p, bool interleaved, int dtype, hipStream_t stream);

struct SelectParams {
  const void* logits;
  int64_t row_stride;
  const float* scores;
  const uint8_t* finished;
  float* scores_out;
  int32_t* parents;
  int32_t* tokens;
  uint8_t* finished_out;
  double* part_sum;    // [rows, parts, 2]: reference and sum of exponentials over it
  uint64_t* part_top;  // [rows, parts, k]: (order of the logit, inverted token), largest first, 0 where none is left
  uint32_t* status;
  int beams, vocab, k, end_token;
  int parts, each;     // as in SelectPlan
};
// How a row is cut up: `parts` workgroups, whose waves take `each` pieces of 16 bytes.
struct SelectPlan {
  int parts, each;
};
SelectPlan plan_select(int64_t rows, int64_t vocab, bitmm_out type);
hipError_t launch_beam_select(SelectParams p, const SelectPlan& plan, int64_t groups, bitmm_out type, hipStream_t stream);

struct ReorderParams {
  const int32_t* table;
  int32_t* table_out;
  const int32_t* lens;
  int32_t* lens_out;
  const int32_t* parents;
  int64_t* slots;
  void* copies;  // 16 bytes a row
  uint32_t* status;
  int64_t pages_per_seq;
  int beams, page_shift, num_pages, first_page, pages_per_group;
  int kv_heads, code_pieces, groups_of_head;  // pieces of 16 bytes of a head's codes
};
// The caches of some layers, by value: they may change with the program's every call.
struct ReorderLayers {
  static constexpr int MOST = 64;
  struct Side {
    uint32_t *codes, *scales;
  };
  struct Layer {
    Side side[2];
  } at[MOST];
};
hipError_t launch_beam_reorder(const ReorderParams& p, const bitmm_kv_cache* caches, int64_t layers, int64_t groups,
                               hipStream_t stream);

}  // namespace attn
}  // namespace bitmm
