// Internal interface of the kernels behind include/bitmm_beam.h. Callers of the launch functions
// have validated every argument.
#pragma once

#include "attn.hpp"

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

}  // namespace attn
}  // namespace bitmm
