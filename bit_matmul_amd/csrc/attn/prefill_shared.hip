// Attention of many query rows: attention_tiles.hpp's kernel as a pass of kv_attention_shared.
#include "attention_tiles.hpp"

namespace bitmm {
namespace attn {

hipError_t launch_attention_tiles_prefix(const AttentionParams& p, int rows_each, unsigned workgroups, int dtype,
                                         hipStream_t stream) {
  return launch_tiles_of<kPrefix>(p, p.cache, rows_each, workgroups, dtype, stream);
}

hipError_t launch_attention_tiles_own(const SharedParams& p, int rows_each, unsigned workgroups, int dtype,
                                      hipStream_t stream) {
  return launch_tiles_of<kOwn>(p, p.own.cache, rows_each, workgroups, dtype, stream);
}

}  // namespace attn
}  // namespace bitmm
