// Attention of many query rows: attention_tiles.hpp's kernel for kv_attention.
#include "attention_tiles.hpp"

namespace bitmm {
namespace attn {

hipError_t launch_attention_tiles(const AttentionParams& p, int rows_each, unsigned workgroups, int dtype,
                                  hipStream_t stream) {
  return launch_tiles_of<kAlone>(p, p.cache, rows_each, workgroups, dtype, stream);
}

}  // namespace attn
}  // namespace bitmm
