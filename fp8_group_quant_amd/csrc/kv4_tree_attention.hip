// kv4_tree_attention.hip — attention over the paged 4-bit cache for drafted tokens that form a tree: a query
// sees the tokens before the draft and those drafted ones that its mask names (kv4_attention_device.h).
#include "kv4_attention_device.h"

namespace fp8q {

int launch_kv4_tree_attention(int dtype, int64_t D, const Kv4AttnParams& p, void* ws, int64_t ws_bytes, hipStream_t stream) {
  return launch_masked<kTree>(dtype, D, p, p.max_tokens, ws, ws_bytes, stream);
}

}  // namespace fp8q
