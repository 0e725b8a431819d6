// kv4_window_attention.hip — attention over the paged 4-bit cache in which a query sees the last `window`
// tokens up to its own and the first `sinks` of its sequence (kv4_attention_device.h).
#include "kv4_attention_device.h"

namespace fp8q {

int launch_kv4_window_attention(int dtype, int64_t D, const Kv4AttnParams& p, void* ws, int64_t ws_bytes, hipStream_t stream) {
  return launch_masked<kWindow>(dtype, D, p, window_tokens(p.max_tokens, p.window, p.sinks), ws, ws_bytes, stream);
}

}  // namespace fp8q
