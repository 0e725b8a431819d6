// kv4_attention.hip — attention over the paged 4-bit cache, causal or not (kv4_attention_device.h).
#include "kv4_attention_device.h"

namespace fp8q {

int64_t kv4_attention_workspace(int dtype, int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_tokens,
                                Mask mask) {
  return attention_shape(current_device_shape().cus, dtype, B, T, Hq, Hkv, D, max_tokens, mask).bytes;
}

int launch_kv4_attention(int dtype, int64_t D, const Kv4AttnParams& p, void* ws, int64_t ws_bytes, hipStream_t stream) {
  return launch_masked<kAll>(dtype, D, p, p.max_tokens, ws, ws_bytes, stream);
}

}  // namespace fp8q
