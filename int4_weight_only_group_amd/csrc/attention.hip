// attention_paged; its kernels and what they rest on are in attention_core.h.
#include "attention_core.h"

namespace w4 {

bool attention_ws_bytes(const AttnArgs& a, size_t& bytes) {
  const Launch x = plan(a);
  bytes = x.few_bytes + x.many_bytes;
  return launchable(x, a);
}

void launch_attention(const AttnArgs& a, void* ws, hipStream_t st) { launch_as<false>(a, ws, st); }

}  // namespace w4
