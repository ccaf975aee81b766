// attention_paged_tree: attention of drafted tokens that form trees.  A row sees the cached tokens before the new
// ones and, of these, those whose bits are set in its mask; the rest is attention_paged's (attention_core.h), whose tiles of old keys
// are seen whole and whose edge tiles take the bits.
#include "attention_core.h"

namespace w4 {

void launch_attention_tree(const AttnArgs& a, void* ws, hipStream_t st) { launch_as<true>(a, ws, st); }

}  // namespace w4
