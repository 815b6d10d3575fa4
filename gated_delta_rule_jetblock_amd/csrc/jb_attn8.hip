// jb_attn8.hip -- attention over a paged cache in 8 bits (jb_attn_core.h).
#include "jb_attn_core.h"

namespace jb {

hipError_t launch_attn8_lists(const AttnCall& attn, const BlockCall& c, hipStream_t stream) {
  return run_lists<true>(attn, c, stream);
}

hipError_t launch_attn8(const AttnCall& c, hipStream_t stream) { return run<true>(c, stream); }

}  // namespace jb
