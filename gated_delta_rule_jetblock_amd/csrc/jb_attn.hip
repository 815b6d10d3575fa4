// jb_attn.hip -- attention over a paged cache in the queries' type (jb_attn_core.h).
#include "jb_attn_core.h"

namespace jb {

int64_t attn_workgroups(const AttnCall& c) { return workgroups(c); }

size_t attn_workspace_bytes(const AttnCall& c) { return layout(c, plan(c)).bytes; }

bool attn_lists_fit(const BlockCall& c) { return list_rows(c); }

size_t attn_lists_bytes(const BlockCall& c) { return list_rows_bytes(c); }

int64_t attn_lists_workgroups(const BlockCall& c) {
  return std::max(list_units(c) * list_pieces(c) * cdiv(list_waves(c.D, c.bits8), 4), cdiv(c.total * c.H, 1024 / c.D));
}

hipError_t launch_attn_lists(const AttnCall& attn, const BlockCall& c, hipStream_t stream) {
  return run_lists<false>(attn, c, stream);
}

hipError_t launch_attn(const AttnCall& c, hipStream_t stream) { return run<false>(c, stream); }

}  // namespace jb
