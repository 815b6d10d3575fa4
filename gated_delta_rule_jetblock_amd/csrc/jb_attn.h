// jb_attn.h -- host-side launchers of the attention-layer operators (jb_attn.hip,
// jb_rope.hip).  Arguments have been validated by jb_layer.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "jb_internal.h"

namespace jb {

struct AttnCall {
  int B, T, H, Hkv, D, page, max_pages, num_pages, max_kv, window;
  int io, out;       // IoType of q and the caches, and of o
  bool packed;       // cu_seqlens given
  int64_t total;     // tokens
  int64_t q_stride, page_stride;
  const int *cu_seqlens, *kv_lens, *page_table;
  const void *q, *k_cache, *v_cache;
  float scale;
  void* o;
  float* lse;
  void* workspace;
};
// pieces and workgroups depend on the sizes only, not on device memory
int64_t attn_workgroups(const AttnCall& c);  // of the largest launch, at most 256 threads each
size_t attn_workspace_bytes(const AttnCall& c);
hipError_t launch_attn(const AttnCall& c, hipStream_t stream);

struct RopeCall {
  int B, T, H, Hkv, D, rot, page, max_pages, num_pages;
  int io, out;
  bool interleaved, norm, packed, paged;
  int64_t total;
  int64_t q_stride, k_stride, v_stride, page_stride;
  const int *cu_seqlens, *kv_lens, *page_table, *positions;
  const void *q, *k, *v, *wq, *wk;
  const float* inv_freq;
  float eps;
  void *q_out, *k_out;   // k_out, v_out: the caches when paged
  void* v_out;
  // backward
  const void *dq_out, *dk_out;
  void *dq, *dk;
  float *dwq, *dwk;
  void* workspace;
};
int64_t rope_workgroups(const RopeCall& c);
hipError_t launch_rope(const RopeCall& c, hipStream_t stream);
size_t rope_backward_workspace_bytes(const RopeCall& c);
hipError_t launch_rope_backward(const RopeCall& c, hipStream_t stream);

}  // namespace jb
