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
  bool bits8;        // a cache in 8 bits, with its scales' exponents; else in the queries' type
  const uint8_t *k_scales, *v_scales;
  int64_t scale_stride;
  int units;         // attention over listed pages: key heads of a token (each a sequence of one), or 0
};
// pieces and workgroups depend on the sizes only, not on device memory
int64_t attn_workgroups(const AttnCall& c);  // of the largest launch, at most 256 threads each
size_t attn_workspace_bytes(const AttnCall& c);
hipError_t launch_attn(const AttnCall& c, hipStream_t stream);
hipError_t launch_attn8(const AttnCall& c, hipStream_t stream);  // over a cache in 8 bits

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
  bool bits8;                    // append to a cache in 8 bits, with its scales' exponents; else in the inputs' type
  uint8_t *k_scales, *v_scales;
  int64_t scale_stride;
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

// Mean keys and scores of pages, their selection, and attention over listed pages
// (jb_blocks.hip).
struct BlockCall {
  int B, T, H, Hkv, D, page, max_pages, num_pages;
  int io;            // IoType of q (and of the cache without scales)
  bool packed;       // cu_seqlens given
  bool bits8;        // a cache in 8 bits
  int64_t total;
  int64_t q_stride, page_stride, scale_stride;
  const int *cu_seqlens, *kv_lens, *page_table;
  const void *q, *k_cache;
  const uint8_t* k_scales;
  float *means, *scores;
  const float* scores_in;   // selection
  int count, first, recent;
  int* blocks;       // written by the selection, read by the attention
};
int64_t block_scores_workgroups(const BlockCall& c);
hipError_t launch_block_scores(const BlockCall& c, hipStream_t stream);
int64_t block_select_workgroups(const BlockCall& c);  // at most, of 256 threads
hipError_t launch_block_select(const BlockCall& c, hipStream_t stream);
int64_t attn_blocks_workgroups(const BlockCall& c, const AttnCall& attn);
// the lists that the decode kernel takes itself (otherwise they become tables in memory)
bool attn_lists_fit(const BlockCall& c);
size_t attn_lists_bytes(const BlockCall& c);
int64_t attn_lists_workgroups(const BlockCall& c);  // at most, of 256 threads
hipError_t launch_attn_lists(const AttnCall& attn, const BlockCall& c, hipStream_t stream);
hipError_t launch_attn8_lists(const AttnCall& attn, const BlockCall& c, hipStream_t stream);
size_t attn_blocks_workspace_bytes(const BlockCall& c, const AttnCall& attn);
hipError_t launch_attn_blocks(const BlockCall& c, const AttnCall& attn, hipStream_t stream);

}  // namespace jb
