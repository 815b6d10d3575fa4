// jb_layer8.hip -- the C ABI of the attention-layer operators for long contexts: a cache in
// 8 bits, and attention over selected pages (declared in include/jetblock.h).  As in
// jb_api.hip, every check comes before the first HIP call.
#include "jb_layer_checks.h"

namespace {

// The calls over pages: their shape, and count where they have one (else 1)
jb_status check_blocks(const char* fn, const jb_attn_shape* s, int64_t total, bool packed, int32_t count, bool cache) {
  jb_status st = check_shape(fn, s, total, packed);
  if (st) return st;
  if (s->flags & ~(cache ? JB_CACHE_E4M3 : 0)) return fail(JB_ERR_INVALID_ARG, "%s: unknown flags 0x%x", fn, (unsigned)s->flags);
  st = check_cache(fn, s, s->flags & JB_CACHE_E4M3);
  if (st) return st;
  if (s->window) return fail(JB_ERR_UNSUPPORTED, "%s: window must be 0", fn);
  if (count < 1) return fail(JB_ERR_INVALID_ARG, "%s: count = %d must be >= 1", fn, count);
  if ((int64_t)count * s->page > (1 << 30)) return fail(JB_ERR_UNSUPPORTED, "%s: count * page exceeds 2^30", fn);
  if (std::max<int64_t>(count, s->max_pages) >= MOST / std::max<int64_t>(total * s->Hkv, 1))
    return fail(JB_ERR_UNSUPPORTED, "%s: tensor sizes exceed the supported range", fn);
  if (total * s->Hkv > MOST_GROUPS) return fail(JB_ERR_UNSUPPORTED, "%s: more workgroups than a launch can have", fn);
  return JB_OK;
}

jb::BlockCall block_call(const jb_attn_shape* s, int64_t total, bool packed) {
  jb::BlockCall c = {};
  c.B = s->B, c.T = s->T, c.H = s->H, c.Hkv = s->Hkv, c.D = s->D;
  c.page = s->page, c.max_pages = s->max_pages, c.num_pages = s->num_pages;
  c.io = io_of(s->io_dtype), c.packed = packed, c.bits8 = s->flags & JB_CACHE_E4M3, c.total = total;
  c.q_stride = s->q_stride ? s->q_stride : (int64_t)s->H * s->D;
  c.page_stride = s->page_stride ? s->page_stride : (int64_t)s->Hkv * s->page * s->D;
  return c;
}

}  // namespace

extern "C" {

jb_status jb_qk_norm_rope_paged8(const jb_attn_shape* s, int64_t total_tokens, const int32_t* cu_seqlens,
                                 const int32_t* kv_lens, const int32_t* page_table, const void* q, const void* k,
                                 const void* v, const void* wq, const void* wk, const float* inv_freq,
                                 const int32_t* positions, float eps, void* q_out, void* k_cache, void* v_cache,
                                 uint8_t* k_scales, uint8_t* v_scales, int64_t scale_stride, void* stream) {
  const char* fn = "jb_qk_norm_rope_paged8";
  jb_status st = check_shape(fn, s, total_tokens, cu_seqlens != nullptr);
  if (!st) st = check_rope(fn, s);
  if (!st) st = check_cache(fn, s, true);
  if (!st) st = check_scales(fn, s, scale_stride);
  if (st) return st;
  if (s->out_dtype != s->io_dtype) return fail(JB_ERR_UNSUPPORTED, "%s: out_dtype must be io_dtype", fn);
  if (!(eps >= 0) || isinf(eps)) return fail(JB_ERR_INVALID_ARG, "%s: eps = %g is not finite and >= 0", fn, (double)eps);
  JB_OPTIONAL(cu_seqlens, 4);
  if (total_tokens == 0) return ok();
  JB_REQUIRE(kv_lens, 4); JB_REQUIRE(page_table, 4);
  JB_REQUIRE(q, 16); JB_REQUIRE(k, 16); JB_REQUIRE(v, 16); JB_OPTIONAL(wq, 16); JB_OPTIONAL(wk, 16);
  if (s->rot) JB_REQUIRE(inv_freq, 4);
  JB_OPTIONAL(positions, 4); JB_REQUIRE(q_out, 16); JB_REQUIRE(k_cache, 16); JB_REQUIRE(v_cache, 16);
  JB_REQUIRE(k_scales, 1); JB_REQUIRE(v_scales, 1);
  jb::RopeCall c = rope_call(s, total_tokens);
  if (!c.norm && (wq || wk)) return fail(JB_ERR_INVALID_ARG, "%s: wq and wk must be NULL with JB_ROPE_NO_NORM", fn);
  c.paged = true, c.packed = cu_seqlens != nullptr;
  c.page = s->page, c.max_pages = s->max_pages, c.num_pages = s->num_pages;
  c.page_stride = s->page_stride ? s->page_stride : (int64_t)s->Hkv * s->page * s->D;
  c.cu_seqlens = cu_seqlens, c.kv_lens = kv_lens, c.page_table = page_table;
  c.q = q, c.k = k, c.v = v, c.wq = wq, c.wk = wk, c.inv_freq = inv_freq, c.positions = positions, c.eps = eps;
  c.q_out = q_out, c.k_out = k_cache, c.v_out = v_cache;
  c.bits8 = true, c.k_scales = k_scales, c.v_scales = v_scales, c.scale_stride = scale_stride_of(s, scale_stride);
  if (jb::rope_workgroups(c) > MOST_GROUPS)
    return fail(JB_ERR_UNSUPPORTED, "%s: more workgroups than a launch can have", fn);
  return hip_status(fn, jb::launch_rope(c, static_cast<hipStream_t>(stream)));
}

jb_status jb_attn_paged8_workspace_size(const jb_attn_shape* s, int64_t total_tokens, int32_t packed, size_t* bytes) {
  const char* fn = "jb_attn_paged8_workspace_size";
  jb_status st = check_attn(fn, s, total_tokens, packed != 0, true);
  if (st) return st;
  if (!bytes) return fail(JB_ERR_INVALID_ARG, "%s: bytes is NULL", fn);
  jb::AttnCall c = attn_call(s, total_tokens, packed != 0);
  c.bits8 = true;
  *bytes = total_tokens ? jb::attn_workspace_bytes(c) : 0;
  return ok();
}

jb_status jb_attn_paged8(const jb_attn_shape* s, int64_t total_tokens, const int32_t* cu_seqlens,
                         const int32_t* kv_lens, const int32_t* page_table, const void* q, const void* k_cache,
                         const void* v_cache, const uint8_t* k_scales, const uint8_t* v_scales, int64_t scale_stride,
                         float scale, void* o, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "jb_attn_paged8";
  const bool packed = cu_seqlens != nullptr;
  jb_status st = check_attn(fn, s, total_tokens, packed, true);
  if (!st) st = check_scales(fn, s, scale_stride);
  if (st) return st;
  if (!(scale >= 0) || isinf(scale))
    return fail(JB_ERR_INVALID_ARG, "%s: scale = %g is not finite and >= 0", fn, (double)scale);
  JB_OPTIONAL(cu_seqlens, 4);
  if (total_tokens == 0) return ok();
  JB_REQUIRE(kv_lens, 4); JB_REQUIRE(page_table, 4); JB_REQUIRE(q, 16); JB_REQUIRE(k_cache, 16);
  JB_REQUIRE(v_cache, 16); JB_REQUIRE(k_scales, 1); JB_REQUIRE(v_scales, 1); JB_REQUIRE(o, 16); JB_OPTIONAL(lse, 4);
  jb::AttnCall c = attn_call(s, total_tokens, packed);
  c.bits8 = true, c.k_scales = k_scales, c.v_scales = v_scales, c.scale_stride = scale_stride_of(s, scale_stride);
  const size_t need = jb::attn_workspace_bytes(c);
  if (need && !workspace) return fail(JB_ERR_WORKSPACE, "%s: workspace is NULL (%zu bytes needed)", fn, need);
  if (workspace_bytes < need)
    return fail(JB_ERR_WORKSPACE, "%s: workspace has %zu bytes, %zu needed", fn, workspace_bytes, need);
  JB_OPTIONAL(workspace, 256);
  c.cu_seqlens = cu_seqlens, c.kv_lens = kv_lens, c.page_table = page_table;
  c.q = q, c.k_cache = k_cache, c.v_cache = v_cache, c.o = o, c.lse = lse, c.workspace = workspace;
  c.scale = scale == 0.f ? 1.f / sqrtf((float)s->D) : scale;
  return hip_status(fn, jb::launch_attn8(c, static_cast<hipStream_t>(stream)));
}

jb_status jb_block_scores(const jb_attn_shape* s, int64_t total_tokens, const int32_t* cu_seqlens,
                          const int32_t* kv_lens, const int32_t* page_table, const void* q, const void* k_cache,
                          const uint8_t* k_scales, int64_t scale_stride, float* means, float* scores, void* stream) {
  const char* fn = "jb_block_scores";
  const bool packed = cu_seqlens != nullptr;
  jb_status st = check_blocks(fn, s, total_tokens, packed, 1, true);
  if (!st) st = check_scales(fn, s, scale_stride);
  if (st) return st;
  const bool bits8 = s->flags & JB_CACHE_E4M3;
  if (!bits8 && k_scales) return fail(JB_ERR_INVALID_ARG, "%s: k_scales must be NULL without JB_CACHE_E4M3", fn);
  JB_OPTIONAL(cu_seqlens, 4);
  if (total_tokens == 0) return ok();
  JB_REQUIRE(kv_lens, 4); JB_REQUIRE(page_table, 4); JB_REQUIRE(k_cache, 16); JB_REQUIRE(means, 16);
  if (bits8) JB_REQUIRE(k_scales, 1);
  if (scores) JB_REQUIRE(q, 16);
  JB_OPTIONAL(scores, 4);
  jb::BlockCall c = block_call(s, total_tokens, packed);
  c.scale_stride = scale_stride_of(s, scale_stride);
  c.cu_seqlens = cu_seqlens, c.kv_lens = kv_lens, c.page_table = page_table;
  c.q = q, c.k_cache = k_cache, c.k_scales = k_scales, c.means = means, c.scores = scores;
  if (jb::block_scores_workgroups(c) > MOST_GROUPS)
    return fail(JB_ERR_UNSUPPORTED, "%s: more workgroups than a launch can have", fn);
  return hip_status(fn, jb::launch_block_scores(c, static_cast<hipStream_t>(stream)));
}

jb_status jb_block_select(const jb_attn_shape* s, int64_t total_tokens, const int32_t* cu_seqlens,
                          const int32_t* kv_lens, const float* scores, int32_t count, int32_t first, int32_t recent,
                          int32_t* blocks, void* stream) {
  const char* fn = "jb_block_select";
  const bool packed = cu_seqlens != nullptr;
  jb_status st = check_blocks(fn, s, total_tokens, packed, count, false);
  if (st) return st;
  if (s->max_pages > 65536) return fail(JB_ERR_UNSUPPORTED, "%s: max_pages = %d exceeds 65536", fn, s->max_pages);
  if (first < 0 || recent < 1 || (int64_t)first + recent > count)
    return fail(JB_ERR_INVALID_ARG, "%s: first = %d, recent = %d: at least 0 and 1, together at most count = %d", fn, first,
                recent, count);
  JB_OPTIONAL(cu_seqlens, 4);
  if (total_tokens == 0) return ok();
  JB_REQUIRE(kv_lens, 4); JB_REQUIRE(scores, 4); JB_REQUIRE(blocks, 4);
  jb::BlockCall c = block_call(s, total_tokens, packed);
  c.cu_seqlens = cu_seqlens, c.kv_lens = kv_lens, c.scores_in = scores, c.blocks = blocks;
  c.count = count, c.first = first, c.recent = recent;
  if (jb::block_select_workgroups(c) > MOST_GROUPS)
    return fail(JB_ERR_UNSUPPORTED, "%s: more workgroups than a launch can have", fn);
  return hip_status(fn, jb::launch_block_select(c, static_cast<hipStream_t>(stream)));
}

jb_status jb_attn_blocks_workspace_size(const jb_attn_shape* s, int64_t total_tokens, int32_t packed, int32_t count,
                                        size_t* bytes) {
  const char* fn = "jb_attn_blocks_workspace_size";
  jb_status st = check_blocks(fn, s, total_tokens, packed != 0, count, true);
  if (st) return st;
  if (!bytes) return fail(JB_ERR_INVALID_ARG, "%s: bytes is NULL", fn);
  jb::AttnCall x = attn_call(s, total_tokens, packed != 0);
  jb::BlockCall c = block_call(s, total_tokens, packed != 0);
  x.bits8 = c.bits8, c.count = count;
  if (total_tokens && jb::attn_blocks_workgroups(c, x) > MOST_GROUPS)
    return fail(JB_ERR_UNSUPPORTED, "%s: more workgroups than a launch can have", fn);
  *bytes = total_tokens ? jb::attn_blocks_workspace_bytes(c, x) : 0;
  return ok();
}

jb_status jb_attn_blocks(const jb_attn_shape* s, int64_t total_tokens, const int32_t* cu_seqlens,
                         const int32_t* kv_lens, const int32_t* page_table, const void* q, const void* k_cache,
                         const void* v_cache, const uint8_t* k_scales, const uint8_t* v_scales, int64_t scale_stride,
                         const int32_t* blocks, int32_t count, float scale, void* o, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream) {
  const char* fn = "jb_attn_blocks";
  const bool packed = cu_seqlens != nullptr;
  jb_status st = check_blocks(fn, s, total_tokens, packed, count, true);
  if (!st) st = check_scales(fn, s, scale_stride);
  if (st) return st;
  const bool bits8 = s->flags & JB_CACHE_E4M3;
  if (!bits8 && (k_scales || v_scales))
    return fail(JB_ERR_INVALID_ARG, "%s: k_scales and v_scales must be NULL without JB_CACHE_E4M3", fn);
  if (!(scale >= 0) || isinf(scale))
    return fail(JB_ERR_INVALID_ARG, "%s: scale = %g is not finite and >= 0", fn, (double)scale);
  JB_OPTIONAL(cu_seqlens, 4);
  if (total_tokens == 0) return ok();
  JB_REQUIRE(kv_lens, 4); JB_REQUIRE(page_table, 4); JB_REQUIRE(q, 16); JB_REQUIRE(k_cache, 16); JB_REQUIRE(v_cache, 16);
  if (bits8) { JB_REQUIRE(k_scales, 1); JB_REQUIRE(v_scales, 1); }
  JB_REQUIRE(blocks, 4); JB_REQUIRE(o, 16); JB_OPTIONAL(lse, 4);
  jb::AttnCall x = attn_call(s, total_tokens, packed);
  jb::BlockCall c = block_call(s, total_tokens, packed);
  x.bits8 = c.bits8, x.k_scales = k_scales, x.v_scales = v_scales, x.scale_stride = scale_stride_of(s, scale_stride);
  c.count = count;
  if (jb::attn_blocks_workgroups(c, x) > MOST_GROUPS)
    return fail(JB_ERR_UNSUPPORTED, "%s: more workgroups than a launch can have", fn);
  const size_t need = jb::attn_blocks_workspace_bytes(c, x);
  if (need && !workspace) return fail(JB_ERR_WORKSPACE, "%s: workspace is NULL (%zu bytes needed)", fn, need);
  if (workspace_bytes < need)
    return fail(JB_ERR_WORKSPACE, "%s: workspace has %zu bytes, %zu needed", fn, workspace_bytes, need);
  JB_OPTIONAL(workspace, 256);
  x.q = q, x.k_cache = k_cache, x.v_cache = v_cache, x.o = o, x.lse = lse, x.workspace = workspace;
  x.scale = scale == 0.f ? 1.f / sqrtf((float)s->D) : scale;
  c.cu_seqlens = cu_seqlens, c.kv_lens = kv_lens, c.page_table = page_table;
  c.blocks = const_cast<int32_t*>(blocks);  // (read only here)
  return hip_status(fn, jb::launch_attn_blocks(c, x, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
