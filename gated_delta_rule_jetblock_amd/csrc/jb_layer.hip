// jb_layer.hip -- the C ABI of the attention-layer operators (declared in
// include/jetblock.h): host-side validation and dispatch.  As in jb_api.hip,
// every check comes before the first HIP call.
#include "jb_layer_checks.h"

extern "C" {

jb_status jb_qk_norm_rope(const jb_attn_shape* s, const void* q, const void* k, const void* wq, const void* wk,
                          const float* inv_freq, const int32_t* positions, float eps, void* q_out, void* k_out,
                          void* stream) {
  const char* fn = "jb_qk_norm_rope";
  jb_status st = check_shape(fn, s, s ? (int64_t)s->B * s->T : 0, false);
  if (!st) st = check_rope(fn, s);
  if (st) return st;
  if (!(eps >= 0) || isinf(eps)) return fail(JB_ERR_INVALID_ARG, "%s: eps = %g is not finite and >= 0", fn, (double)eps);
  if (s->T == 0) return ok();
  JB_REQUIRE(q, 16); JB_REQUIRE(k, 16); JB_OPTIONAL(wq, 16); JB_OPTIONAL(wk, 16);
  if (s->rot) JB_REQUIRE(inv_freq, 4);
  JB_REQUIRE(positions, 4); JB_REQUIRE(q_out, 16); JB_REQUIRE(k_out, 16);
  jb::RopeCall c = rope_call(s, (int64_t)s->B * s->T);
  if (!c.norm && (wq || wk)) return fail(JB_ERR_INVALID_ARG, "%s: wq and wk must be NULL with JB_ROPE_NO_NORM", fn);
  c.q = q, c.k = k, c.wq = wq, c.wk = wk, c.inv_freq = inv_freq, c.positions = positions, c.eps = eps;
  c.q_out = q_out, c.k_out = k_out;
  if (jb::rope_workgroups(c) > MOST_GROUPS)
    return fail(JB_ERR_UNSUPPORTED, "%s: more workgroups than a launch can have", fn);
  return hip_status(fn, jb::launch_rope(c, static_cast<hipStream_t>(stream)));
}

jb_status jb_qk_norm_rope_backward_workspace_size(const jb_attn_shape* s, size_t* bytes) {
  const char* fn = "jb_qk_norm_rope_backward_workspace_size";
  jb_status st = check_shape(fn, s, s ? (int64_t)s->B * s->T : 0, false);
  if (!st) st = check_rope(fn, s);
  if (st) return st;
  if (!bytes) return fail(JB_ERR_INVALID_ARG, "%s: bytes is NULL", fn);
  *bytes = jb::rope_backward_workspace_bytes(rope_call(s, (int64_t)s->B * s->T));
  return ok();
}

jb_status jb_qk_norm_rope_backward(const jb_attn_shape* s, const void* q, const void* k, const void* wq,
                                   const void* wk, const float* inv_freq, const int32_t* positions, float eps,
                                   const void* dq_out, const void* dk_out, void* dq, void* dk, float* dwq, float* dwk,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "jb_qk_norm_rope_backward";
  jb_status st = check_shape(fn, s, s ? (int64_t)s->B * s->T : 0, false);
  if (!st) st = check_rope(fn, s);
  if (st) return st;
  if (!(eps >= 0) || isinf(eps)) return fail(JB_ERR_INVALID_ARG, "%s: eps = %g is not finite and >= 0", fn, (double)eps);
  jb::RopeCall c = rope_call(s, (int64_t)s->B * s->T);
  if (!c.norm && (wq || wk || dwq || dwk))
    return fail(JB_ERR_INVALID_ARG, "%s: wq, wk, dwq and dwk must be NULL with JB_ROPE_NO_NORM", fn);
  if (s->T > 0) {
    JB_REQUIRE(q, 16); JB_REQUIRE(k, 16); JB_OPTIONAL(wq, 16); JB_OPTIONAL(wk, 16);
    if (s->rot) JB_REQUIRE(inv_freq, 4);
    JB_REQUIRE(positions, 4); JB_REQUIRE(dq_out, 16); JB_REQUIRE(dk_out, 16); JB_REQUIRE(dq, 16); JB_REQUIRE(dk, 16);
  }
  JB_OPTIONAL(dwq, 4); JB_OPTIONAL(dwk, 4);
  const size_t need = jb::rope_backward_workspace_bytes(c);
  if (need && !workspace) return fail(JB_ERR_WORKSPACE, "%s: workspace is NULL (%zu bytes needed)", fn, need);
  if (workspace_bytes < need)
    return fail(JB_ERR_WORKSPACE, "%s: workspace has %zu bytes, %zu needed", fn, workspace_bytes, need);
  JB_OPTIONAL(workspace, 256);
  hipStream_t hs = static_cast<hipStream_t>(stream);
  if (s->T == 0) {  // no token, no gradient
    hipError_t e = hipSuccess;
    if (dwq) e = jb::launch_fill_zero(dwq, s->D, hs);
    if (dwk && e == hipSuccess) e = jb::launch_fill_zero(dwk, s->D, hs);
    return hip_status(fn, e);
  }
  c.q = q, c.k = k, c.wq = wq, c.wk = wk, c.inv_freq = inv_freq, c.positions = positions, c.eps = eps;
  c.dq_out = dq_out, c.dk_out = dk_out, c.dq = dq, c.dk = dk, c.dwq = dwq, c.dwk = dwk, c.workspace = workspace;
  return hip_status(fn, jb::launch_rope_backward(c, hs));
}

jb_status jb_qk_norm_rope_paged(const jb_attn_shape* s, int64_t total_tokens, const int32_t* cu_seqlens,
                                const int32_t* kv_lens, const int32_t* page_table, const void* q, const void* k,
                                const void* v, const void* wq, const void* wk, const float* inv_freq,
                                const int32_t* positions, float eps, void* q_out, void* k_cache, void* v_cache,
                                void* stream) {
  const char* fn = "jb_qk_norm_rope_paged";
  jb_status st = check_shape(fn, s, total_tokens, cu_seqlens != nullptr);
  if (!st) st = check_rope(fn, s);
  if (!st) st = check_cache(fn, s);
  if (st) return st;
  if (s->out_dtype != s->io_dtype) return fail(JB_ERR_UNSUPPORTED, "%s: out_dtype must be io_dtype", fn);
  if (!(eps >= 0) || isinf(eps)) return fail(JB_ERR_INVALID_ARG, "%s: eps = %g is not finite and >= 0", fn, (double)eps);
  JB_OPTIONAL(cu_seqlens, 4);
  if (total_tokens == 0) return ok();
  JB_REQUIRE(kv_lens, 4); JB_REQUIRE(page_table, 4);
  JB_REQUIRE(q, 16); JB_REQUIRE(k, 16); JB_REQUIRE(v, 16); JB_OPTIONAL(wq, 16); JB_OPTIONAL(wk, 16);
  if (s->rot) JB_REQUIRE(inv_freq, 4);
  JB_OPTIONAL(positions, 4); JB_REQUIRE(q_out, 16); JB_REQUIRE(k_cache, 16); JB_REQUIRE(v_cache, 16);
  jb::RopeCall c = rope_call(s, total_tokens);
  if (!c.norm && (wq || wk)) return fail(JB_ERR_INVALID_ARG, "%s: wq and wk must be NULL with JB_ROPE_NO_NORM", fn);
  c.paged = true, c.packed = cu_seqlens != nullptr;
  c.page = s->page, c.max_pages = s->max_pages, c.num_pages = s->num_pages;
  c.page_stride = s->page_stride ? s->page_stride : (int64_t)s->Hkv * s->page * s->D;
  c.cu_seqlens = cu_seqlens, c.kv_lens = kv_lens, c.page_table = page_table;
  c.q = q, c.k = k, c.v = v, c.wq = wq, c.wk = wk, c.inv_freq = inv_freq, c.positions = positions, c.eps = eps;
  c.q_out = q_out, c.k_out = k_cache, c.v_out = v_cache;
  if (jb::rope_workgroups(c) > MOST_GROUPS)
    return fail(JB_ERR_UNSUPPORTED, "%s: more workgroups than a launch can have", fn);
  return hip_status(fn, jb::launch_rope(c, static_cast<hipStream_t>(stream)));
}

jb_status jb_attn_paged_workspace_size(const jb_attn_shape* s, int64_t total_tokens, int32_t packed, size_t* bytes) {
  const char* fn = "jb_attn_paged_workspace_size";
  jb_status st = check_attn(fn, s, total_tokens, packed != 0);
  if (st) return st;
  if (!bytes) return fail(JB_ERR_INVALID_ARG, "%s: bytes is NULL", fn);
  *bytes = total_tokens ? jb::attn_workspace_bytes(attn_call(s, total_tokens, packed != 0)) : 0;
  return ok();
}

jb_status jb_attn_paged(const jb_attn_shape* s, int64_t total_tokens, const int32_t* cu_seqlens,
                        const int32_t* kv_lens, const int32_t* page_table, const void* q, const void* k_cache,
                        const void* v_cache, float scale, void* o, float* lse, void* workspace,
                        size_t workspace_bytes, void* stream) {
  const char* fn = "jb_attn_paged";
  const bool packed = cu_seqlens != nullptr;
  jb_status st = check_attn(fn, s, total_tokens, packed);
  if (st) return st;
  if (!(scale >= 0) || isinf(scale))
    return fail(JB_ERR_INVALID_ARG, "%s: scale = %g is not finite and >= 0", fn, (double)scale);
  JB_OPTIONAL(cu_seqlens, 4);
  if (total_tokens == 0) return ok();
  JB_REQUIRE(kv_lens, 4); JB_REQUIRE(page_table, 4); JB_REQUIRE(q, 16); JB_REQUIRE(k_cache, 16);
  JB_REQUIRE(v_cache, 16); JB_REQUIRE(o, 16); JB_OPTIONAL(lse, 4);
  jb::AttnCall c = attn_call(s, total_tokens, packed);
  const size_t need = jb::attn_workspace_bytes(c);
  if (need && !workspace) return fail(JB_ERR_WORKSPACE, "%s: workspace is NULL (%zu bytes needed)", fn, need);
  if (workspace_bytes < need)
    return fail(JB_ERR_WORKSPACE, "%s: workspace has %zu bytes, %zu needed", fn, workspace_bytes, need);
  JB_OPTIONAL(workspace, 256);
  c.cu_seqlens = cu_seqlens, c.kv_lens = kv_lens, c.page_table = page_table;
  c.q = q, c.k_cache = k_cache, c.v_cache = v_cache, c.o = o, c.lse = lse, c.workspace = workspace;
  c.scale = scale == 0.f ? 1.f / sqrtf((float)s->D) : scale;
  return hip_status(fn, jb::launch_attn(c, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
