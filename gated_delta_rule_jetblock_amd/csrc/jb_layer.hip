// jb_layer.hip -- the C ABI of the attention-layer operators (declared in
// include/jetblock.h): host-side validation and dispatch.  As in jb_api.hip,
// every check comes before the first HIP call.
#include <math.h>

#include "../../include/jetblock.h"
#include "jb_attn.h"

namespace {

template <typename... A> jb_status fail(jb_status st, const char* fmt, A... a) {
  return static_cast<jb_status>(jb::api_fail(st, fmt, a...));
}
jb_status ok() { return static_cast<jb_status>(jb::api_ok()); }
jb_status hip_status(const char* fn, hipError_t e) {
  return e == hipSuccess ? ok() : fail(JB_ERR_HIP, "%s: %s", fn, hipGetErrorString(e));
}

#define JB_REQUIRE(p, bytes)                                                                               \
  do {                                                                                                     \
    if (!(p)) return fail(JB_ERR_INVALID_ARG, "%s: %s is NULL", fn, #p);                                   \
    if ((uintptr_t)(p) & ((bytes)-1))                                                                      \
      return fail(JB_ERR_INVALID_ARG, "%s: %s is not %d-byte aligned", fn, #p, bytes);                     \
  } while (0)
#define JB_OPTIONAL(p, bytes)                                                                              \
  do {                                                                                                     \
    if ((uintptr_t)(p) & ((bytes)-1))                                                                      \
      return fail(JB_ERR_INVALID_ARG, "%s: %s is not %d-byte aligned", fn, #p, bytes);                     \
  } while (0)

constexpr int64_t MOST = (int64_t)1 << 40;
// workgroups of 256 threads that a launch can have: its work-items are a 32-bit count
constexpr int64_t MOST_GROUPS = 0xffffffffLL / 256;

// Heads, dtypes, tokens and token strides; total: rows of the token-major tensors.
jb_status check_shape(const char* fn, const jb_attn_shape* s, int64_t total, bool packed) {
  if (!s) return fail(JB_ERR_INVALID_ARG, "%s: shape is NULL", fn);
  if (s->B < 1) return fail(JB_ERR_INVALID_ARG, "%s: B = %d must be >= 1", fn, s->B);
  if (s->B > 65535) return fail(JB_ERR_UNSUPPORTED, "%s: B = %d exceeds 65535", fn, s->B);
  if (s->T < 0) return fail(JB_ERR_INVALID_ARG, "%s: T = %d must be >= 0", fn, s->T);
  if (s->T > (1 << 30)) return fail(JB_ERR_UNSUPPORTED, "%s: T = %d exceeds 2^30", fn, s->T);
  const int64_t most = (int64_t)s->B * s->T;
  if (packed ? total < 0 || total > most : total != most)
    return fail(JB_ERR_INVALID_ARG, "%s: total_tokens = %lld (%s B*T = %lld)", fn, (long long)total,
                packed ? "packed: at most" : "cu_seqlens is NULL: must be", (long long)most);
  if (total > 0x7fffffffLL) return fail(JB_ERR_UNSUPPORTED, "%s: total_tokens exceeds 2^31 - 1", fn);
  if (s->H < 1 || s->H > 256) return fail(JB_ERR_UNSUPPORTED, "%s: H = %d not in [1, 256]", fn, s->H);
  if (s->Hkv < 1 || s->H % s->Hkv) return fail(JB_ERR_UNSUPPORTED, "%s: Hkv = %d does not divide H = %d", fn, s->Hkv, s->H);
  if (s->D != 64 && s->D != 128 && s->D != 256)
    return fail(JB_ERR_UNSUPPORTED, "%s: D = %d not in {64, 128, 256}", fn, s->D);
  if (s->io_dtype != JB_BF16 && s->io_dtype != JB_F32)
    return fail(JB_ERR_INVALID_ARG, "%s: io_dtype = %d is not a jb_dtype", fn, s->io_dtype);
  if (s->out_dtype != JB_BF16 && s->out_dtype != JB_F32)
    return fail(JB_ERR_INVALID_ARG, "%s: out_dtype = %d is not a jb_dtype", fn, s->out_dtype);
  const int per16 = s->io_dtype == JB_BF16 ? 8 : 4;
  const struct { const char* name; int64_t stride; int heads; } st[] = {
      {"q_stride", s->q_stride, s->H}, {"k_stride", s->k_stride, s->Hkv}, {"v_stride", s->v_stride, s->Hkv}};
  for (const auto& x : st) {
    if (x.stride && (x.stride < (int64_t)x.heads * s->D || x.stride % per16))
      return fail(JB_ERR_INVALID_ARG, "%s: %s = %lld is not a multiple of 16 bytes of at least heads * D", fn, x.name,
                  (long long)x.stride);
    if (x.stride >= MOST || std::max<int64_t>(x.stride, (int64_t)x.heads * s->D) >= MOST / std::max<int64_t>(total, 1))
      return fail(JB_ERR_UNSUPPORTED, "%s: tensor sizes exceed the supported range", fn);
  }
  return JB_OK;
}

jb_status check_rope(const char* fn, const jb_attn_shape* s) {
  if (s->rot < 0 || s->rot > s->D || s->rot % 16)
    return fail(JB_ERR_UNSUPPORTED, "%s: rot = %d is not a multiple of 16 in [0, D]", fn, s->rot);
  if (s->flags & ~(JB_ROPE_INTERLEAVED | JB_ROPE_NO_NORM))
    return fail(JB_ERR_INVALID_ARG, "%s: unknown flags 0x%x", fn, (unsigned)s->flags);
  return JB_OK;
}

jb_status check_cache(const char* fn, const jb_attn_shape* s) {
  if (s->page < 16 || s->page > 4096 || (s->page & (s->page - 1)))
    return fail(JB_ERR_UNSUPPORTED, "%s: page = %d is not a power of two in [16, 4096]", fn, s->page);
  if (s->max_pages < 1) return fail(JB_ERR_INVALID_ARG, "%s: max_pages = %d must be >= 1", fn, s->max_pages);
  if (s->num_pages < 1) return fail(JB_ERR_INVALID_ARG, "%s: num_pages = %d must be >= 1", fn, s->num_pages);
  if ((int64_t)s->max_pages * s->page > (1 << 30))
    return fail(JB_ERR_UNSUPPORTED, "%s: max_pages * page exceeds 2^30", fn);
  const int64_t one = (int64_t)s->Hkv * s->page * s->D;
  if (s->page_stride && (s->page_stride < one || s->page_stride % (s->io_dtype == JB_BF16 ? 8 : 4)))
    return fail(JB_ERR_INVALID_ARG, "%s: page_stride = %lld is not a multiple of 16 bytes of at least Hkv * page * D", fn,
                (long long)s->page_stride);
  if (s->page_stride >= MOST || std::max(s->page_stride, one) >= MOST / s->num_pages)
    return fail(JB_ERR_UNSUPPORTED, "%s: tensor sizes exceed the supported range", fn);
  if (s->window < 0 || s->window > (1 << 30))
    return fail(JB_ERR_INVALID_ARG, "%s: window = %d not in [0, 2^30]", fn, s->window);
  if (s->max_kv < 0) return fail(JB_ERR_INVALID_ARG, "%s: max_kv = %d must be >= 0", fn, s->max_kv);
  return JB_OK;
}

int io_of(int32_t dtype) { return dtype == JB_F32 ? jb::IO_F32 : jb::IO_BF16; }

jb::RopeCall rope_call(const jb_attn_shape* s, int64_t total) {
  jb::RopeCall c = {};
  c.B = s->B, c.T = s->T, c.H = s->H, c.Hkv = s->Hkv, c.D = s->D, c.rot = s->rot;
  c.io = io_of(s->io_dtype), c.out = io_of(s->out_dtype);
  c.interleaved = s->flags & JB_ROPE_INTERLEAVED, c.norm = !(s->flags & JB_ROPE_NO_NORM);
  c.total = total;
  c.q_stride = s->q_stride ? s->q_stride : (int64_t)s->H * s->D;
  c.k_stride = s->k_stride ? s->k_stride : (int64_t)s->Hkv * s->D;
  c.v_stride = s->v_stride ? s->v_stride : (int64_t)s->Hkv * s->D;
  return c;
}

jb::AttnCall attn_call(const jb_attn_shape* s, int64_t total, bool packed) {
  jb::AttnCall c = {};
  c.B = s->B, c.T = s->T, c.H = s->H, c.Hkv = s->Hkv, c.D = s->D;
  c.page = s->page, c.max_pages = s->max_pages, c.num_pages = s->num_pages, c.window = s->window;
  const int cap = s->max_pages * s->page;
  c.max_kv = s->max_kv ? std::min(s->max_kv, cap) : cap;
  c.io = io_of(s->io_dtype), c.out = io_of(s->out_dtype);
  c.packed = packed, c.total = total;
  c.q_stride = s->q_stride ? s->q_stride : (int64_t)s->H * s->D;
  c.page_stride = s->page_stride ? s->page_stride : (int64_t)s->Hkv * s->page * s->D;
  return c;
}

jb_status check_attn(const char* fn, const jb_attn_shape* s, int64_t total, bool packed) {
  jb_status st = check_shape(fn, s, total, packed);
  if (!st) st = check_cache(fn, s);
  if (st) return st;
  if (s->flags) return fail(JB_ERR_INVALID_ARG, "%s: flags must be 0", fn);
  if (total && jb::attn_workgroups(attn_call(s, total, packed)) > MOST_GROUPS)
    return fail(JB_ERR_UNSUPPORTED, "%s: more workgroups than a launch can have", fn);
  return JB_OK;
}

}  // namespace

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
