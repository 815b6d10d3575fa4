// jb_layer_checks.h -- host-side checks of the attention-layer operators' arguments, shared by
// their entry points (jb_layer.hip, jb_layer8.hip).
#pragma once

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

jb_status check_cache(const char* fn, const jb_attn_shape* s, bool bits8 = false) {
  if (s->page < 16 || s->page > 4096 || (s->page & (s->page - 1)))
    return fail(JB_ERR_UNSUPPORTED, "%s: page = %d is not a power of two in [16, 4096]", fn, s->page);
  if (s->max_pages < 1) return fail(JB_ERR_INVALID_ARG, "%s: max_pages = %d must be >= 1", fn, s->max_pages);
  if (s->num_pages < 1) return fail(JB_ERR_INVALID_ARG, "%s: num_pages = %d must be >= 1", fn, s->num_pages);
  if ((int64_t)s->max_pages * s->page > (1 << 30))
    return fail(JB_ERR_UNSUPPORTED, "%s: max_pages * page exceeds 2^30", fn);
  const int64_t one = (int64_t)s->Hkv * s->page * s->D;
  if (s->page_stride && (s->page_stride < one || s->page_stride % (bits8 ? 16 : s->io_dtype == JB_BF16 ? 8 : 4)))
    return fail(JB_ERR_INVALID_ARG, "%s: page_stride = %lld is not a multiple of 16 bytes of at least Hkv * page * D", fn,
                (long long)s->page_stride);
  if (s->page_stride >= MOST || std::max(s->page_stride, one) >= MOST / s->num_pages)
    return fail(JB_ERR_UNSUPPORTED, "%s: tensor sizes exceed the supported range", fn);
  if (s->window < 0 || s->window > (1 << 30))
    return fail(JB_ERR_INVALID_ARG, "%s: window = %d not in [0, 2^30]", fn, s->window);
  if (s->max_kv < 0) return fail(JB_ERR_INVALID_ARG, "%s: max_kv = %d must be >= 0", fn, s->max_kv);
  return JB_OK;
}

// distance between the pages of a cache's scales
jb_status check_scales(const char* fn, const jb_attn_shape* s, int64_t scale_stride) {
  const int64_t one = (int64_t)s->Hkv * s->page / 16;
  if (scale_stride && scale_stride < one)
    return fail(JB_ERR_INVALID_ARG, "%s: scale_stride = %lld is less than Hkv * page / 16", fn, (long long)scale_stride);
  if (scale_stride >= MOST || std::max(scale_stride, one) >= MOST / s->num_pages)
    return fail(JB_ERR_UNSUPPORTED, "%s: tensor sizes exceed the supported range", fn);
  return JB_OK;
}
int64_t scale_stride_of(const jb_attn_shape* s, int64_t scale_stride) {
  return scale_stride ? scale_stride : (int64_t)s->Hkv * s->page / 16;
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

jb_status check_attn(const char* fn, const jb_attn_shape* s, int64_t total, bool packed, bool bits8 = false) {
  jb_status st = check_shape(fn, s, total, packed);
  if (!st) st = check_cache(fn, s, bits8);
  if (st) return st;
  if (s->flags) return fail(JB_ERR_INVALID_ARG, "%s: flags must be 0", fn);
  jb::AttnCall c = attn_call(s, total, packed);
  c.bits8 = bits8;
  if (total && jb::attn_workgroups(c) > MOST_GROUPS)
    return fail(JB_ERR_UNSUPPORTED, "%s: more workgroups than a launch can have", fn);
  return JB_OK;
}

}  // namespace
