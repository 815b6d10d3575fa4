// jb_rope.hip -- norm of every query and key head with the position rotation.
//
// A row x of D values (one token's query or key head):
//     r = (mean x^2 + eps)^{-1/2},  n = x r,  y = R (n w)
// R turns each pair (a, b) of the first `rot` values by the angle
// position * inv_freq[pair]: (a cos - b sin, b cos + a sin); pairs are
// (i, i + rot/2) or, interleaved, (2 i, 2 i + 1).  Backward, from dy:
//     g = R^T dy,  dw = sum over rows of g n,  h = g w,
//     dx = r (h - n mean(h n)).
// Without the norm n = x and w = 1.
//
// Bound by HBM: a row is read and written once (backward: read twice, written
// once) against some ten operations a value.  D / 8 lanes hold a row, 8 values
// each (16 bytes of bf16), and take one token through all its heads (or a part
// of them when there are few tokens), so that a token's angles are formed once:
// position * inv_freq in 64 bits, taken to a fraction of a turn before the sine
// and cosine, because a far position's angle keeps no fraction in 32.
// The angles and the weight become two factors a value, y = r (x c + x' s) with
// x' the other member of the pair, fetched from its lane as raw bits.
// dw is summed in fp32 in a fixed order: lanes over their tokens, the
// workgroup through LDS, then one kernel over the workgroups' sums (5 us).
// 64K tokens of 12 + 2 heads of 128, bf16: 87-92 us over the cards, 5.1-5.4 TB/s (a plain
// copy kernel reaches 6.3, the library's copy 5.0); backward 130-137 us, 5.2-5.4
// TB/s, 3 workgroups a CU; fp32 199 and 297 us, 4.7 TB/s; the append of 13K tokens in
// 32 chunks, 16 + 2 heads: 35 us, 3.8 TB/s, a quarter of it the chain of loads that
// finds a token's place (fp32 76 us, 3.4 TB/s).
#include "jb_attn.h"
#include "jb_device.h"
#include "jb_e4m3.h"

namespace jb {

namespace {

struct Args {
  RopeCall c;
  int parts, heads;   // head parts a token is cut into, heads a part
  int64_t units;      // tokens x parts
  float* sums;        // backward: [workgroups][2][D]
  int64_t cells;      // append in 8 bits: places for 16 cache rows with new ones
  int kv_heads;       // and its key heads (c.Hkv is 0: the heads by token are the queries)
};

template <typename T> struct Raw;
template <> struct Raw<bf16_t> {
  uint32_t u[4];
  static constexpr int N = 4;
  __device__ float get(int i) const { return __uint_as_float(i & 1 ? u[i >> 1] & 0xffff0000u : u[i >> 1] << 16); }
};
template <> struct Raw<float> {
  uint32_t u[8];
  static constexpr int N = 8;
  __device__ float get(int i) const { return __uint_as_float(u[i]); }
};
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));
// NT: past the caches: training's loads and stores, and the append's q_out although
// the attention reads that next.  64K tokens take 95.7 us forward and 143 backward
// without, 88.9 and 132.5 with; an append of 13K tokens 36.7 and 35.0 (its loads gain
// nothing).
template <bool NT = false, typename T> __device__ __forceinline__ Raw<T> load8(const T* p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < Raw<T>::N / 4; ++i) {
    const u4_t* a = reinterpret_cast<const u4_t*>(p) + i;
    const u4_t w = NT ? __builtin_nontemporal_load(a) : *a;
#pragma unroll
    for (int e = 0; e < 4; ++e) r.u[4 * i + e] = w[e];
  }
  return r;
}
template <bool NT> __device__ __forceinline__ void put4(void* p, u4_t v) {
  if constexpr (NT) __builtin_nontemporal_store(v, static_cast<u4_t*>(p));
  else *static_cast<u4_t*>(p) = v;
}
template <typename T> __device__ __forceinline__ void store_raw(T* p, const Raw<T>& r) {
#pragma unroll
  for (int i = 0; i < Raw<T>::N / 4; ++i)
    put4<false>(reinterpret_cast<u4_t*>(p) + i, u4_t{r.u[4 * i], r.u[4 * i + 1], r.u[4 * i + 2], r.u[4 * i + 3]});
}
template <bool NT> __device__ __forceinline__ void store8(float* p, const float (&y)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    put4<NT>(p + 4 * i, u4_t{__float_as_uint(y[4 * i]), __float_as_uint(y[4 * i + 1]), __float_as_uint(y[4 * i + 2]),
                             __float_as_uint(y[4 * i + 3])});
}
template <bool NT> __device__ __forceinline__ void store8(bf16_t* p, const float (&y)[8]) {
  u4_t u;
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = f32_to_bf16(y[2 * i]) | (uint32_t)f32_to_bf16(y[2 * i + 1]) << 16;
  put4<NT>(p, u);
}

// sum over a row's D / 8 lanes
template <int L> __device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = L / 2; o >= 1; o >>= 1) v += __shfl_xor(v, o, WAVE);
  return v;
}

// This lane's 8 values of a row in the rotation: cosines and signed sines
// (y_e = cos x_e + sin x'_e), and the lane that holds the x'_e (or this one,
// where pairs lie inside a lane or a value is not rotated).
struct Turn {
  float cos[8], sin[8];
};

template <int D> __device__ __forceinline__ int partner(const RopeCall& c, int s) {
  const int half = c.rot / 16;
  return c.interleaved ? s : s < half ? s + half : s < 2 * half ? s - half : s;
}

// sin and cos of 2 pi t for |t| <= 1/2 (turns): the nearest quarter turn comes
// off (exactly), the rest, at most an eighth, goes through the Taylor series of
// both up to x^9 and x^10; the first terms left out are at most 2^-29 and 2^-33 (at
// pi / 4).  Off by at most 9e-8, with t's own rounding to 24 bits by 1.5e-7.
__device__ __forceinline__ void sincos_turn(float t, float& sn, float& cs) {
  const float n = rintf(4.f * t), x = fmaf(-0.25f, n, t), y = x * x;
  const float s = x * fmaf(y, fmaf(y, fmaf(y, fmaf(y, 42.0586939f, -76.7058598f), 81.6052493f), -41.3417022f), 6.28318531f);
  const float c = fmaf(y, fmaf(y, fmaf(y, fmaf(y, fmaf(y, -26.4262568f, 60.2446414f), -85.4568172f), 64.939394f), -19.7392088f), 1.f);
  const int q = (int)n;
  const float a = q & 1 ? c : s, b = q & 1 ? s : c;
  sn = q & 2 ? -a : a;
  cs = (q + 1) & 2 ? -b : b;
}

typedef float f4u_t __attribute__((ext_vector_type(4), aligned(4)));  // four floats anywhere

// the frequencies of this lane's pairs (8, or 4 interleaved); 0 where nothing turns
// (loads without a branch, from the first row of q where there is nothing to load: several
// then wait together)
__device__ __forceinline__ void frequencies(const RopeCall& c, int s, float (&f)[8]) {
  const bool turns = 8 * s < c.rot;
  const float* p = c.inv_freq + (c.interleaved ? 4 * s : 8 * s < c.rot / 2 ? 8 * s : 8 * s - c.rot / 2);
  if (!turns) p = static_cast<const float*>(c.q);
  const f4u_t u = *reinterpret_cast<const f4u_t*>(p);
  const f4u_t v = *reinterpret_cast<const f4u_t*>(p + (c.interleaved ? 0 : 4));
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = turns ? u[i] : 0.f, f[4 + i] = turns ? v[i] : 0.f;
}

template <int D> __device__ __forceinline__ Turn turn_of(const RopeCall& c, int s, const float (&f)[8], int position) {
  Turn t;
  const double p = (double)position * 0.15915494309189533577;  // turns per radian
  const bool first = 8 * s < c.rot / 2;
  if (c.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double turns = p * (double)f[i];
      float sn, cs;
      sincos_turn((float)(turns - rint(turns)), sn, cs);
      t.cos[2 * i] = t.cos[2 * i + 1] = cs;
      t.sin[2 * i] = -sn;
      t.sin[2 * i + 1] = sn;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double turns = p * (double)f[i];
      float sn, cs;
      sincos_turn((float)(turns - rint(turns)), sn, cs);
      t.cos[i] = cs;
      t.sin[i] = first ? -sn : sn;
    }
  }
  return t;
}

// the other members of this lane's pairs; zeros where the rotation does not reach
// (rot is a multiple of 16, so a lane's values turn or do not together): their sine
// is 0, but 0 times an inf or NaN would not be
template <typename T>
__device__ __forceinline__ Raw<T> others(const Raw<T>& x, bool interleaved, int lane, bool turns) {
  Raw<T> y;
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < Raw<T>::N; ++i)
      y.u[i] = sizeof(T) == 2 ? (x.u[i] >> 16 | x.u[i] << 16) : x.u[sizeof(T) == 2 ? i : i ^ 1];
  } else {
#pragma unroll
    for (int i = 0; i < Raw<T>::N; ++i) y.u[i] = (uint32_t)__shfl((int)x.u[i], lane, WAVE);
  }
#pragma unroll
  for (int i = 0; i < Raw<T>::N; ++i) y.u[i] = turns ? y.u[i] : 0u;
  return y;
}

template <typename T> __device__ __forceinline__ void weights(const RopeCall& c, const void* w, int e0, float (&out)[8]) {
  const Raw<T> r = load8((const T*)(w ? w : c.q) + e0);
#pragma unroll
  for (int i = 0; i < 8; ++i) out[i] = w ? r.get(i) : 1.f;
}

// The sequence of a packed batch that holds `target`, where sequence j's share begins at
// start(its offset, j), which never decreases: its index, offsets and cache length in one
// step, found by the thread that looks at it.  (Offsets that decrease: any one.)
struct Found {
  int b, from, to, kv;
};
template <typename F> __device__ __forceinline__ Found find_sequence(const RopeCall& c, int64_t target, F start) {
  __shared__ __attribute__((aligned(16))) int at[4];
  for (int j = threadIdx.x; j < c.B; j += 256) {
    const int from = c.cu_seqlens[j], to = c.cu_seqlens[j + 1], kv = c.kv_lens[j];
    if ((j == 0 || start(from, j) <= target) && (j + 1 == c.B || start(to, j + 1) > target))
      *reinterpret_cast<int4*>(at) = make_int4(j, from, to, kv);
  }
  __syncthreads();
  return {min(max(__builtin_amdgcn_readfirstlane(at[0]), 0), c.B - 1), __builtin_amdgcn_readfirstlane(at[1]),
          __builtin_amdgcn_readfirstlane(at[2]), __builtin_amdgcn_readfirstlane(at[3])};
}

// workgroup `block` of the heads of all tokens; KV: keys (and values) too, else the queries
template <int D, typename IO, typename OUT, bool PAGED, bool KV>
__device__ __forceinline__ void rope_rows(const Args& a, uint32_t block) {
  constexpr int L = D / 8, GROUPS = 256 / L;
  block = __builtin_amdgcn_readfirstlane(block);
  // rows in use, and as many on their way (64K tokens: 4 take 88.9 us, 2 90.9; an
  // append of 13K tokens 34.5 and 35.0, where 2 need fewer registers)
  constexpr int U = PAGED || sizeof(IO) == 4 ? 2 : 4;
  const RopeCall& c = a.c;
  const int lane = lane_id(), s = lane % L, group = threadIdx.x / L;
  const int64_t unit = (int64_t)block * GROUPS + group;
  bool live = unit < a.units;
  // (fewer than 2^31 units where a token has several)
  int64_t t = !live ? 0 : a.parts == 1 ? unit : (uint32_t)unit / (uint32_t)a.parts;
  const int h0 = a.parts == 1 || !live ? 0 : (int)((uint32_t)unit % (uint32_t)a.parts) * a.heads;
  // what does not depend on the token's place is on its way while that is found
  const int nh = c.H + (!KV ? 0 : PAGED ? 2 : 1) * c.Hkv, h1 = min(h0 + a.heads, nh);
  const IO* q = (const IO*)c.q + t * c.q_stride + 8 * s;
  const IO* k = (const IO*)c.k + t * c.k_stride + 8 * s;
  const IO* v = (const IO*)c.v + (PAGED ? t * c.v_stride + 8 * s : 0);
  Raw<IO> x[U], next[U];
  auto fetch = [&](Raw<IO>(&x)[U], int h) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = min(h + u, h1 - 1);
      x[u] = load8<!PAGED>(i < c.H ? q + (int64_t)i * D : i < c.H + c.Hkv ? k + (int64_t)(i - c.H) * D
                                                              : v + (int64_t)(i - c.H - c.Hkv) * D);
    }
  };
  fetch(x, h0);
  const int es = partner<D>(c, s) * 8, from = (lane & ~(L - 1)) + es / 8;
  float f[8], wq[8], wqp[8], wk[8], wkp[8];
  frequencies(c, s, f);
  weights<IO>(c, c.wq, 8 * s, wq);
  weights<IO>(c, c.wq, es, wqp);
  weights<IO>(c, c.wk, 8 * s, wk);
  weights<IO>(c, c.wk, es, wkp);
  int row = 0;          // the token's row in its sequence's cache
  int64_t slot = -1;    // and in the pool (element offset of key head 0), or -1
  if constexpr (PAGED) {
    int b;
    int64_t i;
    int T = c.T;  // the sequence's tokens (those behind the first c.T are not taken)
    int kv;
    if (c.packed) {
      // the sequence of the workgroup's first token, then on from there
      const int64_t t0 = (int64_t)block * GROUPS / a.parts;
      Found f = find_sequence(c, t0, [](int from, int) { return (int64_t)from; });
      while (f.b + 1 < c.B && f.to <= t) {
        ++f.b;
        f.from = f.to, f.to = c.cu_seqlens[f.b + 1], f.kv = c.kv_lens[f.b];
      }
      b = f.b, kv = f.kv;
      int64_t tok0;
      clamp_span(f.from, f.to, 0x7fffffff, c.total, tok0, T);
      i = t - tok0;
      live = live && i >= 0 && i < min(T, c.T);
    } else {
      b = (int)((uint32_t)t / (uint32_t)c.T);
      i = t - (int64_t)b * c.T;
      kv = c.kv_lens[b];
    }
    const int pshift = __builtin_ctz((unsigned)c.page);
    const int cap = (int)min((int64_t)c.max_pages << pshift, (int64_t)0x7fffffff);
    row = min(max(kv, 0), cap) - T + (int)i;
    if (KV && live && row >= 0) {
      const int pid = c.page_table[(int64_t)b * c.max_pages + (row >> pshift)];
      if (pid >= 0 && pid < c.num_pages) slot = pid * c.page_stride + (int64_t)(row & (c.page - 1)) * D;
    }
  }
  if (!live) return;  // whole lane groups leave; the others shuffle among themselves
  const Turn turn = turn_of<D>(c, s, f, c.positions ? c.positions[t] : row);
  // y = r (x cw + x' sw), for queries and for keys
  float cq[8], sq[8], ck[8], sk[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    cq[i] = wq[i] * turn.cos[i];
    sq[i] = (c.interleaved ? wqp[i ^ 1] : wqp[i]) * turn.sin[i];
    ck[i] = wk[i] * turn.cos[i];
    sk[i] = (c.interleaved ? wkp[i ^ 1] : wkp[i]) * turn.sin[i];
  }
  for (int h = h0; h < h1; h += U) {
    if (h + U < h1) fetch(next, h + U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = h + u;
      if (i >= h1) break;
      if (PAGED && i >= c.H + c.Hkv) {
        if (slot >= 0) store_raw((IO*)c.v_out + slot + (int64_t)(i - c.H - c.Hkv) * c.page * D + 8 * s, x[u]);
        continue;
      }
      float r = 1.f;
      if (c.norm) {
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(x[u].get(e), x[u].get(e), sum);
        r = 1.f / sqrtf(row_sum<L>(sum) * (1.f / D) + c.eps);
      }
      const Raw<IO> xp = others(x[u], c.interleaved, from, 8 * s < c.rot);
      const bool key = i >= c.H;
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        y[e] = r * fmaf(x[u].get(e), key ? ck[e] : cq[e], xp.get(e) * (key ? sk[e] : sq[e]));
      if (!key) store8<true>((OUT*)c.q_out + (t * c.H + i) * D + 8 * s, y);
      else if (!PAGED) store8<true>((OUT*)c.k_out + (t * c.Hkv + i - c.H) * D + 8 * s, y);
      else if (slot >= 0) store8<false>((OUT*)c.k_out + slot + (int64_t)(i - c.H) * c.page * D + 8 * s, y);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = next[u];
  }
}

template <int D, typename IO, typename OUT, bool PAGED>
__global__ __launch_bounds__(256) void rope_kernel(Args a) {
  rope_rows<D, IO, OUT, PAGED, true>(a, blockIdx.x);
}

// Keys that become codes are formed in 64 bits: a value's error flips its code where the value
// lies that near to a border, and the errors of fp32 arithmetic (8e-8 rms) flip 2 of a million
// codes by a whole step, where these flip 0.1 (13K tokens on 2 key heads, on one card: 31.4 us, in fp32 29.9).
//
// a cos + b sin of 2 pi t.  As in sincos_turn the nearest quarter turn comes off (here a sum's
// low bits; |t| < 2^48, what lies past that has no angle in 64 bits); it swaps a and b and
// turns their signs.  The leading terms a + 2 pi x b are in 64 bits, the others, at most 0.3 a and
// 0.1 b, in fp32: off by 7e-9 of hypot(a, b) rms and 2.5 * 2^-24 at most (roundings of f, y and the
// two sums; 7e-8 seen).
template <typename T> __device__ __forceinline__ double turned(T a, T b, double t) {
  const double up = 6755399441055744., at = fma(4., t, up), x = fma(-0.25, at - up, t);  // up: 1.5 * 2^52
  const int q = __double2loint(at);
  const float f = (float)x, y = f * f;
  const float s = f * y * fmaf(y, fmaf(y, fmaf(y, 42.0586939f, -76.7058598f), 81.6052493f), -41.3417022f);
  const float c = y * fmaf(y, fmaf(y, fmaf(y, fmaf(y, -26.4262568f, 60.2446414f), -85.4568172f), 64.939394f), -19.7392088f);
  T u = q & 1 ? b : a, v = q & 1 ? a : b;
  u = q & 2 ? -u : u;
  v = (q + 1) & 2 ? -v : v;
  return fma((double)v, 6.283185307179586 * x, (double)u) + (double)fmaf((float)u, c, (float)v * s);
}

// x to 24 bits, towards the neighbour whose last bit is set where it lies between two: rounded
// again to fewer bits it gives what x itself gives
__device__ __forceinline__ float odd_of(double x) {
  const int lo = __double2loint(x);
  return (float)__hiloint2double(__double2hiint(x), (lo & 0xe0000000) | (lo & 0x1fffffff ? 0x20000000 : 0));
}

// a row's 8 values of this lane: normalised, weighted and turned
template <int L, typename IO>
__device__ __forceinline__ void turned_key(const RopeCall& c, const Raw<IO>& x, const Raw<IO>& xp, const float (&w)[8],
                                           const float (&wp)[8], const float (&f)[8], bool first, int position,
                                           float (&y)[8]) {
  double r = 1.;
  if (c.norm) {
    double sum = 0.;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fma((double)x.get(e), (double)x.get(e), sum);
#pragma unroll
    for (int o = L / 2; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, WAVE);
    const double m = sum * (1. / (8 * L)) + (double)c.eps;
    const float q = 1.f / sqrtf((float)m);
    r = q > 0.f && isfinite(q) ? (double)q * (1.5 - 0.5 * m * (double)q * (double)q) : (double)q;  // a Newton step
  }
  const double p = (double)position * 0.15915494309189533577;  // turns per radian
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const double t = p * (double)(c.interleaved ? f[e >> 1] : f[e]);
    const bool minus = c.interleaved ? !(e & 1) : first;
    const float we = c.interleaved ? wp[e ^ 1] : wp[e];
    double z;
    if constexpr (sizeof(IO) == 2) {  // (16-bit values: their products are exact in fp32)
      const float b = xp.get(e) * we;
      z = turned(x.get(e) * w[e], minus ? -b : b, t);
    } else {
      const double b = (double)xp.get(e) * (double)we;
      z = turned((double)x.get(e) * (double)w[e], minus ? -b : b, t);
    }
    y[e] = odd_of(r * z);
    __builtin_amdgcn_sched_barrier(0);  // (values in turn: together they take half as many registers again)
  }
}

// Exponent e of the smallest scale 2^(e - 127) with most <= 448 times it, 1 at least:
// 448 = 1.75 * 2^8, so it is most's exponent less 8, or less 7 where its fraction is over 1.75.
__device__ __forceinline__ int exponent_for(float most) {
  const uint32_t u = __float_as_uint(most);
  return max((int)(u >> 23) - ((u & 0x7fffffu) > 0x600000u ? 7 : 8), 1);
}
// 2^(127 - e), what values are divided by their scale with
__device__ __forceinline__ float inverse_scale(int e) { return __uint_as_float(e >= 254 ? 1u << 22 : (uint32_t)(254 - e) << 23); }

// 8 values to the nearest codes, ties to even (|x| <= 448; infinities and NaN become NaN)
__device__ __forceinline__ uint2 e4m3_of(const float (&x)[8]) {
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], hi, true);
  return make_uint2(lo, hi);
}

// The append to a cache in 8 bits.  The first a.cells * Hkv workgroups take 16 cache rows
// of one key head each, K and V: its lane groups form the new rows' values, the largest
// finite one sets the scale, and if rows of earlier calls share it the larger of the two
// scales holds: their codes are divided by 2^k (exactly, but for those that fall below the
// smallest normal code, which are rounded again).  Rows behind the new ones keep their codes.
// The other workgroups rotate the queries.
// 32 chunks, 13K tokens of 16 + 2 heads of 128: 30-31 us, 4.1 TB/s; the keys' part by itself
// would be 18 of that and the sums in 64 bits, nearly all the chain of lookups (offsets and length, page
// index, what the page holds) before a workgroup's first store.  One token: 5.4 us.
template <int D, typename IO>
__global__ __launch_bounds__(256) void rope_append8_kernel(Args a) {
  constexpr int L = D / 8, GROUPS = 256 / L, N = 32 / GROUPS;  // rows at once; times for 16 of K and 16 of V
  const RopeCall& c = a.c;
  const uint32_t cells = (uint32_t)a.cells * (uint32_t)a.kv_heads;
  // the keys' workgroups first, which wait for what they look up (13K tokens, with sums in fp32,
  // on one card: in turn with the queries' 30.6 us, so 29.3)
  if (blockIdx.x >= cells) {
    rope_rows<D, IO, IO, true, false>(a, blockIdx.x - cells);
    return;
  }
  const uint32_t cell = blockIdx.x / (uint32_t)a.kv_heads;
  const int head = blockIdx.x - cell * (uint32_t)a.kv_heads;
  const int lane = lane_id(), s = lane % L, group = threadIdx.x / L;
  // the cell's sequence and its place among those that hold the sequence's new rows
  int b, kv, T = c.T, all = c.T;
  int64_t nth, tok0;
  if (c.packed) {
    // sequence j's cells start at cu[j] / 16 + 2 j, which leaves room for all of them
    auto start = [&](int from, int j) { return (min(max((int64_t)from, (int64_t)0), c.total) >> 4) + 2 * (int64_t)j; };
    const Found f = find_sequence(c, cell, start);
    b = f.b, kv = f.kv;
    nth = (int64_t)cell - start(f.from, b);
    clamp_span(f.from, f.to, 0x7fffffff, c.total, tok0, all);
    T = min(all, c.T);
  } else {
    const uint32_t per = (uint32_t)(c.T + 14) / 16 + 1;
    b = (int)(cell / per);
    nth = cell - (uint32_t)b * per;
    tok0 = (int64_t)b * c.T;
    kv = c.kv_lens[b];
  }
  const int pshift = __builtin_ctz((unsigned)c.page), cap = (int)min((int64_t)c.max_pages << pshift, (int64_t)0x7fffffff);
  const int row0 = min(max(kv, 0), cap) - all;  // of the first new token
  const int end = row0 + T;
  const int64_t first = ((int64_t)(max(row0, 0) >> 4) + nth) << 4;
  if (nth < 0 || T == 0 || first >= end) return;
  // the new rows and the page index arrive together, then what the page holds
  const int pid = c.page_table[(int64_t)b * c.max_pages + (first >> pshift)];
  const bool shared = row0 > first;  // rows of earlier calls
  const int es = partner<D>(c, s) * 8, from = (lane & ~(L - 1)) + es / 8;
  Raw<IO> x[N];
  uint2 was[N];
  bool fresh[N], kept[N];
  int position[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int r = n * GROUPS + group, row = (int)first + (r & 15);
    fresh[n] = row >= row0 && row < end;
    kept[n] = row < row0;
    const int64_t t = tok0 + (fresh[n] ? row - row0 : 0);
    x[n] = load8(r < 16 ? (const IO*)c.k + t * c.k_stride + (int64_t)head * D + 8 * s
                        : (const IO*)c.v + t * c.v_stride + (int64_t)head * D + 8 * s);
    position[n] = row;
    if (c.positions && r < 16) position[n] = c.positions[t];
  }
  if (pid < 0 || pid >= c.num_pages) return;
  const int64_t at = pid * c.page_stride + (((int64_t)head << pshift) + (first & (c.page - 1))) * D + 8 * s;
  const int64_t scale = pid * c.scale_stride + ((((int64_t)head << pshift) + (first & (c.page - 1))) >> 4);
  int e_was[2] = {0, 0};
#pragma unroll
  for (int n = 0; n < N; ++n) was[n] = make_uint2(0u, 0u);
  if (shared) {
    e_was[0] = c.k_scales[scale], e_was[1] = c.v_scales[scale];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int r = n * GROUPS + group;
      if (kept[n]) was[n] = *reinterpret_cast<const uint2*>((const char*)(r < 16 ? c.k_out : c.v_out) + at + (int64_t)(r & 15) * D);
    }
  }
  float f[8], wk[8], wkp[8];
  frequencies(c, s, f);
  weights<IO>(c, c.wk, 8 * s, wk);
  weights<IO>(c, c.wk, es, wkp);
  __shared__ float largest[32];
  float y[N][8];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int r = n * GROUPS + group;
    const bool key = r < 16;  // (the same for a wave: 16 rows are a whole number of its lane groups)
    if (key) {
      turned_key<L>(c, x[n], others(x[n], c.interleaved, from, 8 * s < c.rot), wk, wkp, f, 8 * s < c.rot / 2, position[n], y[n]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[n][e] = x[n].get(e);
    }
    float most = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) most = fmaxf(most, isfinite(y[n][e]) ? fabsf(y[n][e]) : 0.f);
#pragma unroll
    for (int o = L / 2; o >= 1; o >>= 1) most = fmaxf(most, __shfl_xor(most, o, WAVE));
    if (s == 0) largest[r] = fresh[n] ? most : 0.f;  // (the others hold the first new token's row)
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int r = n * GROUPS + group, kv = r >> 4;
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) most = fmaxf(most, largest[kv * 16 + i]);
    const int e = shared ? max(exponent_for(most), e_was[kv]) : exponent_for(most);
    char* const cache = (char*)(kv ? c.v_out : c.k_out);
    if (fresh[n]) {
      const float inv = inverse_scale(e);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[n][i] *= inv;
      if (e >= 247) {  // the largest code whose value is less than 2^128, which is no number in fp32 or bf16
        const float top = 0.9375f * __uint_as_float((uint32_t)(382 - e) << 23);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[n][i] = isfinite(y[n][i]) ? fminf(fmaxf(y[n][i], -top), top) : y[n][i];
      }
      *reinterpret_cast<uint2*>(cache + at + (int64_t)(r & 15) * D) = e4m3_of(y[n]);
    } else if (kept[n] && e != e_was[kv]) {
      const float4 lo = floats_of_e4m3(was[n].x, e_was[kv]), hi = floats_of_e4m3(was[n].y, e_was[kv]);
      const float inv = inverse_scale(e);
      const float z[8] = {lo.x * inv, lo.y * inv, lo.z * inv, lo.w * inv, hi.x * inv, hi.y * inv, hi.z * inv, hi.w * inv};
      *reinterpret_cast<uint2*>(cache + at + (int64_t)(r & 15) * D) = e4m3_of(z);
    }
    if ((r & 15) == 0 && s == 0) (kv ? c.v_scales : c.k_scales)[scale] = (uint8_t)e;
  }
}

template <int D, typename IO, typename GR>
__global__ __launch_bounds__(256, 3) void rope_backward_kernel(Args a) {
  constexpr int L = D / 8, GROUPS = 256 / L, U = sizeof(IO) + sizeof(GR) > 4 ? 2 : 4;
  const RopeCall& c = a.c;
  const int lane = lane_id(), s = lane % L, group = threadIdx.x / L;
  const int from = (lane & ~(L - 1)) + partner<D>(c, s);
  float wq[8], wk[8], dwq[8], dwk[8];
  weights<IO>(c, c.wq, 8 * s, wq);
  weights<IO>(c, c.wk, 8 * s, wk);
  float f[8];
  frequencies(c, s, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) dwq[i] = dwk[i] = 0.f;
  for (int64_t unit = (int64_t)blockIdx.x * GROUPS + group; unit < a.units; unit += (int64_t)gridDim.x * GROUPS) {
    const int64_t t = a.parts == 1 ? unit : (uint32_t)unit / (uint32_t)a.parts;
    const int h0 = (int)(unit - t * a.parts) * a.heads, h1 = min(h0 + a.heads, c.H + c.Hkv);
    const Turn turn = turn_of<D>(c, s, f, c.positions[t]);
    const IO* q = (const IO*)c.q + t * c.q_stride + 8 * s;
    const IO* k = (const IO*)c.k + t * c.k_stride + 8 * s;
    for (int h = h0; h < h1; h += U) {
      Raw<IO> x[U];
      Raw<GR> y[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = min(h + u, h1 - 1);
        x[u] = load8<true>(i < c.H ? q + (int64_t)i * D : k + (int64_t)(i - c.H) * D);
        y[u] = load8<true>(i < c.H ? (const GR*)c.dq_out + (t * c.H + i) * D + 8 * s
                             : (const GR*)c.dk_out + (t * c.Hkv + i - c.H) * D + 8 * s);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = h + u;
        if (i >= h1) break;
        const bool key = i >= c.H;
        const Raw<GR> yp = others(y[u], c.interleaved, from, 8 * s < c.rot);
        float g[8];  // R^T dy: the same turn backwards
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = fmaf(y[u].get(e), turn.cos[e], -yp.get(e) * turn.sin[e]);
        if (c.norm) {
          float sum = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) sum = fmaf(x[u].get(e), x[u].get(e), sum);
          const float r = 1.f / sqrtf(row_sum<L>(sum) * (1.f / D) + c.eps);
          float dot = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float n = x[u].get(e) * r;
            if (key) dwk[e] = fmaf(g[e], n, dwk[e]);
            else dwq[e] = fmaf(g[e], n, dwq[e]);
            g[e] *= key ? wk[e] : wq[e];
            dot = fmaf(g[e], n, dot);
          }
          dot = row_sum<L>(dot) * (1.f / D);
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] = r * fmaf(-x[u].get(e) * r, dot, g[e]);
        }
        if (!key) store8<true>((GR*)c.dq + (t * c.H + i) * D + 8 * s, g);
        else store8<true>((GR*)c.dk + (t * c.Hkv + i - c.H) * D + 8 * s, g);
      }
    }
  }
  if (!a.sums) return;
  __shared__ float part[GROUPS][2 * D + 1];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    part[group][8 * s + e] = dwq[e];
    part[group][D + 8 * s + e] = dwk[e];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * D; e += 256) {
    float sum = 0.f;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) sum += part[g][e];
    a.sums[(int64_t)blockIdx.x * 2 * D + e] = sum;
  }
}

// dwq, dwk [D] from n workgroups' sums: 32 columns a workgroup, 32 threads each
__global__ __launch_bounds__(1024) void rope_dw_kernel(const float* sums, int n, int D, float* dwq, float* dwk) {
  __shared__ float part[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x % 32, y = threadIdx.x / 32;
  float sum = 0.f;
#pragma unroll 8
  for (int i = y; i < n; i += 32) sum += sums[(int64_t)i * 2 * D + col];
  part[y][threadIdx.x % 32] = sum;
  __syncthreads();
  if (y == 0) {
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += part[i][threadIdx.x];
    float* out = col < D ? dwq : dwk;
    if (out) out[col < D ? col : col - D] = sum;
  }
}

int64_t cdiv(int64_t x, int64_t y) { return (x + y - 1) / y; }

// A token's heads go to one lane group, which then forms its angles once,
// unless that leaves the chip short of waves.
Args args_of(const RopeCall& c) {
  const int nh = c.H + (c.paged ? 2 : 1) * c.Hkv;
  Args a;
  a.c = c;
  const int64_t groups = (c.paged ? 8192 : 4096) * (512 / c.D);  // lane groups of that many waves
  int64_t parts = std::min<int64_t>(std::max<int64_t>(groups / std::max<int64_t>(c.total, 1), 1), nh);
  a.heads = (int)cdiv(nh, parts);
  a.parts = (int)cdiv(nh, a.heads);
  a.units = c.total * a.parts;
  a.sums = nullptr;
  a.cells = 0, a.kv_heads = 0;
  return a;
}

Args append8_args(const RopeCall& c) {
  RopeCall q = c;
  q.Hkv = 0;
  Args a = args_of(q);
  a.kv_heads = c.Hkv;
  a.cells = c.packed ? (c.total >> 4) + 2 * (int64_t)c.B : (int64_t)c.B * (((int64_t)c.T + 14) / 16 + 1);
  return a;
}
int64_t append8_workgroups(const Args& a) { return a.cells * a.kv_heads + cdiv(a.units, 256 / (a.c.D / 8)); }

template <int D, typename IO, typename OUT> hipError_t forward(const RopeCall& c, hipStream_t stream) {
  if (c.bits8) {
    const Args a = append8_args(c);
    rope_append8_kernel<D, IO><<<dim3((unsigned)append8_workgroups(a)), dim3(256), 0, stream>>>(a);
    return hipGetLastError();
  }
  const Args a = args_of(c);
  const dim3 grid((unsigned)cdiv(a.units, 256 / (D / 8)));
  if (c.paged) rope_kernel<D, IO, OUT, true><<<grid, dim3(256), 0, stream>>>(a);
  else rope_kernel<D, IO, OUT, false><<<grid, dim3(256), 0, stream>>>(a);
  return hipGetLastError();
}

constexpr int BWD_GROUPS = 768;  // workgroups of the backward pass at most: 3 a CU reside

int backward_blocks(const Args& a) { return (int)std::min<int64_t>(cdiv(a.units, 256 / (a.c.D / 8)), BWD_GROUPS); }

template <int D, typename IO, typename GR> hipError_t backward(const RopeCall& c, hipStream_t stream) {
  Args a = args_of(c);
  const int n = backward_blocks(a);
  if (c.dwq || c.dwk) a.sums = static_cast<float*>(c.workspace);
  rope_backward_kernel<D, IO, GR><<<dim3(n), dim3(256), 0, stream>>>(a);
  if (a.sums) rope_dw_kernel<<<dim3(2 * D / 32), dim3(1024), 0, stream>>>(a.sums, n, D, c.dwq, c.dwk);
  return hipGetLastError();
}

template <template <int, typename, typename> class F>
hipError_t dispatch(const RopeCall& c, hipStream_t stream) {
#define JB_ROPE_D(DD)                                                                        \
  case DD:                                                                                   \
    if (c.io == IO_BF16)                                                                     \
      return c.out == IO_BF16 ? F<DD, bf16_t, bf16_t>::run(c, stream) : F<DD, bf16_t, float>::run(c, stream); \
    return c.out == IO_BF16 ? F<DD, float, bf16_t>::run(c, stream) : F<DD, float, float>::run(c, stream)
  switch (c.D) {
    JB_ROPE_D(64);
    JB_ROPE_D(128);
    JB_ROPE_D(256);
  }
#undef JB_ROPE_D
  return hipErrorInvalidValue;
}
template <int D, typename IO, typename OUT> struct Forward {
  static hipError_t run(const RopeCall& c, hipStream_t s) { return forward<D, IO, OUT>(c, s); }
};
template <int D, typename IO, typename OUT> struct Backward {
  static hipError_t run(const RopeCall& c, hipStream_t s) { return backward<D, IO, OUT>(c, s); }
};

}  // namespace

int64_t rope_workgroups(const RopeCall& c) {
  if (c.bits8) return append8_workgroups(append8_args(c));
  return cdiv(args_of(c).units, 256 / (c.D / 8));
}

size_t rope_backward_workspace_bytes(const RopeCall& c) {
  return c.total == 0 ? 0 : (size_t)backward_blocks(args_of(c)) * 2 * c.D * sizeof(float);
}

hipError_t launch_rope(const RopeCall& c, hipStream_t stream) { return dispatch<Forward>(c, stream); }
hipError_t launch_rope_backward(const RopeCall& c, hipStream_t stream) { return dispatch<Backward>(c, stream); }

}  // namespace jb
