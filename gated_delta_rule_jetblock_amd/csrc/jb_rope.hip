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

namespace jb {

namespace {

struct Args {
  RopeCall c;
  int parts, heads;   // head parts a token is cut into, heads a part
  int64_t units;      // tokens x parts
  float* sums;        // backward: [workgroups][2][D]
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
__device__ __forceinline__ void frequencies(const RopeCall& c, int s, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = 0.f;
  if (8 * s < c.rot) {
    const float* p = c.inv_freq + (c.interleaved ? 4 * s : 8 * s < c.rot / 2 ? 8 * s : 8 * s - c.rot / 2);
    const f4u_t u = *reinterpret_cast<const f4u_t*>(p);
    const f4u_t v = c.interleaved ? u : *reinterpret_cast<const f4u_t*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = u[i], f[4 + i] = v[i];
  }
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

template <typename T> __device__ __forceinline__ void weights(const void* w, int e0, float (&out)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) out[i] = 1.f;
  if (w) {
    const Raw<T> r = load8((const T*)w + e0);
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = r.get(i);
  }
}

template <int D, typename IO, typename OUT, bool PAGED>
__global__ __launch_bounds__(256) void rope_kernel(Args a) {
  constexpr int L = D / 8, GROUPS = 256 / L;
  // rows in use, and as many on their way (64K tokens: 4 take 88.9 us, 2 90.9; an
  // append of 13K tokens 34.5 and 35.0, where 2 need fewer registers)
  constexpr int U = PAGED || sizeof(IO) == 4 ? 2 : 4;
  const RopeCall& c = a.c;
  const int lane = lane_id(), s = lane % L, group = threadIdx.x / L;
  const int64_t unit = (int64_t)blockIdx.x * GROUPS + group;
  bool live = unit < a.units;
  // (fewer than 2^31 units where a token has several)
  int64_t t = !live ? 0 : a.parts == 1 ? unit : (uint32_t)unit / (uint32_t)a.parts;
  const int h0 = a.parts == 1 || !live ? 0 : (int)((uint32_t)unit % (uint32_t)a.parts) * a.heads;
  // what does not depend on the token's place is on its way while that is found
  const int nh = c.H + (PAGED ? 2 : 1) * c.Hkv, h1 = min(h0 + a.heads, nh);
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
  weights<IO>(c.wq, 8 * s, wq);
  weights<IO>(c.wq, es, wqp);
  weights<IO>(c.wk, 8 * s, wk);
  weights<IO>(c.wk, es, wkp);
  int row = 0;          // the token's row in its sequence's cache
  int64_t slot = -1;    // and in the pool (element offset of key head 0), or -1
  if constexpr (PAGED) {
    int b;
    int64_t i;
    int T = c.T;  // the sequence's tokens (those behind the first c.T are not taken)
    if (c.packed) {
      // the sequence of the workgroup's first token, then on from there
      const int64_t t0 = (int64_t)blockIdx.x * GROUPS / a.parts;
      int n = 0;
      for (int k = 0; k < c.B; k += 256) {
        const int j = k + threadIdx.x;
        const int m = __syncthreads_count(j < c.B && c.cu_seqlens[j] <= t0);
        n += m;
        if (m < 256) break;
      }
      b = max(n - 1, 0);
      while (b + 1 < c.B && c.cu_seqlens[b + 1] <= t) ++b;
      int64_t tok0;
      clamp_span(c.cu_seqlens[b], c.cu_seqlens[b + 1], 0x7fffffff, c.total, tok0, T);
      i = t - tok0;
      live = live && i >= 0 && i < min(T, c.T);
    } else {
      b = (int)((uint32_t)t / (uint32_t)c.T);
      i = t - (int64_t)b * c.T;
    }
    const int pshift = __builtin_ctz((unsigned)c.page);
    const int cap = (int)min((int64_t)c.max_pages << pshift, (int64_t)0x7fffffff);
    row = min(max(c.kv_lens[b], 0), cap) - T + (int)i;
    if (live && row >= 0) {
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

template <int D, typename IO, typename GR>
__global__ __launch_bounds__(256, 3) void rope_backward_kernel(Args a) {
  constexpr int L = D / 8, GROUPS = 256 / L, U = sizeof(IO) + sizeof(GR) > 4 ? 2 : 4;
  const RopeCall& c = a.c;
  const int lane = lane_id(), s = lane % L, group = threadIdx.x / L;
  const int from = (lane & ~(L - 1)) + partner<D>(c, s);
  float wq[8], wk[8], dwq[8], dwk[8];
  weights<IO>(c.wq, 8 * s, wq);
  weights<IO>(c.wk, 8 * s, wk);
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
  return a;
}

template <int D, typename IO, typename OUT> hipError_t forward(const RopeCall& c, hipStream_t stream) {
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
  return cdiv(args_of(c).units, 256 / (c.D / 8));
}

size_t rope_backward_workspace_bytes(const RopeCall& c) {
  return c.total == 0 ? 0 : (size_t)backward_blocks(args_of(c)) * 2 * c.D * sizeof(float);
}

hipError_t launch_rope(const RopeCall& c, hipStream_t stream) { return dispatch<Forward>(c, stream); }
hipError_t launch_rope_backward(const RopeCall& c, hipStream_t stream) { return dispatch<Backward>(c, stream); }

}  // namespace jb
