// jb_blocks.hip -- attention over selected pages of the cache: the pages' mean keys and
// their scores for each new token, the selection by score, and the lists that the
// attention kernels (jb_attn_core.h) walk.
//
// Token i of a sequence sits at cache row p and sees pages 0 .. p / page.  With mean_j the
// mean of the rows that page j holds of a key head (fp32),
//     score_j = max over the key head's query heads of q . mean_j,
// and of the pages it sees the token reads its first and last ones and the best others.
#include <type_traits>

#include "jb_attn.h"
#include "jb_device.h"
#include "jb_e4m3.h"

namespace jb {

namespace {

typedef unsigned int u4_t __attribute__((ext_vector_type(4)));

struct Args {
  BlockCall c;
  int G, pshift;
  int64_t slots;  // places for a sequence's pages (means) or token tiles (scores)
};

// a sequence's tokens (the first c.T of them) and the cache row of the first one, all
// clamped to the tensors (they come from device memory)
struct Seq {
  int64_t tok0;
  int T, row0;
};
__device__ __forceinline__ Seq seq_of(const Args& a, int b) {
  const BlockCall& c = a.c;
  Seq s;
  int all = c.T;
  s.tok0 = (int64_t)b * c.T;
  if (c.cu_seqlens) clamp_span(c.cu_seqlens[b], c.cu_seqlens[b + 1], 0x7fffffff, c.total, s.tok0, all);
  s.T = min(all, c.T);
  const int cap = (int)min((int64_t)c.max_pages << a.pshift, (int64_t)0x7fffffff);
  s.row0 = min(max(c.kv_lens[b], 0), cap) - all;
  return s;
}

// Place `slot` among the sequences': sequence b's start at per b, or packed at
// (cu[b] >> shift) + more b, which leaves room for all of them and never decreases.
// All threads of the workgroup call this together.
__device__ __forceinline__ int seq_at(const Args& a, int64_t slot, int shift, int more, int64_t per, int64_t& nth) {
  const BlockCall& c = a.c;
  if (!c.cu_seqlens) {
    const int b = (int)((uint32_t)slot / (uint32_t)per);  // (both below 2^31)
    nth = slot - b * per;
    return b;
  }
  auto base = [&](int j) {
    return (min(max((int64_t)c.cu_seqlens[j], (int64_t)0), c.total) >> shift) + more * (int64_t)j;
  };
  int n = 0;
  for (int k = 0; k < c.B; k += blockDim.x) {
    const int j = k + threadIdx.x;
    const int m = __syncthreads_count(j < c.B && base(j) <= slot);
    n += m;
    if (m < (int)blockDim.x) break;
  }
  const int b = max(n - 1, 0);
  nth = slot - base(b);
  return b;
}

// Sequence of token t and its place in it; false: no sequence owns it (or it is one of
// those behind the first c.T).  t0: the workgroup's first token, the same for all threads.
__device__ __forceinline__ bool token_at(const Args& a, int64_t t0, int64_t t, int& b, Seq& s, int& i) {
  const BlockCall& c = a.c;
  int64_t nth;
  b = seq_at(a, t0, 0, 0, max(c.T, 1), nth);
  if (c.cu_seqlens) {
    while (b + 1 < c.B && c.cu_seqlens[b + 1] <= t) ++b;
  } else {
    b = (int)((uint32_t)t / (uint32_t)max(c.T, 1));
  }
  s = seq_of(a, b);
  const int64_t at = t - s.tok0;
  i = (int)at;
  return at >= 0 && at < s.T;
}

// 8 values of a cache row as floats
template <typename KV> __device__ __forceinline__ void row8(const void* p, uint32_t e, float (&x)[8]) {
  if constexpr (sizeof(KV) == 1) {
    const uint2 u = *static_cast<const uint2*>(p);
    const float4 lo = floats_of_e4m3(u.x, e), hi = floats_of_e4m3(u.y, e);
    x[0] = lo.x, x[1] = lo.y, x[2] = lo.z, x[3] = lo.w, x[4] = hi.x, x[5] = hi.y, x[6] = hi.z, x[7] = hi.w;
  } else if constexpr (sizeof(KV) == 2) {
    const u4_t u = *static_cast<const u4_t*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(i & 1 ? u[i >> 1] & 0xffff0000u : u[i >> 1] << 16);
  } else {
    const float4 lo = static_cast<const float4*>(p)[0], hi = static_cast<const float4*>(p)[1];
    x[0] = lo.x, x[1] = lo.y, x[2] = lo.z, x[3] = lo.w, x[4] = hi.x, x[5] = hi.y, x[6] = hi.z, x[7] = hi.w;
  }
}

// Mean key of the first `held` rows of page pid: a workgroup's D / 8 lanes a row, summed in a
// fixed order (a lane group's rows in order, then the groups); threads 0 .. D - 1 have it.
// part: GROUPS x (D + 1) floats of LDS.
template <int D> constexpr int mean_floats = 256 / (D / 8) * (D + 1);
template <int D, typename KV>
__device__ __forceinline__ float mean_key(const Args& a, int pid, int head, int held, float* lds) {
  constexpr int L = D / 8, GROUPS = 256 / L;
  float(*const part)[D + 1] = reinterpret_cast<float(*)[D + 1]>(lds);
  const BlockCall& c = a.c;
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const int64_t row0 = (int64_t)head << a.pshift;
  const char* k = (const char*)c.k_cache + (pid * c.page_stride + row0 * D + 8 * lane) * (int64_t)sizeof(KV);
  const uint8_t* e = sizeof(KV) == 1 ? c.k_scales + pid * c.scale_stride + (row0 >> 4) : nullptr;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int r = group; r < held; r += GROUPS) {
    float x[8];
    row8<KV>(k + (int64_t)r * D * sizeof(KV), sizeof(KV) == 1 ? e[r >> 4] : 0u, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += x[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) part[group][8 * lane + i] = sum[i];
  __syncthreads();
  float total = 0.f;
  if (threadIdx.x < D) {
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) total += part[g][threadIdx.x];
  }
  return total / (float)held;
}

// Mean key of every page that holds new tokens, over the rows that it holds by now: a
// workgroup a page and key head.
template <int D, typename KV>
__global__ __launch_bounds__(256) void block_means_kernel(Args a) {
  const BlockCall& c = a.c;
  const uint32_t slot = blockIdx.x / (uint32_t)c.Hkv;
  const int head = blockIdx.x - slot * (uint32_t)c.Hkv, page = 1 << a.pshift;
  int64_t nth;
  const int b = seq_at(a, slot, a.pshift, 2, ((int64_t)c.T + page - 2) / page + 1, nth);
  const Seq s = seq_of(a, b);
  const int end = s.row0 + s.T;
  const int64_t j = (max(s.row0, 0) >> a.pshift) + nth;  // the page's place in the sequence
  if (nth < 0 || s.T == 0 || j << a.pshift >= end) return;
  const int pid = c.page_table[(int64_t)b * c.max_pages + j];
  if (pid < 0 || pid >= c.num_pages) return;
  const int held = (int)min((int64_t)end - (j << a.pshift), (int64_t)page);
  __shared__ float lds[mean_floats<D>];
  const float mean = mean_key<D, KV>(a, pid, head, held, lds);
  if (threadIdx.x < D) c.means[((int64_t)pid * c.Hkv + head) * D + threadIdx.x] = mean;
}

// the larger of two scores; NaN stays
__device__ __forceinline__ float larger(float m, float x) { return x > m || x != x ? x : m; }

// A score by plain products (mean: NULL for zeros), where the sum over a mean's parts is NaN:
// an infinite query times a part that is 0, or the parts of an infinite mean, are NaN
// where the product itself need not be.  (A call of its own: it is rare, and inline it took
// the registers of the loops.)
template <int D> __device__ __attribute__((noinline)) float plain_score(const bf16_t* q, const float* mean, int G) {
  float best = -INFINITY;
  for (int h = 0; h < G; ++h) {
    float x = 0.f;
    for (int d = 0; d < D; ++d) x = fmaf(__uint_as_float((uint32_t)q[h * D + d] << 16), mean ? mean[d] : 0.f, x);
    best = h ? larger(best, x) : x;
  }
  return best;
}

// The means of NB x 16 pages as operands: lane (page lane % 16, group g) has d = 8 g + e of
// every 32, each value as three bf16 parts: hi + mid + lo are its 24 bits, so products with
// bf16 queries are exact and their sums fp32's.
// They come by way of LDS (a region of 16 D floats for each wave): lanes that lie next to each
// other read one row, where an operand's neighbouring lanes are of different rows and cost
// the vector memory unit a cycle each (a chunk of 2K tokens on 64K rows with the queries
// read so too: 33 us, of which 24 were that).
typedef __attribute__((address_space(3))) u4_t lds_u4;
typedef __attribute__((address_space(3))) char lds_char;

template <int D, int NB> struct Means {
  static constexpr int STEPS = D / 32, LPR = D / 4, RPI = 64 / LPR, LOADS = 16 / RPI;  // lanes a row, rows a load
  float4 x[NB][LOADS];
  bf16x8_t part[NB][STEPS][3];
  // pid[n]: lane n16's page of 16 n + n16, -1 for zeros
  __device__ __forceinline__ void fetch(const Args& a, int head, const int (&pid)[NB]) {
    const int lane = lane_id();
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int from = __shfl(pid[n], i * RPI + lane / LPR, WAVE);
        const float4 v = reinterpret_cast<const float4*>(a.c.means + ((int64_t)max(from, 0) * a.c.Hkv + head) * D)[lane % LPR];
        x[n][i] = from >= 0 ? v : make_float4(0.f, 0.f, 0.f, 0.f);
      }
  }
  // row `row` of the 16 n is `fresh` instead (none: -1)
  __device__ __forceinline__ void split(lds_char* at, const float* fresh, int row) {
    const int lane = lane_id(), n16 = lane & 15, g = lane >> 4;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // what was there is read
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int r = i * RPI + lane / LPR, piece = lane % LPR;
        *(lds_u4*)(at + r * D * 4 + ((piece ^ r) << 4)) = __builtin_bit_cast(u4_t, x[n][i]);
      }
      if (fresh && row >> 4 == n && lane < LPR) {
        const int r = row & 15;
        *(lds_u4*)(at + r * D * 4 + ((lane ^ r) << 4)) = __builtin_bit_cast(u4_t, reinterpret_cast<const float4*>(fresh)[lane]);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
      for (int k = 0; k < STEPS; ++k) {
        const float4 lo = __builtin_bit_cast(float4, *(const lds_u4*)(at + n16 * D * 4 + (((2 * g + 8 * k) ^ n16) << 4)));
        const float4 hi = __builtin_bit_cast(float4, *(const lds_u4*)(at + n16 * D * 4 + (((2 * g + 8 * k + 1) ^ n16) << 4)));
        const float y[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const __bf16 a = (__bf16)y[e];
          const float r = y[e] - (float)a;
          const __bf16 b = (__bf16)r;
          part[n][k][0][e] = a, part[n][k][1][e] = b, part[n][k][2][e] = (__bf16)(r - (float)b);
        }
      }
    }
  }
};

// Scores of tokens of longer chunks, bf16: 16 tokens by 16 pages at a time on matrix cores
// (rows are tokens, columns pages), one product for each query head, their maximum taken in
// the accumulators.  A wave keeps the means of 2 x 16 pages in registers, split once, and
// walks `tiles` tiles of 2 x 16 tokens, the next head's queries on their way while these are
// used; a workgroup takes 4 times as many pages.  2K tokens of 12 heads on 2 at the end of
// 64K rows, pages of 64: 26.6-27.6 us with the launch that forms the means (5); the
// products are 8 of it at the matrix cores' nominal rate and 15.5 at the one that the library's product
// reaches, the scores' bytes 3.
constexpr int PAGES = 128;  // of a workgroup

template <int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void block_scores_kernel(Args a, uint32_t groups, int tiles) {
  constexpr int STEPS = D / 32, TM = 2, NB = 2;
  const BlockCall& c = a.c;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, n16 = lane & 15, g = lane >> 4;
  const uint32_t per = (uint32_t)c.Hkv * groups, place = blockIdx.x / per, rest = blockIdx.x - place * per;
  const int head = rest / groups, j0 = (int)(rest - head * groups) * PAGES + wave * 16 * NB;
  constexpr int PR = D / 8, PER = 32 * PR / 256;  // 16-byte pieces of a row; of 32 rows a thread
  __shared__ __attribute__((aligned(16))) char qs[2][32 * D * 2];  // a head's queries, and the next one's
  __shared__ __attribute__((aligned(16))) char ms[4][16 * D * 4];
  lds_char* const lq = (lds_char*)qs[0];
  auto place_of = [](int r, int piece) { return r * D * 2 + ((piece ^ (PR < 16 ? (r >> 1) & 7 : r & 15)) << 4); };
  Means<D, NB> m;
  int held = -1;  // the sequence whose means these are
  for (int k = 0; k < tiles; ++k) {
    const int64_t slot = (int64_t)place * tiles + k;
    if (slot >= a.slots) break;
    int64_t nth;
    const int b = seq_at(a, slot, 5, 1, ((int64_t)c.T + 31) / 32, nth);
    const Seq s = seq_of(a, b);
    if (nth < 0 || nth * 32 >= s.T) continue;  // (the same for all waves)
    const int i0 = (int)nth * 32, live = min(s.T - i0, 32);
    const int seen = min(((s.row0 + i0 + live - 1) >> a.pshift) + 1, c.max_pages);  // pages that some token sees (or fewer than 1)
    f4_t best[TM][NB];
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
      for (int n = 0; n < NB; ++n) best[t][n] = f4_t{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (j0 - wave * 16 * NB < seen) {  // some wave's pages are seen
      const bf16_t* q[PER];
      u4_t next[PER];
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const int e = u * 256 + threadIdx.x;
        q[u] = (const bf16_t*)c.q + (s.tok0 + i0 + min(e / PR, live - 1)) * c.q_stride + (int64_t)head * a.G * D + e % PR * 8;
        next[u] = *reinterpret_cast<const u4_t*>(q[u]);
      }
      auto put = [&](int h) {
#pragma unroll
        for (int u = 0; u < PER; ++u) {
          const int e = u * 256 + threadIdx.x;
          *(lds_u4*)(lq + (h & 1) * 32 * D * 2 + place_of(e / PR, e % PR)) = next[u];
          next[u] = *reinterpret_cast<const u4_t*>(q[u] + (int64_t)min(h + 1, a.G - 1) * D);
        }
      };
      if (held != b) {
        // (later tiles of the sequence see more pages: all that may ever be seen are taken)
        const int last = min((max(s.row0 + s.T, 1) - 1) >> a.pshift, c.max_pages - 1);
        int pid[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const int j = j0 + 16 * n + n16;
          pid[n] = j <= last ? c.page_table[(int64_t)b * c.max_pages + j] : -1;
          if (pid[n] >= c.num_pages) pid[n] = -1;
        }
        m.fetch(a, head, pid);
        m.split((lds_char*)ms[wave], nullptr, -1);
        held = b;
      }
      __syncthreads();  // (the last tile's queries are read)
      put(0);
      for (int h = 0; h < a.G; ++h) {
        __syncthreads();
        if (h + 1 < a.G) put(h + 1);
        const lds_char* const at = lq + (h & 1) * 32 * D * 2;
        f4_t x[TM][NB];
#pragma unroll
        for (int t = 0; t < TM; ++t)
#pragma unroll
          for (int n = 0; n < NB; ++n) x[t][n] = zero4();
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          bf16x8_t f[TM];
#pragma unroll
          for (int t = 0; t < TM; ++t)
            f[t] = __builtin_bit_cast(bf16x8_t, *(const lds_u4*)(at + place_of(16 * t + n16, 4 * i + g)));
#pragma unroll
          for (int part = 0; part < 3; ++part)
#pragma unroll
            for (int t = 0; t < TM; ++t)
#pragma unroll
              for (int n = 0; n < NB; ++n)
                x[t][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[t], m.part[n][i][part], x[t][n], 0, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < TM; ++t)
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) best[t][n][e] = h ? larger(best[t][n][e], x[t][n][e]) : x[t][n][e];
      }
    }
    if (j0 >= c.max_pages) continue;
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 16 * t + 4 * g + e, own = (s.row0 + i0 + i) >> a.pshift;
        float* out = c.scores + ((s.tok0 + i0 + i) * c.Hkv + head) * c.max_pages;
        if (i < live)
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            const int j = j0 + 16 * n + n16;
            if (j >= c.max_pages) continue;
            float x = j <= own ? best[t][n][e] : -INFINITY;
            if (x != x) {
              const int pid = c.page_table[(int64_t)b * c.max_pages + j];
              x = plain_score<D>((const bf16_t*)c.q + (s.tok0 + i0 + i) * c.q_stride + (int64_t)head * a.G * D,
                                 pid >= 0 && pid < c.num_pages ? c.means + ((int64_t)pid * c.Hkv + head) * D : nullptr, a.G);
            }
            out[j] = x;
          }
      }
  }
}

// Decode (T = 1), bf16: rows are 16 query heads of the one token, columns 16 pages; the
// maximum over the rows is taken across the lanes.  The one page that holds the token is
// averaged by the workgroup that scores it, so the step is one launch.  Bound by what it
// waits for: the length and the page indices, then the means, a wave's 32 pages at once.  64
// sequences of up to 64K rows, 12 heads on 2, pages of 64 (35 MB): 14.4-15.5 us, as many in a
// captured graph; all of 64K rows (67 MB) 19.3, 16 of them 7.1.
template <int D, typename KV>
__global__ __launch_bounds__(256, D == 64 ? 5 : D == 128 ? 3 : 2) void block_scores_one_kernel(Args a, uint32_t groups) {
  constexpr int STEPS = D / 32, NB = 2;
  const BlockCall& c = a.c;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, n16 = lane & 15, g = lane >> 4;
  const uint32_t per = (uint32_t)c.Hkv * groups, t = blockIdx.x / per, rest = blockIdx.x - t * per;
  const int head = rest / groups, group = (int)(rest - head * groups), j0 = group * PAGES + wave * 32;
  int b = t, i = 0;
  Seq s;
  if (c.cu_seqlens) {
    if (!token_at(a, t, t, b, s, i)) return;  // (the same for all threads)
  } else {
    s = seq_of(a, b);
  }
  const int* table = c.page_table + (int64_t)b * c.max_pages;
  int pid[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) pid[n] = j0 + 16 * n + n16 < c.max_pages ? table[j0 + 16 * n + n16] : -1;
  const bf16_t* q = (const bf16_t*)c.q + t * c.q_stride + (int64_t)head * a.G * D + 8 * g;
  u4_t f[STEPS];
#pragma unroll
  for (int k = 0; k < STEPS; ++k) f[k] = *reinterpret_cast<const u4_t*>(q + (int64_t)min(n16, a.G - 1) * D + 32 * k);
  const int p = s.row0 + i, own = p >> a.pshift;  // (negative: no page)
  Means<D, NB> m;
#pragma unroll
  for (int n = 0; n < NB; ++n)
    if (j0 + 16 * n + n16 >= own || pid[n] >= c.num_pages) pid[n] = -1;  // (the own page's is formed here)
  if (j0 <= own) m.fetch(a, head, pid);
  __shared__ __attribute__((aligned(16))) float fresh[D];
  __shared__ __attribute__((aligned(16))) char ms[4][16 * D * 4];
  static_assert(mean_floats<D> * 4 <= sizeof(ms), "the mean's sums fit");
  bool formed = false;
  if (own >= 0 && own / PAGES == group) {
    const int mine = table[own];
    if (mine >= 0 && mine < c.num_pages) {
      const float mean = mean_key<D, KV>(a, mine, head, (p & ((1 << a.pshift) - 1)) + 1, (float*)ms);
      if (threadIdx.x < D) {
        c.means[((int64_t)mine * c.Hkv + head) * D + threadIdx.x] = mean;
        fresh[threadIdx.x] = mean;
      }
      __syncthreads();
      formed = true;
    }
  }
  float best[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) best[n] = -INFINITY;
  if (j0 <= own) {
    m.split((lds_char*)ms[wave], formed ? fresh : nullptr, own - j0);
    for (int h = 0; h < a.G; h += 16) {
      if (h)
#pragma unroll
        for (int k = 0; k < STEPS; ++k) f[k] = *reinterpret_cast<const u4_t*>(q + (int64_t)min(h + n16, a.G - 1) * D + 32 * k);
      f4_t x[NB];
#pragma unroll
      for (int n = 0; n < NB; ++n) x[n] = zero4();
#pragma unroll
      for (int k = 0; k < STEPS; ++k)
#pragma unroll
        for (int part = 0; part < 3; ++part)
#pragma unroll
          for (int n = 0; n < NB; ++n)
            x[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, f[k]), m.part[n][k][part], x[n], 0, 0, 0);
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        float v = larger(larger(x[n][0], x[n][1]), larger(x[n][2], x[n][3]));  // (rows past the heads repeat the last)
        v = larger(v, __shfl_xor(v, 16, WAVE));
        v = larger(v, __shfl_xor(v, 32, WAVE));
        best[n] = h ? larger(best[n], v) : v;
      }
    }
  }
  // lanes 0 .. 31 write the wave's 32 pages
  const int j = j0 + lane;
  if (lane < 32 && j < c.max_pages) {
    float x = j <= own ? (lane < 16 ? best[0] : best[1]) : -INFINITY;
    if (x != x) {
      const int page = table[j];
      const float* mean = page >= 0 && page < c.num_pages ? c.means + ((int64_t)page * c.Hkv + head) * D : nullptr;
      x = plain_score<D>(q - 8 * g, j == own && formed ? fresh : mean, a.G);
    }
    c.scores[((int64_t)t * c.Hkv + head) * c.max_pages + j] = x;
  }
}

// The same in fp32: 16 tokens and 16 pages at a time with fp32 products, TM x 16 tokens and
// 2 x 16 pages a wave.
template <int D>
__global__ __launch_bounds__(256) void block_scores_f32_kernel(Args a, uint32_t groups) {
  constexpr int TM = 2, NB = 2, TOKENS = 16 * TM;
  const BlockCall& c = a.c;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, n16 = lane & 15, g = lane >> 4;
  const uint32_t per = (uint32_t)c.Hkv * groups, slot = blockIdx.x / per, rest = blockIdx.x - slot * per;
  const int head = rest / groups, j0 = (int)(rest - head * groups) * PAGES + wave * 16 * NB;
  int64_t nth;
  const int b = seq_at(a, slot, 5, 1, ((int64_t)c.T + TOKENS - 1) / TOKENS, nth);
  static_assert(TOKENS == 32, "2^5 tokens a slot");
  const Seq s = seq_of(a, b);
  if (nth < 0 || nth * TOKENS >= s.T || j0 >= c.max_pages) return;
  const int i0 = (int)nth * TOKENS, live = min(s.T - i0, TOKENS);
  const int seen = ((s.row0 + i0 + live - 1) >> a.pshift) + 1;  // pages that some token sees (negative rows: none)
  const int* table = c.page_table + (int64_t)b * c.max_pages;
  f4_t best[TM][NB];
#pragma unroll
  for (int t = 0; t < TM; ++t)
#pragma unroll
    for (int n = 0; n < NB; ++n) best[t][n] = f4_t{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  if (j0 < seen) {
    f4_t m[NB][D / 16];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int j = j0 + 16 * n + n16;
      const int pid = j < min(seen, c.max_pages) ? table[j] : -1;
      const bool ok = pid >= 0 && pid < c.num_pages;
      const float* mean = c.means + ((int64_t)(ok ? pid : 0) * c.Hkv + head) * D + 4 * g;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const f4_t v = *reinterpret_cast<const f4_t*>(mean + 16 * k);
#pragma unroll
        for (int e = 0; e < 4; ++e) m[n][k][e] = ok ? v[e] : 0.f;
      }
    }
    for (int h = 0; h < a.G; ++h) {
#pragma unroll
      for (int t = 0; t < TM; ++t) {
        if (t && 16 * t >= live) break;
        const int i = i0 + min(16 * t + n16, live - 1);
        const float* q = (const float*)c.q + (s.tok0 + i) * c.q_stride + (int64_t)(head * a.G + h) * D + 4 * g;
        f4_t x[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) x[n] = zero4();
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const f4_t f = *reinterpret_cast<const f4_t*>(q + 16 * k);
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int n = 0; n < NB; ++n) x[n] = __builtin_amdgcn_mfma_f32_16x16x4f32(f[e], m[n][k][e], x[n], 0, 0, 0);
        }
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) best[t][n][e] = h ? larger(best[t][n][e], x[n][e]) : x[n][e];
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TM; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 16 * t + 4 * g + e;
      if (i >= live) continue;
      const int own = (s.row0 + i0 + i) >> a.pshift;
      float* out = c.scores + ((s.tok0 + i0 + i) * c.Hkv + head) * c.max_pages;
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const int j = j0 + 16 * n + n16;
        if (j < c.max_pages) out[j] = j <= own ? best[t][n][e] : -INFINITY;
      }
    }
}

// Selection by a search for the count-th largest score, bit by bit from the top: a row's
// scores stay in registers as whole numbers in the scores' order, V a lane, and a step
// counts those that reach a candidate (a compare, a scalar bit count).  Once at most 64 are
// undecided they are gathered, one a lane, and the other steps cost one compare each.  W waves
// a row; with one the row needs no barrier.  Places are ascending: lane l of wave w has pages
// (w V + v) 64 + l.
// With at most 64 to select and one wave a row the search is shorter (below): 1 row of 1024
// pages 4.2 us, 4096 rows 8.0; by the steps over all scores 7.6 and 14.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x != x ? -INFINITY : x + 0.f);  // (-0 as 0)
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <int W, int V>
__global__ __launch_bounds__(W == 1 ? 256 : W * 64) void block_select_kernel(Args a) {
  constexpr int ROWS = W == 1 ? 4 : 1;  // rows a workgroup
  const BlockCall& c = a.c;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, w = W == 1 ? 0 : wave;
  // (fewer than 2^24 rows)
  const uint32_t rows = (uint32_t)(c.total * c.Hkv), row0 = blockIdx.x * ROWS, row = row0 + (W == 1 ? wave : 0);
  const uint32_t t = min(row, rows - 1) / (uint32_t)c.Hkv;
  const int at = w * V * 64 + lane;
  // the scores are on their way while the token's place is found
  const float* x = c.scores_in + (int64_t)min(row, rows - 1) * c.max_pages;
  float score[V];
#pragma unroll
  for (int v = 0; v < V; ++v) score[v] = x[min(at + 64 * v, c.max_pages - 1)];
  int b, i;
  Seq s;
  const bool live = token_at(a, row0 / (uint32_t)c.Hkv, t, b, s, i) && row < rows;
  if (!live) return;  // (with W > 1 the workgroup's only row)
  const int own = __builtin_amdgcn_readfirstlane((s.row0 + i) >> a.pshift);  // (of a negative row negative: it sees no page)
  const int nv = min(own + 1, c.max_pages), count = c.count;
  int* const out = c.blocks + (int64_t)row * count;
  if (nv <= count) {  // all of them
    for (int j = W == 1 ? lane : (int)threadIdx.x; j < count; j += W * 64) out[j] = j < nv ? j : -1;
    return;
  }
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int j = at + 64 * v;
    key[v] = order_of(score[v]);
    const int j0 = at - lane + 64 * v;  // (the same for the wave: most of its rows of 64 hold no exception)
    if (j0 < c.first || j0 + 63 > own - c.recent)
      key[v] = j >= nv ? 0u : j < c.first || j > own - c.recent ? 0xffffffffu : key[v];
  }
  __shared__ int2 counts[2][W];
  __shared__ uint32_t few[ROWS][64];
  // the sums of the waves' x and y (scalars of each), and of those before this one
  int turn = 0;
  auto over_waves = [&](int x, int y, int2& before) {
    before = make_int2(0, 0);
    if constexpr (W == 1) return make_int2(x, y);
    if (lane == 0) counts[turn & 1][w] = make_int2(x, y);
    __syncthreads();
    int2 sum = make_int2(0, 0);
#pragma unroll
    for (int u = 0; u < W; ++u) {
      const int2 n = counts[turn & 1][u];
      sum.x += n.x, sum.y += n.y;
      if (u < w) before.x += n.x, before.y += n.y;
    }
    ++turn;
    return sum;
  };
  const uint64_t below = (1ull << lane) - 1;
  if (W == 1 && count <= 64) {
    // The count-th largest of the lanes' largest is reached by at least `count` scores, and
    // by few more: where those are at most 64, the rest is one score a lane.
    uint32_t most = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) most = max(most, key[v]);
    auto nth = [&](uint32_t x, int& n) {  // the largest t that `count` of x reach, and how many do (n: at t = 0)
      uint32_t t = 0;
      for (int bit = 31; bit >= 0 && n != count; --bit) {
        const int m = __builtin_popcountll(__builtin_amdgcn_ballot_w64(x >= (t | 1u << bit)));
        if (m >= count) t |= 1u << bit, n = m;
      }
      return t;
    };
    int n = 64;
    const uint32_t low = max(nth(most, n), 1u);
    n = 0;
    uint64_t all[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      all[v] = __builtin_amdgcn_ballot_w64(key[v] >= low);
      n += __builtin_popcountll(all[v]);
    }
    if (n <= 64) {
      __shared__ uint2 list[ROWS][64];
      int place = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (all[v]) {
          if (key[v] >= low) list[wave][place + __builtin_popcountll(all[v] & below)] = make_uint2(key[v], at + 64 * v);
          place += __builtin_popcountll(all[v]);
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      const uint2 one = lane < n ? list[wave][lane] : make_uint2(0u, 0u);
      const uint32_t t = nth(one.x, n);
      const uint64_t eq = __builtin_amdgcn_ballot_w64(one.x == t);
      const int more = __builtin_popcountll(__builtin_amdgcn_ballot_w64(one.x > t));
      const bool take = one.x > t || (one.x == t && more + __builtin_popcountll(eq & below) < count);
      const uint64_t taken = __builtin_amdgcn_ballot_w64(take);
      if (take) out[__builtin_popcountll(taken & below)] = one.y;
      return;
    }
  }
  int2 before;
  // `reach` scores reach `low`, at least `count`; `above` reach what it may still grow to, fewer
  uint32_t low = 0;
  int reach = nv, above = 0, bit = 31;
  for (; bit >= 0 && reach != count && reach - above > 64; --bit) {
    const uint32_t t = low | 1u << bit;
    int n = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) n += __builtin_popcountll(__builtin_amdgcn_ballot_w64(key[v] >= t));
    n = over_waves(n, 0, before).x;
    if (n >= count) low = t, reach = n;
    else above = n;
  }
  if (bit >= 0 && reach != count) {
    // the undecided ones share the bits above `bit`, and only those
    const uint32_t top = bit == 31 ? 0u : low >> (bit + 1);
    int n = 0, mine = 0;
    auto undecided = [&](int v) { return key[v] && (bit == 31 || key[v] >> (bit + 1) == top); };
    if constexpr (W > 1) {
#pragma unroll
      for (int v = 0; v < V; ++v) mine += __builtin_popcountll(__builtin_amdgcn_ballot_w64(undecided(v)));
      over_waves(mine, 0, before);
      n = before.x;
    }
    uint32_t* const list = few[W == 1 ? wave : 0];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool is = undecided(v);
      const uint64_t all = __builtin_amdgcn_ballot_w64(is);
      if (all) {
        if (is) list[n + __builtin_popcountll(all & below)] = key[v];
        n += __builtin_popcountll(all);
      }
    }
    if constexpr (W > 1) __syncthreads();
    else asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const uint32_t one = lane < reach - above ? list[lane] : 0u;
    const int sure = above;
    for (; bit >= 0 && reach != count; --bit) {
      const uint32_t t = low | 1u << bit;
      const int n = sure + __builtin_popcountll(__builtin_amdgcn_ballot_w64(one >= t));
      if (n >= count) low = t, reach = n;
      else above = n;
    }
  }
  // those above `low`, and of those equal to it the first ones
  int need = 0x7fffffff, taken = 0, equals = 0;  // equal ones to take; taken and equal ones before this wave's
  if (reach != count) need = count - above;
  if constexpr (W > 1) {
    int more = 0, same = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      more += __builtin_popcountll(__builtin_amdgcn_ballot_w64(key[v] > low));
      same += __builtin_popcountll(__builtin_amdgcn_ballot_w64(key[v] == low));
    }
    over_waves(more, same, before);
    equals = before.y;
    taken = before.x + min(equals, need);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    uint64_t all = __builtin_amdgcn_ballot_w64(key[v] >= low);
    if (all) {
      const uint64_t eq = __builtin_amdgcn_ballot_w64(key[v] == low);
      const bool take = key[v] > low || (key[v] == low && equals + __builtin_popcountll(eq & below) < need);
      all = __builtin_amdgcn_ballot_w64(take);
      if (take) out[taken + __builtin_popcountll(all & below)] = at + 64 * v;
      taken += __builtin_popcountll(all);
      equals += __builtin_popcountll(eq);
    }
  }
}

// The pages of every (token, key head), one wave each, as a cache of their own: page
// indices in order and the rows seen.  An entry counts if it is a page that the token sees
// and larger than every one before it; -1 rows: no sequence owns the token.
__global__ __launch_bounds__(256) void block_list_kernel(Args a, int* table, int* kv) {
  const BlockCall& c = a.c;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t units = c.total * c.Hkv, unit0 = (int64_t)blockIdx.x * 4, unit = unit0 + wave;
  const int64_t t = min(unit, units - 1) / c.Hkv;
  int b, i;
  Seq s;
  const bool live = token_at(a, unit0 / c.Hkv, t, b, s, i);
  if (unit >= units) return;
  if (!live) {
    if (lane == 0) kv[unit] = -1;
    return;
  }
  const int p = s.row0 + i, own = p >> a.pshift;
  const int* list = c.blocks + unit * c.count;
  const int* pages = c.page_table + (int64_t)b * c.max_pages;
  int* out = table + unit * c.count;
  int last = -1, n = 0;  // the largest so far, and how many
  for (int k = 0; k < c.count; k += 64) {
    const int x = k + lane < c.count ? list[k + lane] : -1;
    const int mine = x >= 0 && x <= own ? x : -1;
    int most = mine;  // of this lane and those before it
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(most, o, WAVE);
      if (lane >= o) most = max(most, u);
    }
    int before = __shfl_up(most, 1, WAVE);
    before = max(lane ? before : -1, last);
    const bool take = mine > before;
    const uint64_t all = __builtin_amdgcn_ballot_w64(take);
    if (take) out[n + __builtin_popcountll(all & ((1ull << lane) - 1))] = pages[mine];
    n += __builtin_popcountll(all);
    last = max(last, __builtin_amdgcn_readlane(most, 63));
  }
  if (lane == 0) kv[unit] = n && last == own ? ((n - 1) << a.pshift) + (p & ((1 << a.pshift) - 1)) + 1 : n << a.pshift;
}

int64_t cdiv(int64_t x, int64_t y) { return (x + y - 1) / y; }
size_t a256(size_t v) { return (v + 255) & ~(size_t)255; }

Args args_of(const BlockCall& c) {
  Args a;
  a.c = c;
  a.G = c.H / c.Hkv, a.pshift = __builtin_ctz((unsigned)c.page);
  a.slots = 0;
  return a;
}

int64_t mean_slots(const BlockCall& c) {
  return c.packed ? (c.total / c.page) + 2 * (int64_t)c.B : (int64_t)c.B * (((int64_t)c.T + c.page - 2) / c.page + 1);
}
int64_t score_slots(const BlockCall& c) { return c.packed ? c.total / 32 + c.B : (int64_t)c.B * cdiv(c.T, 32); }

// a step of one token each, in bf16: the means and the scores in one launch
bool scores_at_once(const BlockCall& c) { return c.scores && c.T == 1 && c.io != IO_F32; }

template <int D, typename KV> hipError_t means(const Args& a, hipStream_t stream) {
  block_means_kernel<D, KV><<<dim3((unsigned)(mean_slots(a.c) * a.c.Hkv)), dim3(256), 0, stream>>>(a);
  return hipGetLastError();
}

template <int D> hipError_t scores(const BlockCall& c, hipStream_t stream) {
  Args a = args_of(c);
  const bool f32 = c.io == IO_F32;
  const int64_t groups = cdiv(c.max_pages, PAGES);
  if (scores_at_once(c)) {
    const dim3 grid((unsigned)(c.total * c.Hkv * groups));
    if (c.bits8) block_scores_one_kernel<D, uint8_t><<<grid, dim3(256), 0, stream>>>(a, (uint32_t)groups);
    else block_scores_one_kernel<D, bf16_t><<<grid, dim3(256), 0, stream>>>(a, (uint32_t)groups);
    return hipGetLastError();
  }
  const hipError_t e = c.bits8 ? means<D, uint8_t>(a, stream) : f32 ? means<D, float>(a, stream) : means<D, bf16_t>(a, stream);
  if (e != hipSuccess || !c.scores) return e;
  a.slots = score_slots(c);
  if (f32) {
    block_scores_f32_kernel<D><<<dim3((unsigned)(a.slots * c.Hkv * groups)), dim3(256), 0, stream>>>(a, (uint32_t)groups);
  } else {
    // Tiles a workgroup: as many workgroups as the chip holds, where there are more tiles.  With
    // 1, 2, 4 and 8 tiles: 2K tokens at the end of 64K rows, 12 heads on 2 of 128, 32, 28, 36 and 60 us
    // (the rule takes 2); 4K tokens 54, 47, 43 and 62 (4); heads of 64, 4K tokens 37, 36, 36 and 54 (4);
    // 8 on 2 of 256, 2K tokens 61, 51, 47 and 74 (4); 4K 114, 93, 84 and 78 (8); 2K on 16K rows 20, 28,
    // 40 and 68 (1).
    const int64_t all = a.slots * c.Hkv * groups, tiles = std::min<int64_t>(std::max<int64_t>(all / (D == 256 ? 256 : 512), 1), 16);
    block_scores_kernel<D><<<dim3((unsigned)(cdiv(a.slots, tiles) * c.Hkv * groups)), dim3(256), 0, stream>>>(
        a, (uint32_t)groups, (int)tiles);
  }
  return hipGetLastError();
}

// attention over the listed pages: every (token, key head) is a sequence of one token
AttnCall listed(const BlockCall& c, const AttnCall& attn) {
  AttnCall x = attn;
  x.units = c.Hkv;
  x.B = (int)(c.total * c.Hkv), x.T = 1, x.H = c.H / c.Hkv, x.Hkv = 1, x.total = x.B;
  x.max_pages = c.count, x.max_kv = std::min(c.count, c.max_pages) << __builtin_ctz((unsigned)c.page);
  x.packed = false, x.cu_seqlens = nullptr, x.window = 0;
  return x;
}
size_t list_bytes(const BlockCall& c) { return a256((size_t)c.total * c.Hkv * c.count * 4) + a256((size_t)c.total * c.Hkv * 4); }

}  // namespace

int64_t block_scores_workgroups(const BlockCall& c) {
  const int64_t groups = cdiv(c.max_pages, PAGES);
  if (scores_at_once(c)) return c.total * c.Hkv * groups;
  return std::max(mean_slots(c) * c.Hkv, c.scores ? score_slots(c) * c.Hkv * groups : 0);
}

hipError_t launch_block_scores(const BlockCall& c, hipStream_t stream) {
  switch (c.D) {
    case 64: return scores<64>(c, stream);
    case 128: return scores<128>(c, stream);
    case 256: return scores<256>(c, stream);
  }
  return hipErrorInvalidValue;
}

int64_t block_select_workgroups(const BlockCall& c) { return c.total * c.Hkv * (c.max_pages <= 4096 ? 1 : 4); }

hipError_t launch_block_select(const BlockCall& c, hipStream_t stream) {
  const Args a = args_of(c);
  const dim3 grid((unsigned)cdiv(c.total * c.Hkv, c.max_pages <= 1024 ? 4 : 1));
  if (c.max_pages <= 256) block_select_kernel<1, 4><<<grid, dim3(256), 0, stream>>>(a);
  else if (c.max_pages <= 1024) block_select_kernel<1, 16><<<grid, dim3(256), 0, stream>>>(a);
  else if (c.max_pages <= 4096) block_select_kernel<4, 16><<<grid, dim3(256), 0, stream>>>(a);
  else if (c.max_pages <= 16384) block_select_kernel<16, 16><<<grid, dim3(1024), 0, stream>>>(a);
  else block_select_kernel<16, 64><<<grid, dim3(1024), 0, stream>>>(a);
  return hipGetLastError();
}

int64_t attn_blocks_workgroups(const BlockCall& c, const AttnCall& attn) {
  if (attn_lists_fit(c)) return attn_lists_workgroups(c);
  return std::max(attn_workgroups(listed(c, attn)), cdiv(c.total * c.Hkv, 4));
}

size_t attn_blocks_workspace_bytes(const BlockCall& c, const AttnCall& attn) {
  return attn_lists_fit(c) ? attn_lists_bytes(c) : list_bytes(c) + attn_workspace_bytes(listed(c, attn));
}

hipError_t launch_attn_blocks(const BlockCall& c, const AttnCall& attn, hipStream_t stream) {
  if (attn_lists_fit(c)) return c.bits8 ? launch_attn8_lists(attn, c, stream) : launch_attn_lists(attn, c, stream);
  AttnCall x = listed(c, attn);
  char* const ws = static_cast<char*>(attn.workspace);
  int* const table = reinterpret_cast<int*>(ws);
  int* const kv = reinterpret_cast<int*>(ws + a256((size_t)c.total * c.Hkv * c.count * 4));
  block_list_kernel<<<dim3((unsigned)cdiv(c.total * c.Hkv, 4)), dim3(256), 0, stream>>>(args_of(c), table, kv);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  x.page_table = table, x.kv_lens = kv, x.workspace = ws + list_bytes(c);
  return x.bits8 ? launch_attn8(x, stream) : launch_attn(x, stream);
}

}  // namespace jb
