// jb_attn.hip -- attention of each sequence's new tokens over its paged cache.
//
// A sequence has kv rows in the cache, the last T of them its new tokens.  New
// token i sits at row p = kv - T + i and sees rows max(0, p - window + 1) .. p
// (window 0: from row 0).  With x_j = scale q.k_j over those rows:
//     m = max x_j,  l = sum e^{x_j - m},  o = sum e^{x_j - m} v_j / l,
//     lse = m + ln l;   no row seen (or every x_j = -inf): o = 0, lse = -inf.
// The G = H / Hkv query heads of a key head share its rows, so a sequence's
// queries are the T G rows r = i G + g of a matrix that multiplies the same K
// and V.  One pass over the cache rows carries m, l and o (rescaled when m
// grows); nothing of size T x kv exists.
//
// Both kernels for bf16 form S^T = K Q^T with 32x32x16 matrix-core products, so
// that a lane holds one query (column lane % 32) and 16 of 32 cache rows: the
// softmax runs inside a lane but for one exchange with lane + 32, and the
// accumulators, rounded to bf16, are the B operand of O^T += V^T P^T as they
// stand (K order kperm32: slots 0..3 are rows 4 g .. 4 g + 3, slots 4..7 rows
// 8 + 4 g ..).  V's A operand is read down its columns from LDS.
// Rounding: scores, m, l and o are fp32, o is rounded once.  The matrix cores
// take P as bf16, because V is: where o is bf16 and there are many queries, P is
// rounded to it, half a step of each weight (2^-8) next to the half step that o
// itself loses (together 2.0-2.4e-3 of o's norm, o's rounding alone 1.65e-3).
// Where the caller wants o in fp32, and in decode, P is two parts, hi + lo
// (within 2^-15), and their products with V are two: nothing in decode (64
// sequences of 1K to 64K rows 365 us either way), but a third more with many queries
// (2K tokens on 64K rows 766 us, in two parts 1030; an 8K prompt 258 and 346; with
// fp32 o, which also leaves so, 988 and 344).
//   attn_tile_kernel  many queries: 4 waves x 32 rows of one key head walk the
//                     same 64-row cache tiles through two LDS buffers.
//   attn_row_kernel   at most 32 rows (decode): every wave takes its own 32-row
//                     cache tiles, no barrier in the loop, joined in LDS.
// The cache range of a tile of queries may be cut into nsplit pieces; each
// writes its unnormalised o, m and l, and attn_join_kernel adds them up.
// fp32 inputs take attn_f32_kernel, the same tiles on fp32 matrix cores.
//
// Reading the cache: 16 consecutive rows lie in one page, so a wave fetches
// them straight into LDS with one page index and one buffer descriptor that ends
// behind the last row any query of the workgroup sees: rows behind it, and
// pages whose index is out of range, arrive as zeros whatever memory holds.
// A masked weight is 0, and 0 times an inf or NaN is NaN, so a tile that some
// queries see in part only is looked over first: a value in V that is not
// finite counts as 0 on the matrix cores, and is added for the queries that do
// see it by itself.
#include <cmath>

#include "jb_attn.h"
#include "jb_device.h"
#include "jb_dma.h"

namespace jb {

namespace {

typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) bf16x8_t lds_bf16x8;
typedef short s4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s4_t lds_s4;
typedef unsigned int u4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) f4_t lds_f4;
typedef __attribute__((address_space(3))) u4_t lds_u4;
typedef __attribute__((address_space(3))) uint32_t lds_u32;
typedef __attribute__((address_space(3))) uint16_t lds_u16;
typedef __attribute__((address_space(3))) float lds_float;
typedef float f16_t __attribute__((ext_vector_type(16)));
typedef const __attribute__((address_space(4))) int* const_int_p;

constexpr float LN2 = 0.6931471805599453f;

// the unit (sequence, key head) that begins in a run and goes on in the `more`
// next ones; seg: its place among the run's units, 0 the first, 1 any other
struct Shared {
  int b, kvh, more, seg;
};

struct Args {
  int B, T, H, Hkv, G, pshift, max_pages, num_pages, window, nsplit;
  bool few;                                    // attn_row_kernel takes sequences of at most 32 rows
  bool direct;                                 // a unit of those is a workgroup
  int64_t total, q_stride, page_stride;
  int64_t whole, tail;                         // row tiles: the first ones, and those in nsplit pieces
  int pitch;                                   // rows of a tile's piece
  const int* cu;                               // NULL: dense, B x T tokens
  const int* kv_lens;
  const int* table;
  const void *q, *k, *v;
  void* o;
  float* lse;
  float* part_o;   // [nsplit][tail][Hkv][pitch][D]
  float2* part_ml; // [nsplit][tail][Hkv][pitch]
  float* run_o;    // [2 a workgroup][32][D]: attn_row_kernel's shared units
  float2* run_ml;  // [2 a workgroup][32]
  Shared* shared;  // [workgroups]
  float scale;     // times log2 e
  double inv_g;
};

// floor(n / d) from 1 / d in 64 bits, for 0 <= n, d with n < 2^41 and
// n / d < 2^31 (or d < 2^41 and n / d < 2^10): (n + 1/2) / d is at least
// 1 / (2 d) away from a whole number, further than its roundings.  A 64-bit
// division is some 150 instructions, and each stands before a kernel's first load.
__device__ __forceinline__ int64_t quotient(int64_t n, double inv) { return (int64_t)(((double)n + 0.5) * inv); }

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// the token of row r of a sequence's T G
__device__ __forceinline__ int token_of(const Args& a, int64_t r) { return (int)(((double)r + 0.5) * a.inv_g); }

// first token and length of sequence b (the a.T first tokens of a longer one), and
// its cache rows up to the last of them; all clamped to the tensors (they come from
// device memory).  kv - T is -2^30 at least, so a window behind it fits 32 bits.
struct Seq {
  int64_t tok0;
  int T, kv;
};
__device__ __forceinline__ Seq seq_of(const Args& a, int b) {
  Seq s;
  int all = a.T;
  if (a.cu) {
    const_int_p cu = (const_int_p)a.cu;
    clamp_span(cu[b], cu[b + 1], 0x7fffffff, a.total, s.tok0, all);
  } else {
    s.tok0 = (int64_t)b * a.T;
  }
  s.T = min(all, a.T);
  const int cap = (int)min((int64_t)a.max_pages << a.pshift, (int64_t)0x7fffffff);
  s.kv = max(min(max(((const_int_p)a.kv_lens)[b], 0), cap) - (all - s.T), s.T - (1 << 30));
  return s;
}

// Sequence and first row (of its T G) of slot s, tiles of R = 2^rshift rows.
// Packed sequences: sequence b's tiles start at slot base(b) = cu[b] G / R + b, which leaves
// room for all of them and never decreases, so the sequence is the last one
// whose base is not behind s (every thread looks at one base at a time).
__device__ __forceinline__ void slot_of(const Args& a, int64_t s, int rshift, int& b, int64_t& r0) {
  if (!a.cu) {
    const int64_t per = ((int64_t)a.T * a.G + (1 << rshift) - 1) >> rshift;
    b = (int)((uint32_t)s / (uint32_t)per);  // (both below 2^31: a grid's size, T G / R)
    r0 = (s - b * per) << rshift;
    return;
  }
  int n = 0;
  for (int i = 0; i < a.B; i += blockDim.x) {
    const int j = i + threadIdx.x;
    const bool in = j < a.B && (min(max((int64_t)a.cu[j], (int64_t)0), a.total) * a.G >> rshift) + j <= s;
    const int c = __syncthreads_count(in);
    n += c;
    if (c < (int)blockDim.x) break;
  }
  b = uniform(max(n - 1, 0));
  const int64_t base = (min(max((int64_t)((const_int_p)a.cu)[b], (int64_t)0), a.total) * a.G >> rshift) + b;
  r0 = (s - base) * (1 << rshift);
}

// What a workgroup of the tile kernels takes: a slot's key head, and the piece
// `split` of n of its cache range.  The longest ranges first: they end last.
struct Place {
  int kvh, split, n;
  int64_t slot;
  __device__ __forceinline__ explicit Place(const Args& a) {
    const int64_t head = a.whole * a.Hkv;
    n = blockIdx.x < head ? 1 : a.nsplit;
    const uint32_t i = blockIdx.x < head ? blockIdx.x : (uint32_t)(blockIdx.x - head), q = i / (uint32_t)(a.Hkv * n);
    const int combo = i - q * (uint32_t)(a.Hkv * n);
    kvh = combo % a.Hkv, split = combo / a.Hkv;
    slot = (n == 1 && a.whole ? a.whole + a.tail : a.tail) - 1 - q;
  }
  // index of row 0 in the pieces
  __device__ __forceinline__ int64_t part(const Args& a) const {
    return (((int64_t)split * a.tail + slot) * a.Hkv + kvh) * a.pitch;
  }
};

// ---------------------------------------------------------------- bf16 tiles

// LDS image of a tile: rows of D bf16, their 16-byte pieces permuted by row so
// that the reads below meet distinct banks: K fragments read one piece of 32
// rows, V fragments two neighbouring pieces of 4 rows.
template <int D> struct Img {
  static constexpr int PR = D / 8, ROWB = D * 2;
  __device__ static int fk(int r) { return r & (PR < 16 ? PR - 1 : 15); }
  __device__ static int fv(int r) { return PR < 16 ? (r & 3) << 1 : (r & 3) << 2; }
};

// 16 rows of an image (1 KB a transfer) from a buffer descriptor: transfers i =
// 0 .. 3 of 1 KB each; the instruction's offset counts for the buffer and LDS.
__device__ __forceinline__ void dma4(v4i_t desc, int v0, int v1, int v2, int v3, uint32_t lds) {
  uint32_t saved;
  asm volatile(
      "s_nop 4\n\ts_mov_b32 %0, m0\n\ts_mov_b32 m0, %6\n\ts_nop 0\n\t"
      "buffer_load_dwordx4 %1, %5, 0 offen lds\n\t"
      "buffer_load_dwordx4 %2, %5, 0 offen offset:1024 lds\n\t"
      "buffer_load_dwordx4 %3, %5, 0 offen offset:2048 lds\n\t"
      "buffer_load_dwordx4 %4, %5, 0 offen offset:(1024*3) lds\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "v"(v0), "v"(v1), "v"(v2), "v"(v3), "s"(desc), "s"(lds)
      : "memory");
}
__device__ __forceinline__ void dma2(v4i_t desc, int v0, int v1, uint32_t lds) {
  uint32_t saved;
  asm volatile(
      "s_nop 4\n\ts_mov_b32 %0, m0\n\ts_mov_b32 m0, %4\n\ts_nop 0\n\t"
      "buffer_load_dwordx4 %1, %3, 0 offen lds\n\t"
      "buffer_load_dwordx4 %2, %3, 0 offen offset:1024 lds\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "v"(v0), "v"(v1), "s"(desc), "s"(lds)
      : "memory");
}

// Cache rows, 16 at a time, of one sequence and key head into LDS images.
template <int D> struct Loader {
  using I = Img<D>;
  static constexpr int N = I::PR / 4;  // 1 KB transfers for 16 rows
  int vk[N], vv;                       // byte in the rows, less i KB, of transfer i (the same for V's)
  const bf16_t *k, *v;
  const int* table;
  int e0, ents;                        // table entries e0 + lane
  __device__ Loader(const Args& a, int b, int kvh) {
    const int lane = lane_id();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = lane / I::PR, c = lane % I::PR;
      vk[i] = r * I::ROWB + ((c ^ I::fk(i * 64 / I::PR + r)) * 16);
    }
    vv = (lane / I::PR) * I::ROWB + ((lane % I::PR ^ I::fv(lane / I::PR)) * 16);
    k = (const bf16_t*)a.k + ((int64_t)kvh << a.pshift) * D;
    v = (const bf16_t*)a.v + ((int64_t)kvh << a.pshift) * D;
    table = a.table + (int64_t)b * a.max_pages;
    e0 = -64;
  }
  // Page index of row0 < hi <= max_pages * page.  64 entries of the table wait
  // in a register, so that hardly any tile waits for one.
  __device__ int page(const Args& a, int row0) {
    const int e = row0 >> a.pshift;
    if ((unsigned)(e - e0) >= 64u) {
      e0 = e;
      ents = table[min(e + lane_id(), a.max_pages - 1)];
      asm volatile("" : "+v"(ents));  // waited for here
    }
    return __builtin_amdgcn_readlane(ents, e - e0);
  }
  // rows row0 .. row0 + 15 (row0 a multiple of 16) of K and V; zeros from row hi on
  __device__ void load(const Args& a, int row0, int hi, uint32_t ldsk, uint32_t ldsv) {
    const int pid = row0 < hi ? page(a, row0) : -1;
    const bool ok = (unsigned)pid < (unsigned)a.num_pages;
    const int n = ok ? min(max(hi - row0, 0), 16) : 0;
    const int64_t at = (ok ? pid : 0) * a.page_stride + (row0 & ((1 << a.pshift) - 1)) * D;
    const int bytes = n * I::ROWB;
    if constexpr (N == 2) {
      dma2(buf_desc(k + at, bytes), vk[0], vk[1], ldsk);
      dma2(buf_desc(v + at, bytes), vv, vv, ldsv);
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4) {  // (a descriptor for 4 KB: its range check sees every offset)
        const int left = max(bytes - i * 1024, 0);
        dma4(buf_desc(k + at + i * 512, left), vk[i], vk[i + 1], vk[i + 2], vk[i + 3], ldsk + i * 1024);
        dma4(buf_desc(v + at + i * 512, left), vv, vv ^ fv_flip(1), vv, vv ^ fv_flip(1), ldsv + i * 1024);
      }
    }
  }
  // D = 256: a transfer holds 2 rows, so V's piece order takes turns
  static constexpr int fv_flip(int i) { return D == 256 && i ? (2 << 2) * 16 : 0; }
};

__device__ __forceinline__ f16_t mfma32(bf16x8_t a, bf16x8_t b, f16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// lane + 32's (lane - 32's) value
__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32, WAVE); }
// the larger of a value and lane + 32's (lane - 32's), without LDS
__device__ __forceinline__ float half_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// o += weight times value, for the values that are not finite, of the cache rows
// that a query sees (o: D / 2 and s: NB x 16 accumulators of a wave).  A call of
// its own, on memory: it is rare, and inline it took the registers of the loops.
template <int D, int NB>
__device__ __attribute__((noinline)) void add_odd_values(float* o, const float* s, const lds_char* lv, int j0, int p,
                                                         int lw) {
  using I = Img<D>;
  const int g = lane_id() >> 5;
  for (int r = 0; r < NB * 32; ++r) {
    const float mine = s[(r >> 5) * 16 + ((r & 31) >> 3) * 4 + (r & 3)], other = __shfl_xor(mine, 32, WAVE);
    const float w = ((r >> 2) & 1) == g ? mine : other;
    if (j0 + r > p || j0 + r <= lw) continue;
    for (int e = 0; e < D / 2; ++e) {
      const int d = 32 * (e >> 4) + 8 * ((e >> 2) & 3) + 4 * g + (e & 3);
      const uint32_t u = *(const lds_u16*)(lv + r * I::ROWB + (((d >> 3) ^ I::fv(r)) << 4) + (d & 7) * 2);
      const float v = __uint_as_float(u << 16);
      if (!isfinite(v)) o[e] = fmaf(w, v, o[e]);
    }
  }
}

// One wave's 32 queries and what they have gathered so far.
template <int D> struct Wave {
  using I = Img<D>;
  bf16x8_t q[D / 16];
  f16_t o[D / 32];  // O^T: o[db][i] is d = 32 db + 8 (i / 4) + 4 g + i % 4
  float m, l;       // m as the exponent base 2 subtracts it; l of this lane's half of the rows
  int p, lw;        // sees rows lw < j <= p
  int phi, lwlo;    // of the wave's real rows: the last row seen, and the least lw

  __device__ void init(const Args& a, const Seq& s, int kvh, int64_t r0) {
    const int lane = lane_id();
    const int64_t nr = (int64_t)s.T * a.G, r = r0 + (lane & 31);
    const int base = s.kv - s.T;
    const bool real = r < nr;
    const int i = real ? token_of(a, r) : 0, g = real ? (int)(r - (int64_t)i * a.G) : 0;
    p = real ? base + i : -1;
    lw = a.window ? p - a.window : -1;
    const int64_t last = min(r0 + 32, nr) - 1;
    phi = lwlo = -1;
    if (r0 < nr) {
      phi = uniform(base + token_of(a, last));
      if (a.window) lwlo = uniform(base + token_of(a, r0)) - a.window;
    }
    const bf16_t* src = (const bf16_t*)a.q + (s.tok0 + i) * a.q_stride + (int64_t)(kvh * a.G + g) * D + 8 * (lane >> 5);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (real) w = *reinterpret_cast<const uint4*>(src + 16 * k);
      q[k] = __builtin_bit_cast(bf16x8_t, w);
    }
#pragma unroll
    for (int db = 0; db < D / 32; ++db)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[db][e] = 0.f;
    m = -INFINITY;
    l = 0.f;
  }

  // The queries are here: not in the loop, where a wait for them would be one
  // for the transfers in flight.
  __device__ void arrived() {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) asm volatile("" : "+v"(q[k]));
  }

  // S^T of NB x 32 cache rows, their K image at lk; K fragments are read
  // AHEAD steps before their products.
  template <int NB> __device__ void scores(const lds_char* lk, f16_t (&s)[NB]) const {
    const int lane = lane_id(), c = lane & 31, g = lane >> 5;
    const int kb = c * I::ROWB + ((g ^ I::fk(c)) << 4);
    constexpr int AHEAD = 2, STEPS = D / 16;
    bf16x8_t f[STEPS][NB];
    f16_t z;
#pragma unroll
    for (int e = 0; e < 16; ++e) z[e] = 0.f;
    auto read = [&](int k) {
#pragma unroll
      for (int n = 0; n < NB; ++n) f[k][n] = *(const lds_bf16x8*)(lk + (kb ^ (k << 5)) + n * 32 * I::ROWB);
    };
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) read(k);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
      if (k + AHEAD < STEPS) read(k + AHEAD);
#pragma unroll
      for (int n = 0; n < NB; ++n) s[n] = mfma32(f[k][n], q[k], k ? s[n] : z);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // Takes the tile's scores into the running maximum; returns what the
  // exponents subtract.  The maximum subtracted may lag behind the true one:
  // weights up to 2^8 lose nothing in fp32 sums or in bf16's relative
  // precision, and the rescaling of o is left out for all but the first tiles.
  template <int NB> __device__ float take_max(const Args& a, const f16_t (&s)[NB]) {
    float mx = s[0][0];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 16; ++e) mx = fmaxf(mx, s[n][e]);
    mx = half_max(mx) * a.scale;
    if (__any(mx > m + 8.f)) {
      const float mn = fmaxf(m, mx);
      const float f = mn == -INFINITY ? 1.f : fast_exp2(m - mn);
#pragma unroll
      for (int db = 0; db < D / 32; ++db)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[db][e] *= f;
      l *= f;
      m = mn;
    }
    return m == -INFINITY ? 0.f : m;
  }

  // weights of elements e0 .. e0 + n - 1 of the 16-row step k from its scores
  template <int NB> __device__ void weights(const Args& a, f16_t (&s)[NB], float ms, int k, int e0 = 0, int n = 8) {
#pragma unroll
    for (int e = e0; e < e0 + n; ++e) {
      const float x = fast_exp2(fmaf(s[k >> 1][8 * (k & 1) + e], a.scale, -ms));
      s[k >> 1][8 * (k & 1) + e] = x;
      l += x;
    }
  }

  // A tile that every query sees whole.  The maximum and the first weights, which
  // nothing of this wave overlaps, go before the other wave's work, and the
  // products with V, mixed with the other weights, before its products with K
  // (at equal priority 2K tokens on 64K rows take 787 us and an 8K prompt 289; so
  // 755 and 261 on the same card).
  template <int NB, bool TWO> __device__ void full(const Args& a, const lds_char* lk, const lds_char* lv) {
    f16_t s[NB];
    scores<NB>(lk, s);
    __builtin_amdgcn_s_setprio(2);
    const float ms = take_max<NB>(a, s);
    values<NB, true, TWO>(a, lv, s, ms);
    __builtin_amdgcn_s_setprio(0);
  }

  // NB x 32 cache rows from j0 that some queries see in part; false: none sees any
  template <int NB>
  __device__ bool part(const Args& a, const lds_char* lk, int j0, f16_t (&s)[NB]) {
    const int g = lane_id() >> 5;
    if (j0 > phi || j0 + NB * 32 - 1 <= lwlo) return false;
    scores<NB>(lk, s);
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int j = j0 + 32 * n + 8 * (e >> 2) + 4 * g + (e & 3);
        if (j > p || j <= lw) s[n][e] = -INFINITY;
      }
    const float ms = take_max<NB>(a, s);
#pragma unroll
    for (int k = 0; k < 2 * NB; ++k) weights<NB>(a, s, ms, k);
    return true;
  }
  // O^T += V^T P^T, 16 cache rows a step.  EXP: s holds scores yet; the next
  // step's exponentials and reads go between the products of this one.  TWO: P
  // as its upper 16 bits and what they leave, rounded to bf16 (cutting hi off takes
  // fewer operations than rounding it: 2K tokens on 64K rows 1030 us, 1053).
  template <int NB, bool EXP, bool TWO> __device__ void values(const Args& a, const lds_char* lv, f16_t (&s)[NB], float ms) {
    const int lane = lane_id(), g = lane >> 5;
    const int n16 = lane & 15, row = 4 * g + (n16 >> 2), pc = 2 * ((lane >> 4) & 1) + ((n16 & 3) >> 1);
    const int vb = row * I::ROWB + ((pc ^ I::fv(row)) << 4) + (n16 & 1) * 8;
    constexpr int DB = D / 32, STEPS = 2 * NB, PART = 8 / DB, AHEAD = 2;
    bf16x8_t v[STEPS * DB];  // read AHEAD products before its own
    auto read = [&](int i) {
      const lds_char* at = lv + (vb ^ ((i % DB) << 6)) + (i / DB) * 16 * I::ROWB;
      const s4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)at);
      const s4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(at + 8 * I::ROWB));
      v[i] = __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) read(i);
    if constexpr (EXP) {
      weights<NB>(a, s, ms, 0);
      __builtin_amdgcn_s_setprio(1);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
      bf16x8_t w, lo;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = s[k >> 1][8 * (k & 1) + e];
        if constexpr (TWO) {
          const uint32_t hi = __float_as_uint(x) & 0xffff0000u;
          w[e] = __builtin_bit_cast(__bf16, (uint16_t)(hi >> 16));
          lo[e] = (__bf16)(x - __uint_as_float(hi));
        } else {
          w[e] = (__bf16)x;
        }
      }
#pragma unroll
      for (int db = 0; db < DB; ++db) {
        const int i = k * DB + db;
        if (i + AHEAD < STEPS * DB) read(i + AHEAD);
        o[db] = mfma32(v[i], w, o[db]);
        if constexpr (TWO) o[db] = mfma32(v[i], lo, o[db]);
        if constexpr (EXP)
          if (k + 1 < STEPS) weights<NB>(a, s, ms, k + 1, db * PART, PART);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }

  // o += weight times value for the values that are not finite, of rows that are seen
  template <int NB> __device__ void odd_values(const f16_t (&s)[NB], const lds_char* lv, int j0) {
    float so[D / 2], ss[NB * 16];
#pragma unroll
    for (int e = 0; e < D / 2; ++e) so[e] = o[e >> 4][e & 15];
#pragma unroll
    for (int e = 0; e < NB * 16; ++e) ss[e] = s[e >> 4][e & 15];
    add_odd_values<D, NB>(so, ss, lv, j0, p, lw);
#pragma unroll
    for (int e = 0; e < D / 2; ++e) o[e >> 4][e & 15] = so[e];
  }
};

// whether a 16-byte aligned part of a V image holds a value that is not finite
// (exponent all ones); clean_part sets those to 0
__device__ __forceinline__ bool odd_bits(uint32_t u) {
  return (u & 0x7f80u) == 0x7f80u || (u & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ bool odd_part(const lds_char* v, int bytes) {
  bool odd = false;
#pragma unroll 4
  for (int i = lane_id() * 16; i < bytes; i += 1024) {
    const u4_t w = *(const lds_u4*)(v + i);
    odd |= odd_bits(w[0]) || odd_bits(w[1]) || odd_bits(w[2]) || odd_bits(w[3]);
  }
  return __any(odd);
}
__device__ __forceinline__ void clean_part(lds_char* v, int bytes) {
  for (int i = lane_id() * 4; i < bytes; i += 256) {
    uint32_t u = *(const lds_u32*)(v + i);
    if ((u & 0x7f80u) == 0x7f80u) u &= 0xffff0000u;
    if ((u & 0x7f800000u) == 0x7f800000u) u &= 0xffffu;
    *(lds_u32*)(v + i) = u;
  }
}

// the cache rows [lo, hi) that queries r0 .. r1 (of one sequence) see, and the
// part of their R-row tiles that piece `split` of `n` takes
struct Span {
  int lo, hi, t0, t1;
};
__device__ __forceinline__ Span span_of(const Args& a, const Seq& s, int64_t r0, int64_t r1, int R, int split, int n) {
  Span x;
  const int base = s.kv - s.T, first = base + token_of(a, r0);
  x.hi = max(base + token_of(a, r1) + 1, 0);
  x.lo = a.window ? min(max(first - a.window + 1, 0), x.hi) : 0;
  const int n0 = x.lo / R, n1 = (x.hi + R - 1) / R;
  const int per = (n1 - n0 + n - 1) / n;
  x.t0 = min(n0 + split * per, n1);
  x.t1 = min(x.t0 + per, n1);
  return x;
}

// The order in which a workgroup takes its tiles: those that every query r0 ..
// r1 sees whole first (f0 .. f0 + nf - 1), then those before and behind them.
struct Order {
  int t0, f0, nf, nt;
  __device__ Order(const Args& a, const Seq& s, const Span& x, int64_t r0, int64_t r1, int R) {
    // whole: ends by the first query's row and begins behind the last one's window
    const int first = s.kv - s.T + token_of(a, r0), cut = s.kv - s.T + token_of(a, r1) - a.window;
    t0 = x.t0;
    nt = x.t1 - x.t0;
    f0 = min(a.window && cut >= 0 ? max(x.t0, cut / R + 1) : x.t0, x.t1);
    nf = max(min(x.t1, first < 0 ? 0 : (first + 1) / R) - f0, 0);
  }
  __device__ int tile(int n) const { return n < nf ? f0 + n : n - nf < f0 - t0 ? t0 + n - nf : t0 + n; }
};

// element (row r, d .. d + 3) of a wave's staged 32 x D fp32 rows: 16-byte
// pieces permuted by row
template <int D> __device__ __forceinline__ lds_f4* stage_at(lds_char* st, int r, int d) {
  return (lds_f4*)(st + r * D * 4 + (((d >> 2) ^ (r & 15)) << 4));
}

template <typename OUT> __device__ __forceinline__ void store4(OUT* p, f4_t v);
template <> __device__ __forceinline__ void store4<float>(float* p, f4_t v) { *reinterpret_cast<f4_t*>(p) = v; }
template <> __device__ __forceinline__ void store4<bf16_t>(bf16_t* p, f4_t v) {
  uint2 u;
  u.x = f32_to_bf16(v[0]) | (uint32_t)f32_to_bf16(v[1]) << 16;
  u.y = f32_to_bf16(v[2]) | (uint32_t)f32_to_bf16(v[3]) << 16;
  *reinterpret_cast<uint2*>(p) = u;
}

// A wave's staged rows 0 .. rows - 1 to memory, 16 bytes a lane; lane i (and lane
// 32 + i) knows where row i goes.  (Found anew for every row, their places cost 2
// us at every workgroup's end, 5% of the windowed case.)
template <int D, typename T> __device__ __forceinline__ void leave_rows(T* out, lds_char* st, int64_t at, int rows) {
  constexpr int N = 16 / sizeof(T), LPR = D / N;  // values a lane, lanes a row
  const int lane = lane_id(), d = lane % LPR * N;
#pragma unroll
  for (int i0 = 0; i0 < 32; i0 += 64 / LPR) {
    const int i = i0 + lane / LPR;
    const int64_t to = (int64_t)(uint32_t)__shfl((int)at, i, WAVE) | (int64_t)__shfl((int)(at >> 32), i, WAVE) << 32;
    const f4_t v = *stage_at<D>(st, i, d);
    u4_t u = __builtin_bit_cast(u4_t, v);
    if constexpr (N == 8) {
      const f4_t x = *stage_at<D>(st, i, d + 4);
      u = u4_t{f32_to_bf16(v[0]) | (uint32_t)f32_to_bf16(v[1]) << 16, f32_to_bf16(v[2]) | (uint32_t)f32_to_bf16(v[3]) << 16,
               f32_to_bf16(x[0]) | (uint32_t)f32_to_bf16(x[1]) << 16, f32_to_bf16(x[2]) | (uint32_t)f32_to_bf16(x[3]) << 16};
    }
    if (i < rows) *reinterpret_cast<u4_t*>(out + to * D + d) = u;
  }
}

// where row r (of a sequence's T G) of key head kvh goes: row index of o, lse
__device__ __forceinline__ int64_t out_row(const Args& a, const Seq& s, int kvh, int64_t r) {
  const int i = token_of(a, r);
  return (s.tok0 + i) * a.H + kvh * a.G + (r - (int64_t)i * a.G);
}

// Many queries: 4 waves x 32 rows of one key head walk 64-row cache tiles, two in
// LDS: tile n + 1 arrives while n is used, one barrier a tile.
// Bound by the matrix cores and by what feeds them in turn: a wave's tile is 1024
// cycles of products (D = 128) and about 900 of vector work (32 exponentials at a
// quarter of the rate, the maximum, the sums), so two waves of two workgroups
// share a SIMD; 128 rows a workgroup keep two on a CU (64 KB of LDS, 198
// registers) and read every K and V value once for 128 queries.  2K tokens on 64K
// rows, 12 heads on 2: 751-766 us over the cards, 1060-1080 TFLOP/s (the library's
// product of 8192^3 reaches 1226), matrix cores busy 62% of the cycles at the 1.7
// GHz the card then holds, no bank conflicts.  Head size 64, as much vector work for
// half the products: 452 us, 900 TFLOP/s; 256, one wave a SIMD: 1574 us, 1030.
template <int D, typename OUT>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void attn_tile_kernel(Args a) {
  constexpr int NW = 4, R = 64, IMG = R * D * 2;
  constexpr bool TWO = sizeof(OUT) == 4;  // P in two parts
  __shared__ __attribute__((aligned(1024))) char ring[4 * IMG];  // K, V of an even tile, K, V of an odd one
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const Place at(a);
  const int kvh = at.kvh;
  int b;
  int64_t r0;
  slot_of(a, at.slot, 7, b, r0);
  const Seq s = seq_of(a, b);
  const int64_t nr = (int64_t)s.T * a.G;
  if (r0 < 0 || r0 >= nr) return;  // (r0 < 0: offsets that decrease)
  if (a.few && nr <= 32) return;  // attn_row_kernel's
  const int64_t r1 = min(r0 + NW * 32, nr) - 1;
  const Span x = span_of(a, s, r0, r1, R, at.split, at.n);
  Wave<D> w;
  w.init(a, s, kvh, r0 + wave * 32);
  Loader<D> ld(a, b, kvh);
  lds_char* const base = (lds_char*)ring;
  const Order ord(a, s, x, r0, r1, R);
  const int nf = ord.nf, nt = ord.nt;
  auto tile = [&](int n) { return ord.tile(n); };
  auto issue = [&](int n) {
    const int row0 = tile(n) * R + wave * 16;
    const uint32_t to = (uint32_t)(uintptr_t)(base + (n & 1) * 2 * IMG + wave * 16 * D * 2);
    ld.load(a, row0, x.hi, to, to + IMG);
  };
  // the queries and the page indices arrive together, then the first tile leaves
  if (nt > 0) ld.page(a, min(tile(0) * R + wave * 16, x.hi - 1));
  w.arrived();
  if (nt > 0) issue(0);
  auto next = [&](int n) {
    // every wave's transfers of tile n have landed, and every wave has left tile n - 1
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (n + 1 < nt) issue(n + 1);
    return base + (n & 1) * 2 * IMG;
  };
  for (int n = 0; n < nf; ++n) {
    const lds_char* k = next(n);
    w.template full<2, TWO>(a, k, k + IMG);
  }
  for (int n = nf; n < nt; ++n) {
    lds_char* const k = next(n);
    lds_char* const v = k + IMG;
    const bool odd = __syncthreads_or(odd_part(v + wave * (IMG / 4), IMG / 4));
    f16_t s2[2];
    const bool live = w.template part<2>(a, k, tile(n) * R, s2);
    if (odd) {
      if (live) w.template odd_values<2>(s2, v, tile(n) * R);
      __syncthreads();
      clean_part(v + wave * (IMG / 4), IMG / 4);
      __syncthreads();
    }
    if (live) w.template values<2, false, TWO>(a, v, s2, 0.f);
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  // O through LDS (each wave its own rows) so that whole rows leave
  const float l = w.l + other_half(w.l);
  const int c = lane & 31, g = lane >> 5;
  const int64_t r = r0 + wave * 32 + c;
  const bool split_out = at.n > 1;
  const int64_t to = r >= nr ? 0 : split_out ? at.part(a) + wave * 32 + c : out_row(a, s, kvh, r);
  if (g == 0 && r < nr) {
    if (split_out) a.part_ml[to] = make_float2(w.m, l);
    else if (a.lse) a.lse[to] = l == 0.f ? -INFINITY : (w.m + fast_log2(l)) * LN2;
  }
  const float f = split_out ? 1.f : l == 0.f ? 0.f : 1.f / l;
  static_assert(NW * 32 * D * 4 <= 4 * IMG, "staging fits");
  lds_char* st = base + wave * 32 * D * 4;
#pragma unroll
  for (int db = 0; db < D / 32; ++db)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *stage_at<D>(st, c, 32 * db + 8 * e + 4 * g) =
          f4_t{w.o[db][4 * e] * f, w.o[db][4 * e + 1] * f, w.o[db][4 * e + 2] * f, w.o[db][4 * e + 3] * f};
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  const int rows = (int)min(max(nr - r0 - wave * 32, (int64_t)0), (int64_t)32);
  if (split_out) leave_rows<D>(a.part_o, st, to, rows);
  else leave_rows<D>((OUT*)a.o, st, to, rows);
}

// Decode: sequences of at most 32 query rows.  A unit is one key head of one
// such sequence; it walks its cache in steps of NW tiles, one a wave.  The steps
// of all units, end to end, are cut into one equal run for each workgroup (the
// chip's worth of them), so that ragged lengths leave no workgroup waiting; a
// run's first and last units may be shared with its neighbours.
// The lengths live in device memory: every workgroup adds them up itself, and
// says which shared unit begins in its run.
// Bound by HBM: each wave keeps a 16 KB tile on its way (64 KB a CU) while it uses
// another, without a barrier.  64 sequences of 64K rows, 2 key heads of 128: 707
// us, 6.1 TB/s (a plain kernel that only reads reaches 7.2); of 1K to 64K rows: 365
// us, 5.9 TB/s (in an earlier form 361, and 377 cut into 16 even pieces each, without
// regard to the others); 256 of 1K rows: 48 us, 5.6 TB/s.
__device__ __forceinline__ int steps_of(const Args& a, const Seq& s, int rows_a_step) {
  const int64_t nr = (int64_t)s.T * a.G;
  if (nr == 0 || nr > 32) return 0;  // none, or attn_tile_kernel's
  const int hi = max(s.kv, 0), lo = a.window ? min(max(s.kv - s.T - a.window + 1, 0), hi) : 0;
  // (a sequence without rows has its output to write)
  return max((hi + rows_a_step - 1) / rows_a_step - lo / rows_a_step, 1);
}

template <int D, int NW, typename OUT>
__global__ __launch_bounds__(NW * 64, 1) void attn_row_kernel(Args a) {
  constexpr int R = 32, IMG = R * D * 2, STEP = R * NW, NTHR = NW * 64;
  __shared__ __attribute__((aligned(1024))) char ring[NW * 4 * IMG];
  __shared__ int64_t found[2];
  __shared__ int sums[NW];
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  int b;
  int64_t at, end, start;  // this run's steps, and the first sequence's first one
  int64_t run_steps = 0;
  if (a.direct) {         // many units: each is a run
    b = blockIdx.x / (unsigned)a.Hkv;
    const int n = steps_of(a, seq_of(a, b), STEP);
    start = 0;
    at = (int64_t)(blockIdx.x % (unsigned)a.Hkv) * n;
    end = at + n;
  } else {
    // The steps of 64 NW sequences at a time, added up; then this run's place
    // among them, at once where one pass has seen them all.
    if (threadIdx.x == 0) found[0] = found[1] = 0;
    int64_t base, before;  // steps of the sequences up to here, and before this thread's
    int n;                 // this thread's
    auto add = [&](int i) {
      n = i + (int)threadIdx.x < a.B ? steps_of(a, seq_of(a, i + threadIdx.x), STEP) : 0;
      int v = n;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(v, o, WAVE);
        if (lane >= o) v += u;
      }
      if (lane == 63) sums[wave] = v;
      __syncthreads();
      before = base + (int64_t)(v - n) * a.Hkv;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        if (w < wave) before += (int64_t)sums[w] * a.Hkv;
        base += (int64_t)sums[w] * a.Hkv;
      }
      __syncthreads();
    };
    auto look = [&](int i) {
      if (before <= at && at < before + (int64_t)n * a.Hkv) found[0] = i + threadIdx.x, found[1] = before;
    };
    base = 0;
    for (int i = 0; i < a.B; i += NTHR) add(i);
    const int64_t per = quotient(base + gridDim.x - 1, 1.0 / gridDim.x);
    at = min(blockIdx.x * per, base);
    end = min(at + per, base);
    if (a.B <= NTHR) {
      look(0);
    } else {
      base = 0;
      for (int i = 0; i < a.B; i += NTHR) {
        add(i);
        look(i);
      }
    }
    __syncthreads();
    b = uniform((int)found[0]);
    start = found[1];
    run_steps = per;
  }
  Shared shared = {0, 0, 0, 0};

  constexpr int NT = 4 * Loader<D>::N;  // transfers a tile
  lds_char* const base = (lds_char*)ring + wave * 4 * IMG;
  for (int seg = 0; at < end && b < a.B; seg = 1) {
    const Seq s = seq_of(a, b);
    const int steps = steps_of(a, s, STEP);
    if (steps == 0) {  // (only behind a sequence that has some)
      ++b;
      continue;
    }
    const int kvh = uniform((int)quotient(at - start, 1.0 / steps)), s0 = uniform((int)(at - start - (int64_t)kvh * steps));
    const int s1 = uniform((int)min((int64_t)steps, s0 + end - at));
    if (kvh >= a.Hkv) break;  // (lengths that changed meanwhile)
    const int nr = (int)(s.T * a.G);
    Span x;
    x.hi = max(s.kv, 0);
    x.lo = a.window ? min(max(s.kv - s.T - a.window + 1, 0), x.hi) : 0;
    const int n0 = x.lo / STEP * NW;
    x.t0 = max(n0 + s0 * NW, x.lo / R);
    x.t1 = min(n0 + s1 * NW, (x.hi + R - 1) / R);
    Wave<D> w;
    w.init(a, s, kvh, 0);
    Loader<D> ld(a, b, kvh);
    auto issue = [&](int t, int par) {
      const uint32_t to = (uint32_t)(uintptr_t)(base + par * 2 * IMG);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this wave's reads of the buffer are done
      ld.load(a, t * R, x.hi, to, to + IMG);
      ld.load(a, t * R + 16, x.hi, to + 16 * D * 2, to + IMG + 16 * D * 2);
    };
    const Order ord(a, s, x, 0, nr - 1, R);
    const int nf = ord.nf, nt = ord.nt;
    int par = 0;
    // tile n has landed, and the wave's next one is on its way into the other buffer
    auto next = [&](int n) {
      if (n + NW < nt) {
        issue(ord.tile(n + NW), par ^ 1);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(NT) : "memory");
      } else {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      }
      lds_char* const k = base + par * 2 * IMG;
      par ^= 1;
      return k;
    };
    if (wave < nt) ld.page(a, ord.tile(wave) * R);
    w.arrived();
    if (wave < nt) issue(ord.tile(wave), 0);
    int n = wave;
    for (; n < nf; n += NW) {
      const lds_char* k = next(n);
      w.template full<1, true>(a, k, k + IMG);
    }
    for (; n < nt; n += NW) {
      lds_char* const k = next(n);
      lds_char* const v = k + IMG;
      f16_t s1[1];
      if (w.template part<1>(a, k, ord.tile(n) * R, s1)) {
        if (odd_part(v, IMG)) {
          w.template odd_values<1>(s1, v, ord.tile(n) * R);
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
          clean_part(v, IMG);
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
        w.template values<1, false, true>(a, v, s1, 0.f);
      }
    }
    // join the waves: O and (m, l) of each in LDS
    const int c = lane & 31, g = lane >> 5;
    const float l = w.l + other_half(w.l);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    lds_char* const all = (lds_char*)ring;
    constexpr int ST = 32 * D * 4;
    static_assert(NW * ST + NW * 32 * 8 <= NW * 4 * IMG, "staging fits");
    lds_char* st = all + wave * ST;
#pragma unroll
    for (int db = 0; db < D / 32; ++db)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *stage_at<D>(st, c, 32 * db + 8 * e + 4 * g) =
            f4_t{w.o[db][4 * e], w.o[db][4 * e + 1], w.o[db][4 * e + 2], w.o[db][4 * e + 3]};
    lds_float* ml = (lds_float*)(all + NW * ST);  // [2][NW][32]
    if (g == 0) {
      ml[wave * 32 + c] = w.m;
      ml[NW * 32 + wave * 32 + c] = l;
    }
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    // (a unit that is a run has no place for a part, whatever the lengths in memory do meanwhile)
    const bool whole = a.direct || (s0 == 0 && s1 == steps);
    if (s0 == 0 && !whole) {  // (in the grid whatever the lengths in memory do meanwhile)
      const int last = (int)min(quotient(at + steps - 1, 1.0 / run_steps), (int64_t)gridDim.x - 1);
      shared = {b, kvh, last - (int)blockIdx.x, seg};
    }
    const int64_t slot = 2 * (int64_t)blockIdx.x + seg;
    constexpr int LPR = D / 4;
    for (int i = threadIdx.x / LPR; i < nr; i += NTHR / LPR) {
      const int d = (threadIdx.x % LPR) * 4;
      float m = -INFINITY;
#pragma unroll
      for (int n = 0; n < NW; ++n) m = fmaxf(m, ml[n * 32 + i]);
      f4_t sum = zero4();
      float lt = 0.f;
#pragma unroll
      for (int n = 0; n < NW; ++n) {
        const float mn = ml[n * 32 + i];
        // (a wave that saw nothing holds zeros, or NaN that stays)
        const float f = mn == -INFINITY ? 1.f : fast_exp2(mn - m);
        const f4_t v = *stage_at<D>(all + n * ST, i, d);
        lt = fmaf(ml[NW * 32 + n * 32 + i], f, lt);
        sum += v * f;
      }
      if (!whole) {
        if (d == 0) a.run_ml[slot * 32 + i] = make_float2(m, lt);
        *reinterpret_cast<f4_t*>(a.run_o + (slot * 32 + i) * D + d) = sum;
      } else {
        const int64_t to = out_row(a, s, kvh, i);
        const float f = lt == 0.f ? 0.f : 1.f / lt;
        if (d == 0 && a.lse) a.lse[to] = lt == 0.f ? -INFINITY : (m + fast_log2(lt)) * LN2;
        store4((OUT*)a.o + to * D + d, sum * f);
      }
    }
    at += s1 - s0;
    if (at >= end) break;
    if (kvh == a.Hkv - 1) start += (int64_t)steps * a.Hkv, ++b;
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // the staging is read
  }
  if (!a.direct && threadIdx.x == 0) a.shared[blockIdx.x] = shared;
}

// Adds up (m, l, o) pieces in the order they come.
struct Sum {
  float m = -INFINITY, l = 0.f;
  f4_t o = zero4();
  __device__ void add(float pm, float pl, f4_t v) {
    const float mn = fmaxf(m, pm);
    const float f = m == -INFINITY ? 1.f : fast_exp2(m - mn), h = pm == -INFINITY ? 1.f : fast_exp2(pm - mn);
    m = mn;
    l = fmaf(l, f, pl * h);
    o = o * f + v * h;
  }
  // over the SG lane groups of a row, the others' part through LDS: the first has all
  template <int SG, int LPR> __device__ void over(int sg, int r, int d4, f4_t (*so)[256 / SG], float2 (*sml)[256 / SG]) {
    so[sg][r * LPR + d4] = o;
    sml[sg][r * LPR + d4] = make_float2(m, l);
    __syncthreads();
    if (sg == 0)
#pragma unroll
      for (int i = 1; i < SG; ++i) add(sml[i][r * LPR + d4].x, sml[i][r * LPR + d4].y, so[i][r * LPR + d4]);
  }
  template <typename OUT, int D> __device__ void store(const Args& a, int64_t row, int d) const {
    const float f = l == 0.f ? 0.f : 1.f / l;
    if (d == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : (m + fast_log2(l)) * LN2;
    store4((OUT*)a.o + row * D + d, o * f);
  }
};

// The units that runs share: one workgroup for each query row of the unit that
// begins in run blockIdx.x / rows, its lane groups sharing the runs.
template <int D, typename OUT>
__global__ __launch_bounds__(256) void attn_row_join_kernel(Args a, int rows) {
  constexpr int LPR = D / 4, SG = 256 / LPR;
  const int w0 = blockIdx.x / (unsigned)rows, r = blockIdx.x % (unsigned)rows;
  const Shared u = a.shared[w0];
  if (u.more == 0) return;
  const Seq s = seq_of(a, u.b);
  if (r >= s.T * a.G) return;
  const int d4 = threadIdx.x % LPR, sg = threadIdx.x / LPR;
  Sum x;
#pragma unroll 4
  for (int i = sg; i <= u.more; i += SG) {
    // (it is the first unit of every run but the one it begins in)
    const int64_t at = (2 * (int64_t)(w0 + i) + (i ? 0 : u.seg)) * 32 + r;
    const float2 ml = a.run_ml[at];
    x.add(ml.x, ml.y, *reinterpret_cast<const f4_t*>(a.run_o + at * D + d4 * 4));
  }
  __shared__ f4_t so[SG][LPR];
  __shared__ float2 sml[SG][LPR];
  x.template over<SG, LPR>(sg, 0, d4, so, sml);
  if (sg == 0) x.template store<OUT, D>(a, out_row(a, s, u.kvh, r), d4 * 4);
}

// Adds up the pieces of every row of the tiles (of 2^rshift rows) that are in
// pieces, SG lane groups a row; a workgroup's rows are of one tile (the pitch is
// a multiple of 16).
template <int D, int SG, typename OUT>
__global__ __launch_bounds__(256) void attn_join_kernel(Args a, int rshift) {
  constexpr int LPR = D / 4, RPB = 256 / (LPR * SG);
  const int d = (threadIdx.x % LPR) * 4, sg = threadIdx.x / LPR % SG, i = threadIdx.x / (LPR * SG);
  const uint32_t each = (uint32_t)a.pitch / RPB, unit = blockIdx.x / each, slot = unit / (uint32_t)a.Hkv;
  const int kvh = unit - slot * (uint32_t)a.Hkv, row = (blockIdx.x - unit * each) * RPB + i;
  int b;
  int64_t r0;
  slot_of(a, slot, rshift, b, r0);
  const Seq s = seq_of(a, b);
  const int64_t nr = (int64_t)s.T * a.G, r = r0 + row;
  if (r0 < 0 || (a.few && nr <= 32)) return;
  const bool own = r < nr;
  Sum x;
  if (own) {
    const int64_t n = a.tail * a.Hkv * a.pitch, at = (int64_t)unit * a.pitch + row;
#pragma unroll 4
    for (int i = sg; i < a.nsplit; i += SG) {
      const float2 ml = a.part_ml[i * n + at];
      x.add(ml.x, ml.y, *reinterpret_cast<const f4_t*>(a.part_o + (i * n + at) * D + d));
    }
  }
  if constexpr (SG > 1) {
    __shared__ f4_t so[SG][RPB * LPR];
    __shared__ float2 sml[SG][RPB * LPR];
    x.template over<SG, LPR>(sg, i, threadIdx.x % LPR, so, sml);
  }
  if (own && sg == 0) x.template store<OUT, D>(a, out_row(a, s, kvh, r), d);
}

// ------------------------------------------------------------------ fp32 mode
// S^T = K Q^T and O^T += V^T P^T on 16x16x4 fp32 matrix cores, a tile of cache
// rows at a time in LDS.  Lane: query lane % 16, cache rows 4 g + i of each 16.
// Everything stays fp32.  4 waves x 16 query rows share 32-row tiles; for at
// most 16 query rows (decode, SHARE) every wave has the same queries and takes
// 16 of a tile's 64 cache rows, joined in LDS at the end.  16 sequences of 8K
// rows, 2 key heads of 128: 68 us, 4.0 TB/s; 1K tokens on 4K rows, 8 heads: 201
// us, 75 TFLOP/s (the library's fp32 product reaches 154).
template <int D, bool SHARE, typename OUT>
__global__ __launch_bounds__(256, 1) void attn_f32_kernel(Args a) {
  constexpr int R = SHARE ? 64 : 32, LD = D + 4, NW = 4, QR = SHARE ? 16 : NW * 16;
  constexpr int NB = SHARE ? 1 : 2;  // 16-row blocks of a tile that a wave takes
  __shared__ __attribute__((aligned(16))) float kv[2 * R * LD];
  float *const sk = kv, *const sv = kv + R * LD;
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const Place at(a);
  const int kvh = at.kvh;
  int b;
  int64_t r0;
  slot_of(a, at.slot, SHARE ? 4 : 6, b, r0);
  const Seq s = seq_of(a, b);
  const int64_t nr = (int64_t)s.T * a.G;
  if (r0 < 0 || r0 >= nr) return;
  const Span x = span_of(a, s, r0, min(r0 + QR, nr) - 1, R, at.split, at.n);
  const int64_t r = r0 + (SHARE ? 0 : wave * 16) + c;
  const int block = SHARE ? wave * 16 : 0;  // of this wave's rows in a tile
  const bool real = r < nr;
  const int i0 = real ? token_of(a, r) : 0, g0 = real ? (int)(r - (int64_t)i0 * a.G) : 0;
  const int p = real ? s.kv - s.T + i0 : -1, lw = a.window ? p - a.window : -1;
  const float* src = (const float*)a.q + (s.tok0 + i0) * a.q_stride + (int64_t)(kvh * a.G + g0) * D + 4 * g;
  float4 q[D / 16];
  f4_t o[D / 16];
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    q[k] = real ? *reinterpret_cast<const float4*>(src + 16 * k) : make_float4(0.f, 0.f, 0.f, 0.f);
    o[k] = zero4();
  }
  float m = -INFINITY, l = 0.f;
  // Tile t + 1 is on its way into registers while tile t is used: the pages of
  // its rows are known a tile before that.
  constexpr int PER = R * (D / 4) / 256;
  float4 kn[PER], vn[PER];
  int pages[R / 16];
  auto fetch = [&](int t) {
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int e = u * 256 + threadIdx.x, rr = e / (D / 4), d = (e % (D / 4)) * 4, j = t * R + rr;
      int pid = pages[0];
#pragma unroll
      for (int h = 1; h < R / 16; ++h) pid = rr >= 16 * h ? pages[h] : pid;
      kn[u] = vn[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (j >= x.lo && j < x.hi && pid >= 0 && pid < a.num_pages) {
        const int64_t at = pid * a.page_stride + (((int64_t)kvh << a.pshift) + (j & ((1 << a.pshift) - 1))) * D + d;
        kn[u] = *reinterpret_cast<const float4*>((const float*)a.k + at);
        vn[u] = *reinterpret_cast<const float4*>((const float*)a.v + at);
      }
    }
  };
  auto look_up = [&](int t) {
#pragma unroll
    for (int h = 0; h < R / 16; ++h) {
      const int j = t * R + 16 * h;
      pages[h] = t < x.t1 && j < x.hi ? ((const_int_p)a.table)[(int64_t)b * a.max_pages + (j >> a.pshift)] : -1;
    }
  };
  look_up(x.t0);
  if (x.t0 < x.t1) fetch(x.t0);
  look_up(x.t0 + 1);
  for (int t = x.t0; t < x.t1; ++t) {
    __syncthreads();
    bool bad = false;
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int e = u * 256 + threadIdx.x, rr = e / (D / 4), d = (e % (D / 4)) * 4;
      const float4 kx = kn[u], vx = vn[u];
      bad |= !(isfinite(vx.x) && isfinite(vx.y) && isfinite(vx.z) && isfinite(vx.w));
      *reinterpret_cast<float4*>(sk + rr * LD + d) = kx;
      *reinterpret_cast<float4*>(sv + rr * LD + d) = vx;
    }
    if (t + 1 < x.t1) {
      fetch(t + 1);
      look_up(t + 2);
    }
    const bool slow = __syncthreads_or(bad);
    f4_t y[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      y[n] = zero4();
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const float4 kx = *reinterpret_cast<const float4*>(sk + (block + 16 * n + c) * LD + 16 * k + 4 * g);
        y[n] = __builtin_amdgcn_mfma_f32_16x16x4f32(kx.x, q[k].x, y[n], 0, 0, 0);
        y[n] = __builtin_amdgcn_mfma_f32_16x16x4f32(kx.y, q[k].y, y[n], 0, 0, 0);
        y[n] = __builtin_amdgcn_mfma_f32_16x16x4f32(kx.z, q[k].z, y[n], 0, 0, 0);
        y[n] = __builtin_amdgcn_mfma_f32_16x16x4f32(kx.w, q[k].w, y[n], 0, 0, 0);
      }
    }
    float mx = -INFINITY;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = t * R + block + 16 * n + 4 * g + e;
        y[n][e] = j > p || j <= lw ? -INFINITY : y[n][e] * a.scale;
        mx = fmaxf(mx, y[n][e]);
      }
    mx = fmaxf(mx, __shfl_xor(mx, 16, WAVE));
    mx = fmaxf(mx, __shfl_xor(mx, 32, WAVE));
    const float mn = fmaxf(m, mx), ms = mn == -INFINITY ? 0.f : mn;
    const float f = m == -INFINITY ? 0.f : fast_exp2(m - ms);
    m = mn;
    l *= f;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[n][e] = fast_exp2(y[n][e] - ms);
        l += y[n][e];
      }
    if (mn != -INFINITY)
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[k][e] *= f;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = sv[(block + 16 * n + 4 * g + e) * LD + 16 * k + c];
          if (slow && !isfinite(v)) v = 0.f;
          o[k] = __builtin_amdgcn_mfma_f32_16x16x4f32(v, y[n][e], o[k], 0, 0, 0);
        }
    if (slow) {
      for (int rr = 0; rr < NB * 16; ++rr) {
        float w = 0.f;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) w = n * 16 + e == (rr & 16) + (rr & 3) ? y[n][e] : w;
        w = __shfl(w, ((rr >> 2) & 3) * 16 + c, WAVE);
        const int j = t * R + block + rr;
        if (j <= p && j > lw)
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float v = sv[(block + rr) * LD + 16 * k + 4 * g + e];
              if (!isfinite(v)) o[k][e] = fmaf(w, v, o[k][e]);
            }
      }
    }
  }
  l += __shfl_xor(l, 16, WAVE);
  l += __shfl_xor(l, 32, WAVE);
  if constexpr (SHARE) {
    // the waves' parts, the first wave adding them up in its registers
    __syncthreads();
    float* const so = kv;                      // [NW][16][LD]
    float* const sml = kv + NW * 16 * LD;      // [NW][2][16]
    static_assert(NW * 16 * LD + NW * 32 <= 2 * R * LD, "staging fits");
#pragma unroll
    for (int k = 0; k < D / 16; ++k) *reinterpret_cast<f4_t*>(so + (wave * 16 + c) * LD + 16 * k + 4 * g) = o[k];
    if (g == 0) sml[wave * 32 + c] = m, sml[wave * 32 + 16 + c] = l;
    __syncthreads();
    if (wave) return;
    float mt = m;
#pragma unroll
    for (int w = 1; w < NW; ++w) mt = fmaxf(mt, sml[w * 32 + c]);
    // (a wave that saw nothing holds zeros, or NaN that stays)
    const float f0 = m == -INFINITY ? 1.f : fast_exp2(m - mt);
    l *= f0;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) o[k] *= f0;
#pragma unroll
    for (int w = 1; w < NW; ++w) {
      const float mw = sml[w * 32 + c], fw = mw == -INFINITY ? 1.f : fast_exp2(mw - mt);
      l = fmaf(sml[w * 32 + 16 + c], fw, l);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) o[k] += *reinterpret_cast<const f4_t*>(so + (w * 16 + c) * LD + 16 * k + 4 * g) * fw;
    }
    m = mt;
  }
  if (!real) return;
  const bool split_out = at.n > 1;
  const int64_t to = split_out ? at.part(a) + r - r0 : out_row(a, s, kvh, r);
  if (g == 0) {
    if (split_out) a.part_ml[to] = make_float2(m, l);
    else if (a.lse) a.lse[to] = l == 0.f ? -INFINITY : (m + fast_log2(l)) * LN2;
  }
  const float f = split_out ? 1.f : l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    const f4_t v = o[k] * f;
    if (split_out) *reinterpret_cast<f4_t*>(a.part_o + to * D + 16 * k + 4 * g) = v;
    else store4((OUT*)a.o + to * D + 16 * k + 4 * g, v);
  }
}

// ------------------------------------------------------------------ launches

struct Plan {
  bool tiles, rows;   // which of the bf16 kernels run
  int64_t slots;      // row tiles, over all sequences
  int64_t tail;       // those, the last to run, whose cache ranges are in pieces
  int nsplit;         // pieces
  int rshift, pitch;  // rows of a tile (2^rshift), and of its piece
  bool share;         // fp32 decode: the waves of attn_f32_kernel share the queries
  bool direct;        // attn_row_kernel: a unit a workgroup
  int64_t runs;       // its workgroups
  int rows_a_unit;    // query rows of its units, at most
};

int64_t cdiv(int64_t x, int64_t y) { return (x + y - 1) / y; }
size_t a256(size_t v) { return (v + 255) & ~(size_t)255; }

constexpr int row_waves(int D) { return D == 256 ? 2 : 4; }  // of attn_row_kernel: two tiles each in LDS

Plan plan(const AttnCall& c) {
  Plan p;
  const int64_t G = c.H / c.Hkv, per = (int64_t)c.T * G;
  const bool f32 = c.io == IO_F32;
  p.share = f32 && per <= 16;
  p.rshift = p.share ? 4 : f32 ? 6 : 7;
  const int R = 1 << p.rshift;
  p.pitch = (int)std::min<int64_t>(R, (per + 15) & ~(int64_t)15);
  // bf16 sequences of at most 32 rows go to attn_row_kernel.  A packed batch may
  // hold both kinds, and gets both kernels unless no cache range is longer than a
  // workgroup of the tile kernel walks while others still work.  12 heads on 2 of
  // 128, the tile kernel alone and both kernels.  Ranges up to 2048: 16 sequences of 1
  // to 1024 tokens under a window of 1152 95 and 106 us, 60 single tokens and 4 chunks
  // of 512 46 and 64, 252 and 4 90 and 102.  Longer ones that are alike lose too (60 and
  // 4 on 4K rows: 109 and 140; on 16K and more either), but unlike ones need the
  // equal runs: one of 64K rows among 255 of 1K 538 and 463, and single tokens
  // packed without a planned length 291 and 151.
  const int64_t reach = c.window ? std::min(c.max_kv, c.window) : c.max_kv;
  p.tiles = f32 || per > 32;
  p.rows = !f32 && (per <= 32 || (c.packed && c.total < (int64_t)c.B * c.T && reach > 2048));
  p.slots = c.packed ? c.total * G / R + c.B : c.B * cdiv(per, R);
  p.nsplit = 1;
  p.tail = 0;
  // Decode: as many workgroups as the chip holds, of a step at least; with
  // thousands of units, or one step each, there is nothing to even out.
  p.rows_a_unit = (int)std::min<int64_t>(per, 32);
  const int64_t units = (int64_t)c.B * c.Hkv, range = c.window ? std::min<int64_t>(c.max_kv, c.window + 32) : c.max_kv;
  const int step = 32 * row_waves(c.D);
  p.direct = units >= 4096 || range <= step;
  p.runs = p.direct ? units : std::min<int64_t>(c.D == 64 ? 512 : 256, units * cdiv(range, step));
  if (!p.tiles) return p;
  if (f32) {
    // pieces for about so many workgroups, by measurement; registers hold fewer at
    // once in some (chunks: 1024, 768 and 256 by the head size; decode: 768, 512, 256).
    // For 256, 512, 768 and 1024 workgroups: 1K tokens on 4K rows, 8 heads on 8, head
    // size 64 168, 117, 108 and 102 us, 128 284, 203, 188 and 203, 256 522, 477, 493 and
    // 502; decode of 16 x 8K rows, 2 key heads, 64 59, 49, 49 and 52, 128 84, 69, 87 and
    // 74, 256 142, 154, 178 and 179.
    const int64_t hold = std::min((p.share ? 65536 : 131072) / c.D, 1024);
    const int64_t want = cdiv(hold, p.slots * c.Hkv), most = cdiv(reach, 64);
    p.nsplit = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(want, most), 128));
    p.tail = p.nsplit > 1 ? p.slots : 0;
    return p;
  }
  // Tiles: the least of the rounds the pieces take on the chip's workgroup slots
  // (tiles of 64 rows, in the mean over the queries, and some 4 tiles' worth of
  // start and end each; the longest range alone is a bound too) plus the join's
  // traffic.  A workgroup alone on its CU walks a tile in 1.7 us (D = 128), 2.0
  // with a second one there, so a last round of at most 256 costs less than a
  // whole one.  2K tokens, 16 heads on 2 (256 units) under a window of 1152: 1
  // piece 33 us, 2 41; 2K tokens on 64K rows (192 units): 6 pieces 892 us, 8
  // (three whole rounds) 753, 16 783; an 8K prompt (1024 units): 1 piece 261
  // us, 2 301.
  const int cu = c.D == 64 ? 3 : c.D == 128 ? 2 : 1;  // workgroups a CU holds
  // (a packed batch has more slots than tiles; half a tile of each sequence is a guess)
  const int64_t work = (c.packed ? cdiv(c.total * G, R) + c.B / 2 : p.slots) * c.Hkv;
  auto tiles = [&](int64_t kv) { return (double)cdiv(c.window ? std::min<int64_t>(kv, c.window + R / G) : kv, 64); };
  const double longest = tiles(c.max_kv), mean = tiles(std::max<int64_t>(c.max_kv - c.T / 2, 1));
  const double rows = (double)c.total * c.H;
  auto walk = [&](int64_t on_a_cu) { return on_a_cu ? 1.7 * (1 + 0.2 * (on_a_cu - 1)) * c.D / 128 : 0.; };
  auto rounds = [&](int64_t n) { return n / (256 * cu) * walk(cu) + walk(cdiv(n % (256 * cu), 256)); };
  auto join = [&](double rows, int n) { return n > 1 ? 5 + rows * c.D * 8 * n / 6e6 : 0.; };
  double best = 0;
  for (int n = 1; n <= 64 && n <= std::max(longest / 4, 1.0); ++n) {
    const double t = std::max((mean / n + 4) * rounds(work * n), (longest / n + 4) * walk(1)) + join(rows, n);
    if (n == 1 || t < best) best = t, p.nsplit = n;
  }
  p.tail = p.nsplit > 1 ? p.slots : 0;
  // Whole ranges in more than one round: those of the last, partial round (the
  // shortest) may be in pieces (12 heads on 2 of 128: 528 units under a window of
  // 1152 take 62 us so, 75 whole; 600 under one of 2304 116, 132).
  const int64_t rest = work % (256 * cu);
  if (p.nsplit == 1 && work > 256 * cu && rest) {
    const double shortest = tiles(std::max<int64_t>(c.max_kv - c.T, 1));
    best = (shortest + 4) * rounds(rest);
    for (int n = 2; n <= 16 && n <= shortest / 4; ++n) {
      const double t = (shortest / n + 4) * rounds(rest * n) + join((double)rest * R, n);
      if (t < best) best = t, p.nsplit = n, p.tail = std::min(cdiv(rest, c.Hkv), p.slots);
    }
  }
  return p;
}

// workspace: the tile kernels' pieces, then the decode runs'
struct Layout {
  size_t part_o, part_ml, run_o, run_ml, shared, bytes;
};
Layout layout(const AttnCall& c, const Plan& p) {
  Layout w = {};
  const size_t rows = (size_t)p.tail * c.Hkv * p.pitch * p.nsplit;
  const size_t runs = p.rows && !p.direct ? (size_t)p.runs * 2 * 32 : 0;
  w.part_ml = w.part_o + a256(rows * c.D * sizeof(float));
  w.run_o = w.part_ml + a256(rows * sizeof(float2));
  w.run_ml = w.run_o + a256(runs * c.D * sizeof(float));
  w.shared = w.run_ml + a256(runs * sizeof(float2));
  w.bytes = w.shared + a256(runs / 64 * sizeof(Shared));
  return w;
}

int64_t tile_workgroups(const AttnCall& c, const Plan& p) { return (p.slots + p.tail * (p.nsplit - 1)) * c.Hkv; }

template <int D, typename OUT>
hipError_t launch(const AttnCall& c, const Plan& p, const Args& a, hipStream_t stream) {
  const dim3 tiles((unsigned)tile_workgroups(c, p));
  if (c.io == IO_F32) {
    if (p.share) attn_f32_kernel<D, true, OUT><<<tiles, dim3(256), 0, stream>>>(a);
    else attn_f32_kernel<D, false, OUT><<<tiles, dim3(256), 0, stream>>>(a);
  } else {
    constexpr int NW = row_waves(D);
    if (p.tiles) attn_tile_kernel<D, OUT><<<tiles, dim3(256), 0, stream>>>(a);
    if (p.rows) {
      attn_row_kernel<D, NW, OUT><<<dim3((unsigned)p.runs), dim3(NW * 64), 0, stream>>>(a);
      if (!p.direct)
        attn_row_join_kernel<D, OUT><<<dim3((unsigned)(p.runs * p.rows_a_unit)), dim3(256), 0, stream>>>(a, p.rows_a_unit);
    }
  }
  // many pieces: a workgroup a row, its lane groups sharing the pieces
  constexpr int SG = 256 / (D / 4);
  const int64_t rows = p.tail * c.Hkv * p.pitch;
  if (p.nsplit > 8) attn_join_kernel<D, SG, OUT><<<dim3((unsigned)rows), dim3(256), 0, stream>>>(a, p.rshift);
  else if (p.nsplit > 1) attn_join_kernel<D, 1, OUT><<<dim3((unsigned)(rows / SG)), dim3(256), 0, stream>>>(a, p.rshift);
  return hipGetLastError();
}

}  // namespace

int64_t attn_workgroups(const AttnCall& c) {
  const Plan p = plan(c);
  const int64_t tiles = p.tiles ? tile_workgroups(c, p) : 0, join = p.tail * c.Hkv * p.pitch;
  return std::max(std::max(tiles, join), !p.rows ? 0 : p.direct ? p.runs : p.runs * p.rows_a_unit);
}

size_t attn_workspace_bytes(const AttnCall& c) { return layout(c, plan(c)).bytes; }

hipError_t launch_attn(const AttnCall& c, hipStream_t stream) {
  const Plan p = plan(c);
  Args a;
  a.B = c.B, a.T = c.T, a.H = c.H, a.Hkv = c.Hkv, a.G = c.H / c.Hkv;
  a.pshift = __builtin_ctz((unsigned)c.page), a.max_pages = c.max_pages, a.num_pages = c.num_pages;
  a.window = c.window, a.nsplit = p.nsplit, a.few = p.rows;
  a.total = c.total, a.q_stride = c.q_stride, a.page_stride = c.page_stride;
  a.cu = c.packed ? c.cu_seqlens : nullptr;
  a.kv_lens = c.kv_lens, a.table = c.page_table;
  a.q = c.q, a.k = c.k_cache, a.v = c.v_cache, a.o = c.o, a.lse = c.lse;
  const Layout w = layout(c, p);
  char* ws = static_cast<char*>(c.workspace);
  a.part_o = reinterpret_cast<float*>(ws + w.part_o);
  a.part_ml = reinterpret_cast<float2*>(ws + w.part_ml);
  a.run_o = reinterpret_cast<float*>(ws + w.run_o);
  a.run_ml = reinterpret_cast<float2*>(ws + w.run_ml);
  a.shared = reinterpret_cast<Shared*>(ws + w.shared);
  a.direct = p.direct;
  a.scale = c.scale * 1.4426950408889634f;
  a.inv_g = 1.0 / a.G;
  a.whole = p.slots - p.tail, a.tail = p.tail, a.pitch = p.pitch;
  const bool bf = c.out == IO_BF16;
  switch (c.D) {
    case 64: return bf ? launch<64, bf16_t>(c, p, a, stream) : launch<64, float>(c, p, a, stream);
    case 128: return bf ? launch<128, bf16_t>(c, p, a, stream) : launch<128, float>(c, p, a, stream);
    case 256: return bf ? launch<256, bf16_t>(c, p, a, stream) : launch<256, float>(c, p, a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace jb
