/* Host side of the attention-layer entry points (norm with rotation, cache append, paged
 * attention) under AddressSanitizer and UndefinedBehaviorSanitizer: workspace queries and
 * rejected calls over shapes up to and past the documented limits, so that an overflow in the
 * planning shows.  Pointers are stand-ins that are never dereferenced; every call is one that
 * the library refuses before HIP (a short workspace, a bad field). */
#include <stdint.h>
#include <stdio.h>

#include "../../include/jetblock.h"

int hipGetDeviceCount(int* count);

static int fails = 0, checks = 0;
#define EXPECT(cond, ...) do { ++checks; if (!(cond)) { ++fails; fprintf(stderr, "line %d: ", __LINE__); \
  fprintf(stderr, __VA_ARGS__); fprintf(stderr, " [last error: %s]\n", jb_last_error()); } } while (0)
#define N(a) (sizeof(a) / sizeof(a[0]))

int main(void) {
  int ndev = 0;
  if (hipGetDeviceCount(&ndev) == 0 && ndev > 0) {
    printf("skipped: a GPU is visible and this driver passes stand-in pointers\n");
    return 0;
  }
  const int Bs[] = {1, 3, 65535, 65536, 0}, Ts[] = {0, 1, 33, 70000, 1 << 30, 0x7fffffff, -1};
  const int Hs[][2] = {{1, 1}, {12, 2}, {256, 1}, {256, 256}, {257, 1}, {6, 4}, {6, 0}};
  const int Ds[] = {64, 128, 256, 96}, pages[][2] = {{16, 1}, {64, 1024}, {4096, 1 << 18}, {4096, 0x7fffffff}, {17, 1}};
  const int kvs[] = {0, 1, 1 << 30, 0x7fffffff}, windows[] = {0, 1, 1152, 1 << 30, 0x7fffffff};
  const int64_t strides[] = {0, 1 << 20, 1LL << 41, INT64_MAX, INT64_MIN, -8};
  void* p = (void*)(uintptr_t)0x100000;
  for (size_t b = 0; b < N(Bs); ++b)
    for (size_t t = 0; t < N(Ts); ++t)
      for (size_t h = 0; h < N(Hs); ++h)
        for (size_t d = 0; d < N(Ds); ++d)
          for (size_t g = 0; g < N(pages); ++g)
            for (size_t k = 0; k < N(kvs); ++k)
              for (size_t w = 0; w < N(windows); ++w)
                for (size_t x = 0; x < N(strides); ++x)
                  for (int f32 = 0; f32 < 2; ++f32) {
                    jb_attn_shape s = {Bs[b], Ts[t], Hs[h][0], Hs[h][1], Ds[d], 64, pages[g][0], pages[g][1], 0x7fffffff,
                                       kvs[k], windows[w], f32, f32, 0, strides[x], 0, 0, g == 0 ? strides[x] : 0};
                    s.num_pages = g == 3 ? 0x7fffffff : 1 << 12;
                    const int64_t all = (int64_t)s.B * s.T;
                    const int good = b < 3 && t < 5 && h < 4 && d < 3 && g < 3 && w < 4;
                    for (int packed = 0; packed < 2; ++packed) {
                      const int64_t total = packed ? (all > 0 ? all / 2 : all) : all;
                      size_t bytes = 0;
                      jb_status st = jb_attn_paged_workspace_size(&s, total, packed, &bytes);
                      EXPECT(good || st != JB_OK, "a shape past the limits was accepted");
                      if (st == JB_OK && bytes && total) {
                        /* two pieces of every row; or only those of a last round: at least 16 rows, at most
                         * 16 pieces of the 128 rows of 3 tiles a CU (and what rounds them up to whole heads) */
                        const size_t row = (size_t)s.D * 4 + 8;
                        EXPECT(bytes >= (size_t)total * s.H * s.D * 8 ||
                                   (bytes >= 2 * 16 * row && bytes <= (size_t)(768 + 255) * 128 * 16 * row + 65536 * row),
                               "workspace %zu is neither of all rows nor of a last round", bytes);
                        st = jb_attn_paged(&s, total, packed ? p : NULL, p, p, p, p, p, 0.f, p, p, p, bytes - 1, NULL);
                        EXPECT(st == JB_ERR_WORKSPACE, "short workspace gave %s", jb_status_string(st));
                      }
                    }
                    if (g == 0 && k == 0 && w == 0) {
                      size_t bytes = 0;
                      jb_status st = jb_qk_norm_rope_backward_workspace_size(&s, &bytes);
                      EXPECT((b < 3 && t < 5 && h < 4 && d < 3) || st != JB_OK, "a shape past the limits was accepted");
                      if (st == JB_OK && s.T) {
                        EXPECT(bytes > 0 && bytes <= 2u * 256 * 1024 * 4, "backward workspace %zu", bytes);
                        st = jb_qk_norm_rope_backward(&s, p, p, p, p, p, p, 1e-6f, p, p, p, p, p, p, p, bytes - 1, NULL);
                        EXPECT(st == JB_ERR_WORKSPACE, "short workspace gave %s", jb_status_string(st));
                      }
                      s.rot = 24;
                      EXPECT(jb_qk_norm_rope(&s, p, p, p, p, p, p, 1e-6f, p, p, NULL) != JB_OK, "rot = 24 was accepted");
                      EXPECT(jb_qk_norm_rope_paged(&s, all, NULL, p, p, p, p, p, p, p, p, p, 1e-6f, p, p, p, NULL) != JB_OK,
                             "rot = 24 was accepted");
                    }
                  }
  if (fails) {
    fprintf(stderr, "%d of %d checks failed\n", fails, checks);
    return 1;
  }
  printf("host validation under sanitizers: %d checks passed\n", checks);
  return 0;
}
