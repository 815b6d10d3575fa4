/* Host side of the entry points for long contexts (a cache in 8 bits, selected pages) under
 * AddressSanitizer and UndefinedBehaviorSanitizer, as layer_driver.c does for the others:
 * workspace queries and rejected calls over shapes up to and past the documented limits.
 * Pointers are stand-ins that are never dereferenced. */
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
  const int counts[] = {1, 32, 1 << 18, 1 << 26, 0x7fffffff, 0, -1};
  const int64_t strides[] = {0, 1 << 20, 1LL << 41, INT64_MAX, INT64_MIN, -8};
  void* p = (void*)(uintptr_t)0x100000;
  for (size_t b = 0; b < N(Bs); ++b)
    for (size_t t = 0; t < N(Ts); ++t)
      for (size_t h = 0; h < N(Hs); ++h)
        for (size_t d = 0; d < N(Ds); ++d)
          for (size_t g = 0; g < N(pages); ++g)
            for (size_t n = 0; n < N(counts); ++n)
              for (size_t x = 0; x < N(strides); ++x)
                for (int f32 = 0; f32 < 2; ++f32)
                  for (int bits8 = 0; bits8 < 2; ++bits8) {
                    jb_attn_shape s = {Bs[b], Ts[t], Hs[h][0], Hs[h][1], Ds[d], 64, pages[g][0], pages[g][1], 1 << 12,
                                       0, 0, f32, f32, 0, strides[x], 0, 0, g == 0 ? strides[x] : 0};
                    const int64_t all = (int64_t)s.B * s.T;
                    const int good = b < 3 && t < 5 && h < 4 && d < 3 && g < 3;
                    for (int packed = 0; packed < 2; ++packed) {
                      const int64_t total = packed ? (all > 0 ? all / 2 : all) : all;
                      const int32_t* cu = packed ? p : NULL;
                      size_t bytes = 0;
                      if (n == 0 && bits8) {
                        jb_status st = jb_attn_paged8_workspace_size(&s, total, packed, &bytes);
                        EXPECT(good || st != JB_OK, "a shape past the limits was accepted");
                        if (st == JB_OK && bytes && total) {
                          st = jb_attn_paged8(&s, total, cu, p, p, p, p, p, p, p, 0, 0.f, p, p, p, bytes - 1, NULL);
                          EXPECT(st == JB_ERR_WORKSPACE, "short workspace gave %s", jb_status_string(st));
                        }
                        s.rot = 24;
                        st = jb_qk_norm_rope_paged8(&s, total, cu, p, p, p, p, p, p, p, p, p, 1e-6f, p, p, p, p, p, strides[x], NULL);
                        EXPECT(st != JB_OK, "rot = 24 was accepted");
                        s.rot = 64;
                        /* every check of a good shape but the last pointer's */
                        st = jb_qk_norm_rope_paged8(&s, total, cu, p, p, p, p, p, p, p, p, p, 1e-6f, p, p, p, p, NULL, strides[x], NULL);
                        EXPECT(st != JB_OK || total == 0, "no v_scales were accepted");
                      }
                      s.flags = bits8 ? JB_CACHE_E4M3 : 0;
                      jb_status st = jb_attn_blocks_workspace_size(&s, total, packed, counts[n], &bytes);
                      EXPECT((good && n < 4) || st != JB_OK, "a shape past the limits was accepted");
                      if (st == JB_OK && total && (f32 || counts[n] > 2048))
                        EXPECT(bytes >= (size_t)total * s.Hkv * (counts[n] + 1) * 4, "workspace %zu holds no lists", bytes);
                      if (st == JB_OK && total && bytes) {
                        uint8_t* e = bits8 ? p : NULL;
                        st = jb_attn_blocks(&s, total, cu, p, p, p, p, p, e, e, 0, p, counts[n], 0.f, p, p, p, bytes - 1, NULL);
                        EXPECT(st == JB_ERR_WORKSPACE, "short workspace gave %s", jb_status_string(st));
                      }
                      st = jb_block_scores(&s, total, cu, p, p, p, p, bits8 ? p : NULL, strides[x], NULL, p, NULL);
                      EXPECT(st != JB_OK || total == 0, "no means were accepted");
                      s.flags = 0;
                      st = jb_block_select(&s, total, cu, p, p, counts[n], 0, 1, NULL, NULL);
                      EXPECT(st != JB_OK || total == 0, "no blocks were accepted");
                    }
                  }
  if (fails) {
    fprintf(stderr, "%d of %d checks failed\n", fails, checks);
    return 1;
  }
  printf("host validation under sanitizers: %d checks passed\n", checks);
  return 0;
}
