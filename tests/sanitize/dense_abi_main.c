/*
 * Sanitizer driver for the host side of the operators on dense rows: the
 * sizing arithmetic, the plans of tiles and splits, and the checks of rows,
 * views and gradients over extreme sizes. Every call made here returns before
 * any device work (a refusal or a pure sizing call), so the driver needs no
 * GPU.
 */
#include <limits.h>
#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "sps.h"

#define CHECK(c)                                                              \
  do {                                                                        \
    if (!(c)) {                                                               \
      fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #c);         \
      exit(2);                                                                \
    }                                                                         \
  } while (0)

static int is_status(sps_status s) { return s <= 0 && s >= SPS_ERR_UNSUPPORTED; }
static void *at(uintptr_t a) { return (void *)a; }

static const int64_t kSizes[] = {0, 1, 2, 15, 16, 127, 255, 257, 4095, 65536, 65537, 131072, 131073,
                                 2000000, 4194304, 4194305, 2147483646LL, 2147483647LL, 2147483648LL,
                                 INT64_MAX / 4, INT64_MAX, -1, INT64_MIN};
enum { N = (int)(sizeof kSizes / sizeof *kSizes) };

static sps_scores view(uintptr_t p, int32_t dtype, int64_t rows, int64_t cols, int64_t ld) {
  sps_scores v;
  memset(&v, 0, sizeof v);
  v.data = at(p);
  v.dtype = dtype;
  v.n_rows = rows;
  v.n_cols = cols;
  v.ld = ld;
  return v;
}

/* every size of queries, items and dims: a size or a refusal, and as large a
 * workspace for more gradients */
static void sizing(void) {
  for (int i = 0; i < N; ++i)
    for (int j = 0; j < N; ++j)
      for (int k = 0; k < N; ++k)
        for (int32_t t = -1; t <= 3; ++t) {
          sps_scores q = view(0x10000, t, kSizes[i], kSizes[k], kSizes[k]);
          sps_scores m = view(0x20000, t, kSizes[j], kSizes[k], kSizes[k]);
          size_t alone = 0, one = 0, both = 0;
          sps_status s = sps_dense_ce_workspace_size(&q, &m, 0, 0, &alone);
          CHECK(is_status(s));
          CHECK(s == sps_dense_ce_workspace_size(&q, &m, 1, 0, &one));
          CHECK(s == sps_dense_ce_workspace_size(&q, &m, 1, 1, &both));
          if (s == SPS_OK) CHECK(one <= both);
          /* no workspace: refused, or nothing to do (no rows: not called here) */
          if (s == SPS_OK && kSizes[i] > 0 && kSizes[j] > 0) {
            CHECK(sps_dense_ce(&q, &m, at(0x1000), NULL, 1.0f, NULL, at(1ull << 60), NULL, 0, NULL, 0, t,
                               NULL, 0, NULL) == SPS_ERR_INVALID_ARGUMENT);
            CHECK(sps_dense_ce(&q, &m, at(0x1000), NULL, 1.0f, NULL, at(1ull << 60), NULL, 0, NULL, 0, t,
                               at(0x100000), 255, NULL) == SPS_ERR_WORKSPACE_TOO_SMALL);
          }
        }
}

/* 8-bit rows of every size and ld without values, and outputs inside them */
static void rows8(void) {
  for (int i = 0; i < N; ++i)
    for (int j = 0; j < N; ++j)
      for (int l = 0; l < N; ++l) {
        sps_int8_rows r;
        memset(&r, 0, sizeof r);
        r.n_rows = kSizes[i];
        r.dim = kSizes[j];
        r.ld = kSizes[l];
        sps_int8_rows o = r;
        o.values = at(0x100000);
        o.scales = at(0x200000);
        CHECK(is_status(sps_dequantize_rows(&r, NULL, SPS_F32, kSizes[l], NULL)));
        if (r.n_rows > 0) CHECK(sps_dequantize_rows(&r, NULL, SPS_F32, kSizes[l], NULL) != SPS_OK);
        if (r.n_rows > 0)
          CHECK(sps_dequantize_rows(&o, at(0x100000), SPS_F32, kSizes[l], NULL) != SPS_OK);
        sps_scores x = view(0x100000, SPS_F16, kSizes[i], kSizes[j], kSizes[j]);
        if (x.n_rows > 0) CHECK(sps_quantize_rows(&x, at(0x100000), kSizes[l], at(0x40), NULL) != SPS_OK);
        if (r.n_rows > 0) CHECK(sps_int8_scores(&r, &o, at(0x400), SPS_BF16, kSizes[l], NULL) != SPS_OK);
        if (r.n_rows > 0)
          CHECK(sps_int8_scores(&o, &o, at(0x100000), SPS_F32, kSizes[i], NULL) != SPS_OK);
      }
}

int main(void) {
  sizing();
  rows8();
  printf("clean\n");
  return 0;
}
