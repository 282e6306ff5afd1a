/*
 * Sanitizer driver for the host side of the operators on rows of scores: the
 * sizing arithmetic and the checks of views, lists, states and CSRs over
 * extreme sizes. Every call made here returns before any device work (a
 * refusal, a pure sizing call, or nothing to do), so the driver needs no GPU.
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

static const int64_t kSizes[] = {0, 1, 2, 255, 1024, 8192, 2000000, 4194303, 16777216, 2147483646LL,
                                 2147483647LL, 2147483648LL, INT64_MAX / 4, INT64_MAX, -1, INT64_MIN};
enum { N = (int)(sizeof kSizes / sizeof *kSizes) };
static const int32_t kKs[] = {INT32_MIN, -1, 0, 1, 7, 256, 257, 1024, 1025, INT32_MAX};
enum { K = (int)(sizeof kKs / sizeof *kKs) };

static void sizing(void) {
  for (int i = 0; i < N; ++i)
    for (int j = 0; j < N; ++j)
      for (int k = 0; k < K; ++k) {
        size_t b = 0;
        CHECK(is_status(sps_select_workspace_size(kSizes[i], kSizes[j], kKs[k], &b)));
        for (int m = 0; m < K; ++m)
          CHECK(is_status(sps_beam_workspace_size(kSizes[i], kSizes[j], kKs[m], kKs[k], &b)));
        CHECK(is_status(sps_distill_workspace_size(kSizes[i], kKs[k], &b)));
        CHECK(is_status(sps_cosine_grad_both_workspace_size(kSizes[i], kSizes[j], &b)));
      }
}

/* views whose sizes are refused, or whose workspaces are: never a launch */
static void views(void) {
  for (int i = 0; i < N; ++i)
    for (int j = 0; j < N; ++j)
      for (int l = 0; l < N; ++l) {
        sps_scores v;
        memset(&v, 0, sizeof v);
        v.data = at(0x10000);
        v.dtype = (int32_t)(i + j + l) % 5 - 1;
        v.n_rows = kSizes[i];
        v.n_cols = kSizes[j];
        v.ld = kSizes[l];
        v.col_begin = kSizes[(i + l) % N];
        CHECK(is_status(sps_select_chunk(&v, NULL, 8, 1, NULL, NULL, NULL, 0, NULL)));
        CHECK(is_status(sps_beam_select(&v, NULL, 1, 8, NULL, NULL, NULL, NULL, 0, NULL)));
        CHECK(is_status(sps_distill_rows(&v, at(0x10000), at(0x10000), NULL, 8, 1.0f, NULL, NULL,
                                         at(0x10000), v.dtype, kSizes[(j + l) % N], at(0x10000),
                                         SIZE_MAX, NULL)));
        sps_csr q = {kSizes[i], 100, kSizes[l], at(0x10000), at(0x10000), at(0x10000)};
        sps_csr m = {kSizes[j], 100, kSizes[(l + 3) % N], at(0x10000), at(0x10000), at(0x10000)};
        CHECK(is_status(sps_cosine_grad_both(&q, &m, &v, at(0x10000), at(0x10000), NULL, 0, NULL)));
        CHECK(is_status(sps_cosine_grad(&q, NULL, 0, &v, 0, 1, NULL, NULL, 0, NULL)));
        CHECK(is_status(sps_cosine_grad_values(&q, NULL, NULL, NULL)));
      }
}

static void states(void) {
  for (int i = 0; i < N; ++i)
    for (int j = 0; j < N; ++j)
      for (int l = 0; l < N; ++l) {
        /* the second state's output overlaps its source, or its sizes are refused */
        sps_state s[2] = {{at(0x10000), at(0x80000000u), 4, 4, 4},
                          {at(0x20000), at(0x20000), kSizes[i], kSizes[j], kSizes[l]}};
        if (kSizes[i] == 0) s[1].dst_stride = -1;
        CHECK(sps_reorder_states(s, 2, at(0x10000), 8, 8, NULL) < 0);
        CHECK(is_status(sps_reorder_states(s, 2, NULL, kSizes[j], kSizes[l], NULL)));
        CHECK(is_status(sps_reorder_states(NULL, 2, at(0x10000), kSizes[j], kSizes[l], NULL)));
      }
}

static void lists(void) {
  const float taus[] = {0.0f, -1.0f, 1e-30f, 1e30f, NAN};
  for (int i = 0; i < N; ++i)
    for (int k = 0; k < K; ++k) {
      sps_distill *h = at(1);
      for (int t = 0; t < 5; ++t)
        CHECK(sps_distill_prepare(at(0x10000), at(0x10000), NULL, kSizes[i], kKs[k], 100, taus[t],
                                  at(0x10000), SIZE_MAX, NULL, &h) < 0);
      CHECK(h == NULL);
      CHECK(is_status(sps_beam_join(NULL, NULL, kSizes[i], kKs[k], kKs[(k + 3) % K],
                                    kKs[(k + 5) % K], NULL, NULL, NULL, NULL)));
    }
  /* an empty batch's handle lives and dies without a device */
  sps_distill *h = NULL;
  CHECK(sps_distill_prepare(NULL, NULL, NULL, 0, 4, 100, 1.0f, NULL, 0, NULL, &h) == SPS_OK && h);
  sps_scores v = {NULL, SPS_F32, 0, 100, 100, 0};
  CHECK(sps_distill_chunk(h, &v, 1, NULL) == SPS_OK);
  CHECK(sps_distill_loss(h, NULL, NULL, NULL) == SPS_OK);
  CHECK(sps_distill_chunk_grad(h, &v, NULL, NULL, SPS_F32, 100, NULL) == SPS_OK);
  v.col_begin = 1;
  CHECK(sps_distill_chunk(h, &v, 1, NULL) == SPS_ERR_INVALID_ARGUMENT);
  sps_distill_destroy(h);
}

int main(void) {
  sizing();
  views();
  states();
  lists();
  printf("clean\n");
  return 0;
}
