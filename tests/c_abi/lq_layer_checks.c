/*
 * The convolution, scan and block norm entry points from plain C: one refusal of
 * each, and the workspace sizes.  No GPU work: every call fails its checks before
 * anything is launched, and no pointer is dereferenced.
 */
#include <stdint.h>
#include <stdio.h>

#include "leapquant.h"

#define EXPECT(call, want)                                                       \
  do {                                                                           \
    const long long rc_ = (long long)(call);                                     \
    if (rc_ != (want)) {                                                         \
      fprintf(stderr, "%s returned %lld, expected %d\n", #call, rc_, (int)(want)); \
      return 1;                                                                  \
    }                                                                            \
  } while (0)

static float arena[1 << 16] __attribute__((aligned(64)));

int main(void) {
  float *const w = arena, *const far = arena + (1 << 15);
  const int32_t *cu = (const int32_t *)(arena + 64);
  lq_rows x = {arena + 1024, 16, 16}, y = {far, 16, 16};

  lq_conv cv = {4, 1, 16, 4, LQ_ACT_SILU, LQ_F32, w, NULL};
  EXPECT(leapquant_conv_forward(NULL, cu, &x, &y, NULL, NULL, NULL), LQ_ERR_NULL);
  EXPECT(leapquant_conv_forward(&cv, cu, &x, &x, NULL, NULL, NULL), LQ_ERR_ALIAS);
  EXPECT(leapquant_conv_step(&cv, NULL, 3, &x, &y, w, w, NULL), LQ_ERR_SHAPE); /* four rows, three slots */
  EXPECT(leapquant_conv_backward(&cv, cu, &x, &y, &x, NULL, NULL, NULL, NULL, NULL, NULL, 0, NULL), LQ_ERR_ALIAS);
  if (leapquant_conv_workspace(&cv) <= 0) return fprintf(stderr, "no convolution workspace\n"), 1;
  cv.width = 5;
  EXPECT(leapquant_conv_workspace(&cv), LQ_ERR_UNSUPPORTED);

  lq_scan sc = {4, 1, 16, 16, 1, LQ_F32, LQ_SCAN_SOFTPLUS, w, NULL, NULL};
  EXPECT(leapquant_scan_workspace(&sc, 0), 0);
  if (leapquant_scan_workspace(&sc, 1) <= 0) return fprintf(stderr, "no scan workspace\n"), 1;
  EXPECT(leapquant_scan_forward(&sc, cu, &x, &x, &x, &x, NULL, &x, NULL, NULL, NULL, 0, 0, NULL), LQ_ERR_ALIAS);
  EXPECT(leapquant_scan_forward(&sc, cu, &x, &x, &x, &x, NULL, &y, NULL, NULL, NULL, 0, 1, NULL), LQ_ERR_NULL);
  EXPECT(leapquant_scan_step(&sc, NULL, 4, &x, &x, &x, &x, NULL, &y, NULL, NULL, NULL), LQ_ERR_NULL);
  EXPECT(leapquant_scan_backward(&sc, cu, &x, &x, &x, &x, NULL, &x, &y, &y, &y, &y, NULL, w, NULL, NULL, NULL, NULL,
                                 far, 16, NULL), LQ_ERR_SHAPE); /* too little workspace */
  sc.states = 12;
  EXPECT(leapquant_scan_workspace(&sc, 0), LQ_ERR_UNSUPPORTED);

  lq_block_norm bn = {4, 1, 16, LQ_F32, LQ_F32, LQ_ACT_NONE, 1, 1e-6f, 1.f, NULL, NULL};
  EXPECT(leapquant_block_norm(&bn, &x, NULL, NULL, NULL, NULL, NULL), LQ_ERR_NULL);
  EXPECT(leapquant_block_norm(&bn, &x, NULL, NULL, &y, &y, NULL), LQ_ERR_ALIAS);
  EXPECT(leapquant_block_norm_backward(&bn, &x, NULL, NULL, NULL, NULL, &y, NULL, NULL, NULL, NULL, NULL, 0, NULL),
         LQ_ERR_NULL);
  if (leapquant_block_norm_workspace(4, 1, 16) <= 0) return fprintf(stderr, "no norm workspace\n"), 1;
  bn.dim = 12;
  EXPECT(leapquant_block_norm(&bn, &x, NULL, NULL, &y, NULL, NULL), LQ_ERR_SHAPE);
  printf("layer checks passed\n");
  return 0;
}
