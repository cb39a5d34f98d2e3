/*
 * The sequence and head norm entry points from plain C: one refusal of each,
 * and the workspace sizes.  No GPU work: every call fails its checks before
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
  lq_sequence sq = {16, 1, 1, 1, 128, 128, LQ_GATE_GDN, 0u, LQ_F32};
  lq_rows x = {arena, 128, 128}, g = {arena, 1, 1}, none = {NULL, 128, 128};
  const int32_t *cu = (const int32_t *)arena;

  if (leapquant_sequence_workspace(&sq, 1) <= 0) return fprintf(stderr, "no workspace\n"), 1;
  EXPECT(leapquant_sequence_workspace(&sq, 0), 0); /* 16 tokens go token by token */
  EXPECT(leapquant_sequence_workspace(NULL, 0), LQ_ERR_NULL);
  sq.gate = LQ_GATE_KDA;
  EXPECT(leapquant_sequence_workspace(&sq, 1), LQ_ERR_UNSUPPORTED);
  sq.gate = LQ_GATE_GDN;
  EXPECT(leapquant_sequence_forward(NULL, cu, &x, &x, &x, &g, &g, &x, NULL, NULL, NULL, 0, 0, NULL), LQ_ERR_NULL);
  EXPECT(leapquant_sequence_forward(&sq, cu, &x, &x, &none, &g, &g, &x, NULL, NULL, NULL, 0, 0, NULL), LQ_ERR_NULL);
  EXPECT(leapquant_sequence_forward(&sq, cu, &x, &x, &x, &g, &g, &x, NULL, NULL, NULL, 0, 0, NULL), LQ_ERR_ALIAS);
  EXPECT(leapquant_sequence_backward(&sq, cu, &x, &x, &g, &g, &x, NULL, &x, &x, &x, &g, &g, NULL, NULL, 0, NULL),
         LQ_ERR_NULL); /* no workspace */
  EXPECT(leapquant_sequence_backward(&sq, cu, &x, &x, &g, &g, &x, NULL, &x, &x, &x, &g, &g, NULL, arena, 64, NULL),
         LQ_ERR_SHAPE); /* too little */
  sq.dk = 64;
  EXPECT(leapquant_sequence_forward(&sq, cu, &x, &x, &x, &g, &g, &x, NULL, NULL, NULL, 0, 0, NULL),
         LQ_ERR_UNSUPPORTED);

  lq_head_norm nm = {16, 1, 1, 128, LQ_NORM_L2, LQ_F32, LQ_F32, 0, 0, 1e-6f, 1.f, NULL, NULL, NULL, NULL};
  lq_rows y = {arena + 4096, 128, 128};
  EXPECT(leapquant_head_norm(NULL, &x, &x, &y, &y, NULL), LQ_ERR_NULL);
  EXPECT(leapquant_head_norm(&nm, &x, &x, &y, &y, NULL), LQ_ERR_ALIAS); /* both outputs in one place */
  EXPECT(leapquant_head_norm_backward(&nm, &x, &x, &y, &y, &x, &y, NULL, NULL, NULL, 0, NULL), LQ_ERR_ALIAS);
  if (leapquant_head_norm_workspace(16, 1, 1) <= 0) return fprintf(stderr, "no norm workspace\n"), 1;
  EXPECT(leapquant_head_norm_workspace(-1, 1, 1), LQ_ERR_SHAPE);
  nm.rot = 64;
  EXPECT(leapquant_head_norm(&nm, &x, &x, &y, &y, NULL), LQ_ERR_NULL); /* a rotation without positions */
  nm.eps = 0.f;
  EXPECT(leapquant_head_norm(&nm, &x, &x, &y, &y, NULL), LQ_ERR_SHAPE);
  printf("sequence checks passed\n");
  return 0;
}
