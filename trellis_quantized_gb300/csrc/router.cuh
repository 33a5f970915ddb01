// router.cuh -- arguments of the router's kernels (router_logits.cu, route.cu).
#pragma once

#include "exl3_common.cuh"

namespace exl3 {

namespace rt {

struct Args {
  const void *logits;       // [T][E], rows `stride` elements apart
  int64_t stride;
  int T, E, topk;
  const float *bias;        // [E] or null
  int score, groups, kept, group_score, renormalise;
  float scale;
  int32_t *ids;             // [T][topk]
  float *weights;           // [T][topk]
  int group_shift;          // lanes per group, as a power of two: the most with groups * lanes <= 32
  int group_size, group_inverse;   // E / groups; 2^20 over it, rounded up
  int smem_per_warp;
};

// logits[t][e] = x[t] . w[e] (+ bias[e]).
struct LogitArgs {
  const __half *x;          // [T][k], rows x_stride elements apart
  int64_t x_stride;
  const __half *w;          // [E][k], or [2][E][k]: high and low parts
  const float *w_scale;     // [E] powers of two of the parts, or null
  const float *bias;        // [E] or null
  float *logits;            // [T][E]
  int T, E, k;
  int *err;
  // tensor cores: experts of a tile, ring stages, floats between rows of sums,
  // bytes of ring or sums
  int bn, stages, pitch, data_bytes;
  uint32_t tmem_cols;
};

}  // namespace rt
}  // namespace exl3
