// head_transform.cuh -- arguments of the head transform kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace exl3 {
namespace ht {

struct Args {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;   // elements between tokens
  int T, Hq, Hkv;
  const void *q_norm, *k_norm;            // fp16 weights or null
  float eps, magnitude;
  const float *inv_freq;
  int rotary_dim, layout;
  const int *positions;                   // or null (append: the cache index)
  void *q_out, *k_out;
  int f32out;
  // append
  const int *q_start, *kv_len, *table;
  int B, max_pages, page_size, num_pages;
  void *k_cache, *v_cache;
  int64_t stride_page, stride_token, stride_head;
  int *err;
};

}  // namespace ht
}  // namespace exl3

cudaError_t exl3_launch_head_transform(const exl3::ht::Args &a, int D, bool f32in, bool append, cudaStream_t s);
