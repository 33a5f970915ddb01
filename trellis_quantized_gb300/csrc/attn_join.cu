// attn_join.cu -- joins the parts of the units that the attention kernels
// cut between CTAs:
//
//   w_c = l_c 2^(m_c - max_c m_c),  y = sum_c w_c y_c / sum_c w_c
//
// with the largest score m_c of a part and its sum of weights l_c, which are
// kept apart: at scores past 2^20, log2(l_c) would be lost in their sum.
//
// A CTA leaves at most one unit unfinished for its successors: the blocks
// (c, .) share the rows of the one that CTA c left, if there is one, up to 8
// each after the tensor-core kernel and 2 after the step kernel.  A warp per
// row works out the parts' weights, then the block adds: a thread holds
// four neighbouring elements of a row, and where the rows do not fill the
// block several groups of threads share the parts (a single user's long
// sequence is cut into one per CTA of its key head, up to the whole grid) and
// are added at the end in their order.  After steps bound by the latency of
// dependent reads of L2, where the parts were just written: the record, then
// maxima and sums together with the first eight parts of every thread (8 users
// x 5 tokens at 256-wide heads: the call takes 37.4 us; 39.9 with 8 rows to a
// block and the parts read after them).
//
// Joining inside the attention kernel, by the CTA that arrived last, cost 115
// us for eight sequences of up to 20,000 tokens at 256-wide heads against 66
// us with a kernel of its own: one CTA has too few reads in flight.
#include "attn_common.cuh"

namespace exl3 {
namespace attn {

constexpr int kJoinThreads = 256, kJoinRows = 8, kJoinMaxCtas = 512;
constexpr int kRead = 8;                     // parts that a thread reads at once

template <int D>
__global__ void __launch_bounds__(kJoinThreads, 4)
    attn_join_kernel(const Args a, int ctas, int tile_rows) {
  constexpr int C4 = D / 4;                  // threads per row
  __shared__ float weight[kJoinRows][kJoinMaxCtas];
  __shared__ float row_lse[kJoinRows];
  __shared__ float4 red[kJoinThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int first = blockIdx.x;
  pdl_trigger();
  pdl_wait();
  const int4 cut = __ldcg(reinterpret_cast<const int4 *>(a.cuts + first));   // rows, last, t, h
  const int block_rows = max(2, (cut.x + (int)gridDim.y - 1) / (int)gridDim.y);    // at most kJoinRows
  const int r0 = blockIdx.y * block_rows, rows = min(cut.x - r0, block_rows);
  if (rows <= 0) return;
  const int parts = min(min(cut.y, ctas - 1) - first + 1, kJoinMaxCtas);
  // row r of part p: slot 1 of the first CTA, slot 0 of the others
  const auto place = [&](int p, int r) { return ((int64_t)(first + p) * 2 + (p == 0 ? 1 : 0)) * tile_rows + r0 + r; };
  const int items = rows * C4;
  const int groups = items < kJoinThreads ? kJoinThreads / items : 1;
  const int g = items < kJoinThreads ? tid / items : 0;
  int i = items < kJoinThreads ? tid - g * items : tid;
  // a thread's values of kRead parts from part p on
  const auto read = [&](int p, float4(&v)[kRead]) {
#pragma unroll
    for (int k = 0; k < kRead; ++k, p += groups)
      v[k] = g < groups && i < items && p < parts
                 ? __ldcg(reinterpret_cast<const float4 *>(a.part_o + place(p, i / C4) * D + (i % C4) * 4))
                 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  };
  float4 v[kRead];
  read(g, v);                                  // under way while the weights are worked out
  for (int r = warp; r < rows; r += kJoinThreads / 32) {
    // (between the two passes the sums stay in the weights' places, the first
    // 96 parts' maxima in registers)
    const auto take = [&](int p) {
      const float2 ml = __ldcg(a.part_ml + place(p, r));
      weight[r][p] = ml.y;
      return ml.x;
    };
    float m[3], mx = neg_inf();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      m[k] = lane + 32 * k < parts ? take(lane + 32 * k) : neg_inf();
      mx = fmaxf(mx, m[k]);
    }
    for (int p = lane + 96; p < parts; p += 32) mx = fmaxf(mx, take(p));
#pragma unroll
    for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    float sum = 0.0f;
    const auto weigh = [&](int p, float m_p) {
      const float f = weight[r][p] * (m_p == neg_inf() ? 0.0f : exp2_approx(m_p - mx));   // (a NaN sum stays)
      weight[r][p] = f;
      sum += f;
    };
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (lane + 32 * k < parts) weigh(lane + 32 * k, m[k]);
    for (int p = lane + 96; p < parts; p += 32) weigh(p, __ldcg(a.part_ml + place(p, r)).x);
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);  // (NaN stays)
    __syncwarp();
    for (int p = lane; p < parts; p += 32) weight[r][p] *= inv;
    if (lane == 0) row_lse[r] = natural_lse(mx, sum);
  }
  __syncthreads();
  for (int i0 = 0; i0 < items; i0 += kJoinThreads) {
    if (i0) i += kJoinThreads;
    const bool mine = g < groups && i < items;
    const int r = mine ? i / C4 : 0, c4 = (i % C4) * 4;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int p0 = g; p0 < parts; p0 += kRead * groups) {
      if (i0 || p0 != g) read(p0, v);
#pragma unroll
      for (int k = 0; k < kRead; ++k) {
        const int p = p0 + k * groups;
        const float f = p < parts ? weight[r][p] : 0.0f;
        acc.x = fmaf(f, v[k].x, acc.x);
        acc.y = fmaf(f, v[k].y, acc.y);
        acc.z = fmaf(f, v[k].z, acc.z);
        acc.w = fmaf(f, v[k].w, acc.w);
      }
    }
    if (groups > 1) {
      red[tid] = acc;
      __syncthreads();
      if (g == 0)
        for (int k = 1; k < groups; ++k) {
          const float4 v = red[k * items + i];
          acc.x += v.x;
          acc.y += v.y;
          acc.z += v.z;
          acc.w += v.w;
        }
    }
    if (mine && g == 0) {
      const int64_t head = out_head(a, cut.z, cut.w, r0 + r);
      store4(a, head * D + c4, acc);
      if (a.lse && c4 == 0) a.lse[head] = row_lse[r];
    }
  }
}

}  // namespace attn
}  // namespace exl3

// `ctas`: the attention launch's grid; `tile_rows`: rows of its units.
cudaError_t exl3_launch_attn_join(const exl3::attn::Args &a, int D, int ctas, int tile_rows, cudaStream_t s) {
  using namespace exl3::attn;
  if (ctas > kJoinMaxCtas) return cudaErrorInvalidConfiguration;
  const dim3 grid(ctas, tile_rows > 16 ? tile_rows / kJoinRows : tile_rows / 2), block(kJoinThreads);
  switch (D) {
    case 64: return exl3::launch_pdl(attn_join_kernel<64>, grid, block, 0, s, a, ctas, tile_rows);
    case 128: return exl3::launch_pdl(attn_join_kernel<128>, grid, block, 0, s, a, ctas, tile_rows);
    default: return exl3::launch_pdl(attn_join_kernel<256>, grid, block, 0, s, a, ctas, tile_rows);
  }
}
