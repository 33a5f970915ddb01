// attn_join.cu -- joins the parts of the units that the attention kernels
// cut between CTAs:
//
//   y = sum_c 2^(lse_c - max) y_c / sum_c 2^(lse_c - max)
//
// A CTA leaves at most one unit unfinished for its successors, so the records
// of all CTAs (at most a few hundred) give the list of rows; every block works
// the list out for itself with one scan, and a warp takes a row: its lanes
// first hold the parts' weights, then walk over the parts together, eight
// rows of 4 D bytes in flight.  Bound by the latency of those reads (they are
// in L2, just written): a long sequence of one user is cut into up to 76 parts
// per key head.  Joining inside the attention kernel, by the CTA that arrived
// last, cost 115 us for eight sequences of up to 20,000 tokens at 256-wide
// heads against 72 us this way: one CTA has too few loads in flight.
#include "attn_common.cuh"

namespace exl3 {
namespace attn {

constexpr int kJoinWarps = 8, kJoinMaxCtas = 1024;

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32, 6) attn_join_kernel(const Args a, int ctas, int tile_rows) {
  constexpr int V = D / 32;                  // elements per lane: 2, 4 or 8
  __shared__ int first[kJoinMaxCtas + 1];    // rows before each CTA's record
  __shared__ int sums[kJoinWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  pdl_wait();
  int run = 0;
  for (int c0 = 0; c0 < ctas; c0 += kJoinWarps * 32) {
    const int c = c0 + tid;
    const int rows = c < ctas ? __ldcg(&a.cuts[c].rows) : 0;
    int inc = rows;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += o;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int before = run, all = 0;
    for (int w = 0; w < kJoinWarps; ++w) {
      before += w < warp ? sums[w] : 0;
      all += sums[w];
    }
    if (c < ctas) first[c] = before + inc - rows;
    run += all;
    __syncthreads();
  }
  const int total = run;
  for (int i = blockIdx.x * kJoinWarps + warp; i < total; i += gridDim.x * kJoinWarps) {
    int lo = 0, hi = ctas - 1;               // the last record that begins at or before row i
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (first[mid] <= i) lo = mid;
      else hi = mid - 1;
    }
    const Cut cut = a.cuts[lo];
    const int r = i - first[lo], parts = min(cut.last, ctas - 1) - lo + 1;
    const auto place = [&](int p) { return ((int64_t)(lo + p) * 2 + (p == 0 ? 1 : 0)) * tile_rows + r; };
    float mx = neg_inf();
    for (int p = lane; p < parts; p += 32) mx = fmaxf(mx, __ldcg(a.part_lse + place(p)));
#pragma unroll
    for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    float sum = 0.0f, acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.0f;
    for (int p0 = 0; p0 < parts; p0 += 32) {
      float wgt = 0.0f;
      if (p0 + lane < parts) {
        const float ls = __ldcg(a.part_lse + place(p0 + lane));
        wgt = ls == neg_inf() ? 0.0f : exp2_approx(ls - mx);
      }
      const int n = min(32, parts - p0);
#pragma unroll 4
      for (int k = 0; k < n; ++k) {
        const float f = __shfl_sync(0xffffffffu, wgt, k);
        const float *src = a.part_o + place(p0 + k) * D + lane * V;
        sum += f;
        if constexpr (V == 2) {
          const float2 v = __ldcg(reinterpret_cast<const float2 *>(src));
          acc[0] = fmaf(f, v.x, acc[0]);
          acc[1] = fmaf(f, v.y, acc[1]);
        } else {
#pragma unroll
          for (int j = 0; j < V; j += 4) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(src + j));
            acc[j] = fmaf(f, v.x, acc[j]);
            acc[j + 1] = fmaf(f, v.y, acc[j + 1]);
            acc[j + 2] = fmaf(f, v.z, acc[j + 2]);
            acc[j + 3] = fmaf(f, v.w, acc[j + 3]);
          }
        }
      }
    }
    const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);    // (NaN stays)
    const int64_t head = out_head(a, cut.t, cut.h, r);
    if constexpr (V == 2) {
      const float2 o = make_float2(acc[0] * inv, acc[1] * inv);
      if (a.f32out) *reinterpret_cast<float2 *>(static_cast<float *>(a.y) + head * D + lane * V) = o;
      else *reinterpret_cast<__half2 *>(static_cast<__half *>(a.y) + head * D + lane * V) = __floats2half2_rn(o.x, o.y);
    } else {
#pragma unroll
      for (int j = 0; j < V; j += 4)
        store4(a, head * D + lane * V + j,
               make_float4(acc[j] * inv, acc[j + 1] * inv, acc[j + 2] * inv, acc[j + 3] * inv));
    }
    if (a.lse && lane == 0) a.lse[head] = sum == 0.0f ? neg_inf() : (mx + log2f(sum)) * 0.69314718055994530942f;
  }
}

}  // namespace attn
}  // namespace exl3

// `ctas`: the attention launch's grid; `tile_rows`: rows of its units.
cudaError_t exl3_launch_attn_join(const exl3::attn::Args &a, int D, int ctas, int tile_rows, cudaStream_t s) {
  using namespace exl3::attn;
  if (ctas > kJoinMaxCtas) return cudaErrorInvalidConfiguration;
  // a warp per row as far as that many can be resident
  const int most = (ctas * tile_rows + kJoinWarps - 1) / kJoinWarps, resident = 6 * exl3_sm_count();
  const dim3 grid(most < resident ? most : resident), block(kJoinWarps * 32);
  switch (D) {
    case 64: return exl3::launch_pdl(attn_join_kernel<64>, grid, block, 0, s, a, ctas, tile_rows);
    case 128: return exl3::launch_pdl(attn_join_kernel<128>, grid, block, 0, s, a, ctas, tile_rows);
    default: return exl3::launch_pdl(attn_join_kernel<256>, grid, block, 0, s, a, ctas, tile_rows);
  }
}
