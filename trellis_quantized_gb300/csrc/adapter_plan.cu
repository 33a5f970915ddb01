// adapter_plan.cu -- a step's rows in the order of their adapters.
//
// Sequences (rows q_start[b] .. q_start[b + 1] - 1, one adapter each) are
// counted by adapter, each gets its place behind the earlier ones of its
// adapter, and every adapter's run of rows is cut into tiles.  Rows without an
// adapter come last, as tiles of adapter -1.  One CTA: a step's batch is small,
// and one plan serves every linear of every layer.  Sequences of one adapter keep
// their order, so the same batch makes the same tiles every time (a row's last
// bits go by how many rows its tile has).
#include "adapter.cuh"

namespace exl3 {
namespace ad {

constexpr int kThreads = 1024;

// Exclusive scan over the block, 1024 threads; *total gets the sum.
__device__ int block_scan(int v, int *warp_sums, int *total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) warp_sums[w] = incl;
  __syncthreads();
  if (w == 0) {
    const int ws = warp_sums[lane];
    int wi = ws;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, wi, o);
      if (lane >= o) wi += t;
    }
    warp_sums[lane] = wi - ws;
    if (lane == 31) *total = wi;
  }
  __syncthreads();
  const int r = warp_sums[w] + incl - v;
  __syncthreads();
  return r;
}

__global__ void __launch_bounds__(kThreads) adapter_plan_kernel(const PlanArgs p) {
  __shared__ int count[kMaxCount + 1], next[kMaxCount + 1];
  __shared__ int warp_sums[32], total;
  pdl_trigger();
  pdl_wait();
  const int N1 = p.N + 1;                                  // the last: rows without an adapter
  for (int i = threadIdx.x; i < N1; i += kThreads) count[i] = 0;
  // starts that decrease or leave the call's rows: nothing is planned at all
  int bad = 0;
  for (int b = threadIdx.x; b < p.B; b += kThreads) {
    const int s = p.q_start[b], e = p.q_start[b + 1];
    bad |= s < 0 || e < s || e > p.T;
  }
  bad = __syncthreads_or(bad);
  int err = bad ? kErrBounds : 0;
  const int B = bad ? 0 : p.B;
  for (int b = threadIdx.x; b < B; b += kThreads) {
    int a = p.adapter[b];
    if (a < -1 || a >= p.N) err |= kErrExpertId;
    if (a < 0 || a >= p.N) a = p.N;
    atomicAdd(&count[a], p.q_start[b + 1] - p.q_start[b]);
  }
  err = __syncthreads_or(err);      // (any thread's bits: told apart below)
  if (threadIdx.x == 0) p.ctrl[kPlanErr] |= bad ? kErrBounds : err ? kErrExpertId : 0;

  int rows = 0, steps = 0, tcs = 0, cost = 0;                        // before this stretch of adapters
  for (int i0 = 0; i0 < N1; i0 += kThreads) {
    const int i = i0 + threadIdx.x, c = i < N1 ? count[i] : 0;
    const int first = rows + block_scan(c, warp_sums, &total);
    rows += total;
    __syncthreads();
    if (i < N1) next[i] = first;
    const int id = i < p.N ? i : -1;
    const int ns = (c + kStepRows - 1) / kStepRows, nt = (c + kTcRows - 1) / kTcRows;
    const int s0 = steps + block_scan(ns, warp_sums, &total);
    steps += total;
    __syncthreads();
    const int t0 = tcs + block_scan(nt, warp_sums, &total);
    tcs += total;
    __syncthreads();
    const int w0 = cost + block_scan(c + nt * kTileCost, warp_sums, &total);
    cost += total;
    __syncthreads();
    for (int j = 0; j < ns; ++j)
      if (s0 + j < p.max_step_tiles)
        p.step_tiles[s0 + j] = make_int4(id, first + j * kStepRows, min(kStepRows, c - j * kStepRows), 0);
    for (int j = 0; j < nt; ++j)
      if (t0 + j < p.max_tc_tiles)
        p.tc_tiles[t0 + j] =
            make_int4(id, first + j * kTcRows, min(kTcRows, c - j * kTcRows), w0 + j * (kTcRows + kTileCost));
  }
  if (threadIdx.x == 0) {
    p.ctrl[kPlanStepTiles] = min(steps, p.max_step_tiles);
    p.ctrl[kPlanTcTiles] = min(tcs, p.max_tc_tiles);
    p.ctrl[kPlanCost] = cost;
    p.ctrl[kPlanT] = p.T;
    p.ctrl[kPlanB] = p.B;
    p.ctrl[kPlanN] = p.N;
  }
  __syncthreads();
  // each sequence's place: behind its adapter's earlier ones, 1024 at a time
  __shared__ int ids[kThreads], sizes[kThreads];
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    const int b = b0 + threadIdx.x, here = min(kThreads, B - b0);
    int a = -1, n = 0;
    if (b < B) {
      a = p.adapter[b];
      if (a < 0 || a >= p.N) a = p.N;
      n = p.q_start[b + 1] - p.q_start[b];
    }
    ids[threadIdx.x] = a;
    sizes[threadIdx.x] = n;
    __syncthreads();
    int before = 0;
    for (int j = 0; j < here; ++j)                         // (every thread reads the same one)
      if (j < (int)threadIdx.x && ids[j] == a) before += sizes[j];
    if (b < B) p.base[b] = next[a] + before;
    __syncthreads();
    if (b < B) atomicAdd(&next[a], n);                     // (sums of integers: any order)
    __syncthreads();
  }
  // each row's place: its sequence is the last one that starts at or before it
  const int lo0 = B ? p.q_start[0] : 0, hi0 = B ? p.q_start[B] : 0;
  for (int t = lo0 + threadIdx.x; t < hi0; t += kThreads) {
    int lo = 0, hi = B;                                    // q_start[lo] <= t < q_start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.q_start[mid] <= t) lo = mid; else hi = mid;
    }
    p.perm[p.base[lo] + t - p.q_start[lo]] = t;
  }
}

}  // namespace ad
}  // namespace exl3

using namespace exl3;

cudaError_t exl3_launch_adapter_plan(const ad::PlanArgs &p, cudaStream_t s) {
  return launch_pdl(ad::adapter_plan_kernel, dim3(1), dim3(ad::kThreads), 0, s, p);
}
