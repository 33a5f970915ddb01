// adapter_step.cu -- low-rank adapters on few rows:
//
//   out[t] = y[t] + scale (x[t] A^T) B^T
//
// A tile is up to 16 rows of one adapter; a cluster of S CTAs takes it.  First
// each CTA forms h = x A^T over its share of k, the cluster adds the shares up
// (distributed shared memory, in the order of the CTAs: no atomics, no second
// launch), then each CTA adds h B^T to its share of the n columns.  What bounds
// it is one read of A, B, y and one write of out; with one row, start-up and
// the chain plan -> x, A -> h -> out.
//
// Products are mma.sync m16n8k16 on fragments loaded straight from global
// memory: a sum does not depend on the order that its terms are named in, so a
// lane takes eight neighbouring k of x and A (or eight ranks of h and B) and
// feeds them to two products; every load is 16 bytes and nothing passes
// through shared memory.  (tcgen05 wants 64 or 128 rows; these tiles have one to
// 16.)  The columns of B are dealt out so that a lane ends up with eight
// neighbouring outputs.
//
// h is an operand of the second product in two fp16 parts, hi + lo, after each
// row is brought to [2^14, 2^15) by a power of two: 22 bits of every h, so that
// an fp32 out is as good as its fp32 sums.  Up to eight rows (most tiles of a step)
// hi takes the upper half of the product's 16 rows and lo the lower, and the lane
// that holds both results adds them: one product where 9 to 16 rows take two (64 users
// of ranks to 64, 17408 columns: 16.0 us, 17.9 with two products for every tile).
#include "adapter.cuh"
#include "tc_ptx.cuh"

namespace exl3 {
namespace ad {

constexpr int kStepThreads = 256, kStepWarps = 8;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two products over 32 values of the summed index, eight neighbours per lane.
__device__ __forceinline__ void mma_pair(float (&d)[4], const uint4 &lo, const uint4 &hi, const uint4 &b) {
  mma16816(d, lo.x, hi.x, lo.y, hi.y, b.x, b.y);
  mma16816(d, lo.z, hi.z, lo.w, hi.w, b.z, b.w);
}

__device__ __forceinline__ uint4 load16(const __half *p, bool ok) {
  return ok ? __ldg(reinterpret_cast<const uint4 *>(p)) : make_uint4(0, 0, 0, 0);
}

// Eight neighbouring elements of y, and out = y + v.
template <bool F32>
struct Out;
template <>
struct Out<false> {
  uint4 y;
  __device__ __forceinline__ void load(const void *p, int64_t at) {
    y = *reinterpret_cast<const uint4 *>(static_cast<const __half *>(p) + at);
  }
  __device__ __forceinline__ void add_store(const float (&v)[8], void *p, int64_t at) const {
    uint4 o = y;
    __half2 *h = reinterpret_cast<__half2 *>(&o);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 t = __half22float2(h[j]);
      h[j] = __floats2half2_rn(t.x + v[2 * j], t.y + v[2 * j + 1]);
    }
    *reinterpret_cast<uint4 *>(static_cast<__half *>(p) + at) = o;
  }
};
template <>
struct Out<true> {
  float4 y0, y1;
  __device__ __forceinline__ void load(const void *p, int64_t at) {
    const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
    y0 = src[0];
    y1 = src[1];
  }
  __device__ __forceinline__ void add_store(const float (&v)[8], void *p, int64_t at) const {
    float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p) + at);
    dst[0] = make_float4(y0.x + v[0], y0.y + v[1], y0.z + v[2], y0.w + v[3]);
    dst[1] = make_float4(y1.x + v[4], y1.y + v[5], y1.z + v[6], y1.w + v[7]);
  }
};

// RT: 8-wide tiles of ranks per warp; RG warps share the ranks (RT 8: up to 64 each).
template <int RT, int RG, bool F32>
__global__ void __launch_bounds__(kStepThreads, 2) adapter_step_kernel(const Args a) {
  constexpr int RMAX = RT * RG * 8, KW = kStepWarps / RG;       // warps that share k
  constexpr int HP = RMAX + 8;                                  // halves between rows of h: other banks
  constexpr int NC = RMAX > 32 ? 2 : 1;                         // blocks of 32 ranks of B held ahead
  __shared__ __align__(16) float part[KW][kStepRows][RMAX];     // each warp's sums
  __shared__ __align__(16) float own[kStepRows][RMAX];          // this CTA's
  // the cluster's, and its hi and lo, where the warps' sums were (read before the cluster's barrier)
  float(*sum)[RMAX] = part[0];
  __half(*hs)[kStepRows][HP] = reinterpret_cast<__half(*)[kStepRows][HP]>(&part[1][0][0]);
  static_assert(2 * HP * 2 <= (KW - 1) * RMAX * 4, "h in place of the warps' sums");
  __shared__ float back[kStepRows];                             // scale 2^-p
  const int S = gridDim.x, split = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  pdl_trigger();
  pdl_wait();
  const int tiles = plan_tiles(a, kPlanStepTiles);
  if ((int)blockIdx.y >= tiles) return;                         // (the whole cluster)
  const int4 tile = a.tiles[blockIdx.y];                        // (not before: another call's plan may be shorter)
  if (tile.x < 0) {
    copy_rows<F32>(a, tile, split, S, kStepThreads);
    return;
  }
  const int rank = adapter_rank(a, tile.x), R8 = (rank + 7) / 8;
  const __half *A = a.a + (int64_t)tile.x * a.R * a.k, *B = a.b + (int64_t)tile.x * a.n * a.R;
  const bool ok0 = g < tile.z, ok1 = g + 8 < tile.z;
  const int64_t t0 = ok0 ? a.perm[tile.y + g] : 0, t1 = ok1 ? a.perm[tile.y + g + 8] : 0;

  {  // h over this CTA's share of k, 32 at a time
    float acc[RT][4];
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
    const int rg = warp % RG, j0 = rg * RT, units = a.k / 32;
    const int u0 = (int)((int64_t)units * split / S), u1 = (int)((int64_t)units * (split + 1) / S);
    const __half *x0 = a.x + t0 * a.x_stride + q * 8, *x1 = a.x + t1 * a.x_stride + q * 8;
    const __half *ar = A + (int64_t)(j0 * 8 + g) * a.k + q * 8;
    // (all of a warp's loads on their way at once where the registers allow it)
#pragma unroll(RT <= 2 ? 4 : 2)
    for (int u = u0 + warp / RG; u < u1; u += KW) {
      const uint4 lo = load16(x0 + u * 32, ok0), hi = load16(x1 + u * 32, ok1);
      uint4 w[RT];
#pragma unroll
      for (int j = 0; j < RT; ++j) w[j] = load16(ar + (int64_t)j * 8 * a.k + u * 32, j0 + j < R8);
#pragma unroll
      for (int j = 0; j < RT; ++j) mma_pair(acc[j], lo, hi, w[j]);
    }
    float *p = &part[warp / RG][0][0] + j0 * 8;
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      *reinterpret_cast<float2 *>(p + g * RMAX + j * 8 + 2 * q) = make_float2(acc[j][0], acc[j][1]);
      *reinterpret_cast<float2 *>(p + (g + 8) * RMAX + j * 8 + 2 * q) = make_float2(acc[j][2], acc[j][3]);
    }
  }
  // the first columns' B and y, on their way while h is put together
  const int units = a.n / 32, R32 = (rank + 31) / 32, ustep = S * kStepWarps;
  const int ncol = 8 * (g >> 1) + (g & 1);                      // column g of the j-th tile: ncol + 2 j
  const auto load_b = [&](int u, int c, uint4 (&w)[4]) {
    const __half *br = B + (int64_t)(u * 32 + ncol) * a.R + c * 32 + q * 8;
    const bool ok = u < units && c * 4 + q < R8;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = load16(br + (int64_t)2 * j * a.R, ok);
  };
  const auto load_y = [&](int u, Out<F32> (&y)[2]) {
    if (u < units && ok0) y[0].load(a.y, t0 * a.y_stride + u * 32 + q * 8);
    if (u < units && ok1) y[1].load(a.y, t1 * a.y_stride + u * 32 + q * 8);
  };
  // (two column blocks in flight per warp, each taken up where it was loaded)
  uint4 w[2][NC][4];
  Out<F32> y[2][2] = {};
  const auto load = [&](int u, int at) {
#pragma unroll
    for (int c = 0; c < NC; ++c) load_b(u, c, w[at][c]);
    load_y(u, y[at]);
  };
  int u = split * kStepWarps + warp;
  load(u, 0);
  load(u + ustep, 1);
  __syncthreads();
  for (int i = threadIdx.x; i < kStepRows * RMAX; i += kStepThreads) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < KW; ++w) v += (&part[w][0][0])[i];
    (&own[0][0])[i] = v;
  }
  cluster_arrive();
  cluster_wait();
  {  // the cluster's sum of the tile's rows, four ranks at a time
    const int R4 = (R8 * 8) / 4, items = tile.z * R4;
    const auto total = [&](int i) {
      const uint32_t at = tc::smem_u32(&own[i / R4][i % R4 * 4]);
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
      for (int s = 0; s < S; ++s) {
        const float4 p = ld_cluster4(map_rank(at, s));
        v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
      }
      return v;
    };
    if (S * items <= 4096) {                                    // everybody adds up everything,
      for (int i = threadIdx.x; i < items; i += kStepThreads)
        *reinterpret_cast<float4 *>(&sum[i / R4][i % R4 * 4]) = total(i);
    } else {                                                    // or its share, and hands it out
      for (int i = items * split / S + threadIdx.x; i < items * (split + 1) / S; i += kStepThreads) {
        const float4 v = total(i);
        const uint32_t at = tc::smem_u32(&sum[i / R4][i % R4 * 4]);
        for (int s = 0; s < S; ++s) st_cluster4(map_rank(at, s), v);
      }
      cluster_arrive();
      cluster_wait();
    }
    __syncthreads();
  }
  {  // as two fp16 parts: 16 threads per row
    const int r = threadIdx.x >> 4, c0 = threadIdx.x & 15;
    constexpr int PER = (RMAX + 15) / 16;
    float v[PER], top = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      v[i] = r < tile.z && c0 + 16 * i < rank ? sum[r][c0 + 16 * i] : 0.0f;
      top = fmaxf(top, fabsf(v[i]));
    }
#pragma unroll
    for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int p = row_exponent(top);
    const float f = scalbnf(1.0f, p);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (c0 + 16 * i < RMAX) split_h(v[i] * f, isinf(top), hs[0][r][c0 + 16 * i], hs[1][r][c0 + 16 * i]);
    if (c0 == 0) back[r] = __ldg(a.scale + tile.x) * scalbnf(1.0f, -p);
  }
  cluster_arrive();                                             // (its sums may go once the others have read them)
  __syncthreads();

  // this CTA's columns, 32 per warp and turn
  const bool few = tile.z <= 8;                                 // hi and lo in one product
  const float f0 = back[g], f1 = back[g + 8];
  const auto block = [&](int at) {
    float d[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) d[j][i] = 0.0f;
    const auto product = [&](int c, const uint4 (&b)[4]) {
      const int k = c * 32 + q * 8;
      const bool ok = c * 4 + q < R8;
      const auto part_of = [&](int part, int row) {
        return ok ? *reinterpret_cast<const uint4 *>(&hs[part][row][k]) : make_uint4(0, 0, 0, 0);
      };
      if (few) {
        const uint4 hi = part_of(0, g), lo = part_of(1, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_pair(d[j], hi, lo, b[j]);
      } else {
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const uint4 upper = part_of(part, g), lower = part_of(part, g + 8);
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_pair(d[j], upper, lower, b[j]);
        }
      }
    };
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (c < R32) product(c, w[at][c]);
    if (RMAX > 64)
      for (int c = NC; c < R32; ++c) {
        load_b(u, c, w[at][0]);
        product(c, w[at][0]);
      }
    if (few)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        d[j][0] += d[j][2];
        d[j][1] += d[j][3];
      }
#pragma unroll
    for (int r = 0; r < 2; ++r)
      if (r ? ok1 : ok0) {
        const float f = r ? f1 : f0;
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[2 * j] = f * d[j][2 * r];
          v[2 * j + 1] = f * d[j][2 * r + 1];
        }
        y[at][r].add_store(v, a.out, (r ? t1 : t0) * a.out_stride + u * 32 + q * 8);
      }
    load(u + 2 * ustep, at);
    u += ustep;
  };
  while (u < units) {
    block(0);
    if (u >= units) break;
    block(1);
  }
  cluster_wait();
}

}  // namespace ad
}  // namespace exl3

using namespace exl3;

namespace {

template <int RT, int RG>
cudaError_t launch_step(const ad::Args &a, bool f32, int S, cudaStream_t s) {
  auto kfn = f32 ? ad::adapter_step_kernel<RT, RG, true> : ad::adapter_step_kernel<RT, RG, false>;
  if (S > 8) {
    // (sixteen CTAs are more than every device has to grant: asked for per function and device)
    static std::atomic<bool> granted[2][kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kMaxDevices || !granted[f32][dev].load(std::memory_order_acquire)) {
      e = cudaFuncSetAttribute(kfn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      if (dev < kMaxDevices) granted[f32][dev].store(true, std::memory_order_release);
    }
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = S;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(S, a.max_tiles);
  cfg.blockDim = dim3(ad::kStepThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kfn, a);
}

}  // namespace

cudaError_t exl3_launch_adapter_step(const ad::Args &a, bool f32, cudaStream_t s) {
  // The largest cluster of which all run at once at two CTAs per SM (30 of eight and
  // 72 of four on 152 SMs; 128 users on 48 adapters: 12.5 us in clusters of eight, 9.0 in
  // fours); sixteen pay for few tiles only (one of rank 64, 17408 columns: 12.8 and 15
  // us, eight of rank 16: 6.8 and 6.1; the border of four lies between the two)
  const int sms = exl3_sm_count();
  const int S = a.max_tiles <= 4 ? 16 : a.max_tiles <= sms * 30 / 152 ? 8 : a.max_tiles <= sms * 72 / 152 ? 4 : 2;
  if (a.R <= 16) return launch_step<2, 1>(a, f32, S, s);
  if (a.R <= 32) return launch_step<4, 1>(a, f32, S, s);
  if (a.R <= 64) return launch_step<8, 1>(a, f32, S, s);
  return launch_step<8, 2>(a, f32, S, s);
}
