// router_logits.cu -- the router's product: logits[t][e] = x[t] . w[e] (+ bias[e]),
// x and w fp16, sums and logits fp32.
//
// Weights kept in fp32 come packed as two fp16 parts and a power of two per
// expert (pack_kernel): w = 2^-p (hi + 2^-11 lo) with the row's largest value
// in [2^14, 2^15), so the parts hold 22 bits of every weight down to 2^-28 of
// the largest and steps of 2^-49 of it below.  Both parts go through the same products; nothing is
// rounded before the fp32 sums.
//
// Few tokens (T <= kGemvRows): a CTA per expert, every thread its share of k,
// all loads of a thread in flight at once.  One read of the weights bounds it;
// at the usual sizes (1 MB) start-up does.
//
// More tokens: tcgen05.  A tile is 128 tokens by all experts that fit 256
// accumulator columns (an expert's two parts are two columns), so x is read
// once; k is split over a cluster of up to eight CTAs, since a layer's tokens
// make too few tiles for the SMs (4096 tokens: 32).  The CTAs of a cluster put
// their sums in shared memory and each adds up its share of the rows from all
// of them (distributed shared memory, always in the order of k): no partial
// sums in HBM, no second launch, the same bits every time.
#include <algorithm>

#include "exl3_common.cuh"
#include "router.cuh"
#include "tc_ptx.cuh"

namespace exl3 {
namespace rt {

constexpr int BM = 128, BK = 64;
constexpr int kGemvThreads = 128;
constexpr int kLogitThreads = 192;
constexpr float kLoScale = 0x1p-11f;

// ------------------------------------------------------------------ packing

// A CTA per expert: the power of two from the row's largest value, then both
// parts.  w 2^p - hi is exact in fp32, so lo takes what hi left.
__global__ void __launch_bounds__(256) pack_kernel(const float *__restrict__ w, int E, int k, __half *__restrict__ out,
                                                   float *__restrict__ scale) {
  __shared__ float top[8];
  const int e = blockIdx.x;
  const float *row = w + (int64_t)e * k;
  float m = 0.0f;
  for (int j = threadIdx.x; j < k; j += blockDim.x) m = fmaxf(m, fabsf(row[j]));
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = m;
  __syncthreads();
  for (int i = 0; i < 8; ++i) m = fmaxf(m, top[i]);
  int p = 0;
  if (m > 0.0f && isfinite(m)) p = min(14 - ilogbf(m), 100);   // (2^-p stays a normal number)
  const float f = scalbnf(1.0f, p);
  for (int j = threadIdx.x; j < k; j += blockDim.x) {
    const float v = row[j] * f;
    const __half hi = isfinite(v) ? __float2half_rn(v) : __float2half_rn(__int_as_float(0x7fffffff));
    out[(int64_t)e * k + j] = hi;
    out[(int64_t)(E + e) * k + j] = __float2half_rn((v - __half2float(hi)) * 0x1p11f);
  }
  if (threadIdx.x == 0) scale[e] = scalbnf(1.0f, -p);
}

// --------------------------------------------------------------- few tokens

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
  const __half2 *h = reinterpret_cast<const __half2 *>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __half22float2(h[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

// R tokens from blockIdx.y * R on; PACKED: two parts and a power of two.
template <int R, bool PACKED>
__global__ void __launch_bounds__(kGemvThreads) logits_gemv_kernel(const LogitArgs a) {
  __shared__ float part[kGemvThreads / 32][R];
  pdl_trigger();
  pdl_wait();
  const int e = blockIdx.x, t0 = blockIdx.y * R, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const __half *w = a.w + (int64_t)e * a.k, *w2 = w + (int64_t)a.E * a.k;
  float acc[R];
#pragma unroll
  for (int r = 0; r < R; ++r) acc[r] = 0.0f;
#pragma unroll 2
  for (int j = threadIdx.x * 8; j < a.k; j += kGemvThreads * 8) {
    float wf[8];
    unpack8(__ldg(reinterpret_cast<const uint4 *>(w + j)), wf);
    if (PACKED) {
      float lo[8];
      unpack8(__ldg(reinterpret_cast<const uint4 *>(w2 + j)), lo);
#pragma unroll
      for (int i = 0; i < 8; ++i) wf[i] = fmaf(lo[i], kLoScale, wf[i]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float xf[8];
      // (a row past the last one repeats it and is not stored)
      unpack8(__ldg(reinterpret_cast<const uint4 *>(a.x + min(t0 + r, a.T - 1) * a.x_stride + j)), xf);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[r] = fmaf(xf[i], wf[i], acc[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int o = 16; o; o >>= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], o);
    if (lane == 0) part[warp][r] = acc[r];
  }
  __syncthreads();
  if (threadIdx.x < R && t0 + (int)threadIdx.x < a.T) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kGemvThreads / 32; ++i) v += part[i][threadIdx.x];
    if (PACKED) v *= __ldg(a.w_scale + e);
    if (a.bias) v += __ldg(a.bias + e);
    a.logits[(int64_t)(t0 + threadIdx.x) * a.E + e] = v;
  }
}

// -------------------------------------------------------------- tensor cores

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;\n" ::: "memory");
}

// Four floats at a shared-memory address of CTA `rank` of the cluster.
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr, int rank) {
  uint32_t r;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(r)
               : "memory");
  return v;
}

// Grid (splits, token tiles, expert tiles), clusters along x.  Warp 0 brings
// the operands, warp 1 issues the products, warps 2 to 5 empty the accumulator.
template <bool PACKED>
__global__ void __launch_bounds__(kLogitThreads, 1) logits_tc_kernel(const __grid_constant__ CUtensorMap mx,
                                                                     const __grid_constant__ CUtensorMap mw,
                                                                     const LogitArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = tc::smem_u32(smem_raw);
  uint8_t *smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const int cols = PACKED ? 2 * a.bn : a.bn;                  // accumulator columns
  const int stage_bytes = BM * BK * 2 + cols * BK * 2;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + a.data_bytes);
  uint64_t *empty = full + a.stages, *done = empty + a.stages;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  volatile int *failed = reinterpret_cast<volatile int *>(tmem_slot + 1), *used = failed + 1;   // (uses of the ring)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = gridDim.x, split = blockIdx.x, m0 = blockIdx.y * BM, n0 = blockIdx.z * a.bn;
  const int KB = (a.k + BK - 1) / BK;
  const int kb0 = (int)((int64_t)KB * split / S), kb1 = (int)((int64_t)KB * (split + 1) / S);

  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    tc::mbar_init(done, 1);
    *failed = 0;
    *used = kb1 - kb0;
    tc::fence_mbar_init();
    tc::prefetch_tmap(&mx);
    tc::prefetch_tmap(&mw);
  }
  pdl_wait();
  const auto bring = [&](int st, int kb) {                  // (one thread)
    uint8_t *sa = smem + st * stage_bytes, *sb = sa + BM * BK * 2;
    tc::mbar_arrive_expect_tx(&full[st], stage_bytes);
    tc::tma_load_2d(sa, &mx, &full[st], kb * BK, m0);
    tc::tma_load_2d(sb, &mw, &full[st], kb * BK, n0);
    if (PACKED) tc::tma_load_2d(sb + a.bn * BK * 2, &mw, &full[st], kb * BK, a.E + n0);
  };
  const int ahead = min(kb1, kb0 + a.stages);
  if (threadIdx.x == 0)                                     // the ring's first round
    for (int kb = kb0; kb < ahead; ++kb) bring(kb - kb0, kb);
  // TMEM only now: nobody ahead on the stream waits for it, and what comes next
  // may start once all of this kernel has its own
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, a.tmem_cols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();

  if (warp == 0) {
    if (lane == 0) {
      int st = 0;
      uint32_t phase = 0;
      for (int kb = ahead; kb < kb1; ++kb) {
        if (!tc::mbar_wait(&empty[st], phase)) {
          *failed = 1;
          *used = kb - kb0;
          break;
        }
        bring(st, kb);
        if (++st == a.stages) { st = 0; phase ^= 1; }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t idesc = tc::idesc_f16(BM, cols);
    int st = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!__all_sync(0xffffffffu, tc::mbar_wait(&full[st], phase))) {
        *failed = 1;
        break;
      }
      tc::tc_fence_after();
      const uint64_t ad = tc::sdesc_k_sw128(smem + st * stage_bytes);
      const uint64_t bd = tc::sdesc_k_sw128(smem + st * stage_bytes + BM * BK * 2);
      if (tc::elect_one()) {
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          tc::mma_f16(tmem, ad + 2 * kk, bd + 2 * kk, idesc, (kb != kb0 || kk != 0) ? 1u : 0u);
        tc::mma_commit(&empty[st]);
      }
      __syncwarp();
      if (++st == a.stages) { st = 0; phase ^= 1; }
    }
    if (tc::elect_one()) tc::mma_commit(done);
    __syncwarp();
  } else {
    // the operands' place becomes the sums' once every product is done (no
    // load is in flight then: each was waited for by a product)
    if (!__all_sync(0xffffffffu, tc::mbar_wait(done, 0))) *failed = 1;
    tc::tc_fence_after();
    if (!*failed) {
      const int row = 32 * (warp & 3) + lane;
      const uint32_t from = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
      float *dst = reinterpret_cast<float *>(smem) + row * a.pitch;
      bool far = false;
      for (int c = 0; c < a.bn; c += 32) {
        float v[32];
        tc::tmem_ld32(from + c, v);
        if (PACKED) {                                       // (half as much to exchange)
          float lo[32];
          tc::tmem_ld32(from + a.bn + c, lo);
          tc::tmem_ld_wait();
          far |= !isfinite(v[0]);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = fmaf(lo[i], kLoScale, v[i]);
        }
        tc::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          if (c + i < a.bn) *reinterpret_cast<float4 *>(dst + c + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      }
      // An infinity in x makes a row's high parts infinite or NaN for all experts; the low
      // parts, whose signs are their own, are left out of it.  (Here, since among the
      // columns above it cost 0.2 us of 7.2.)
      if (PACKED && __any_sync(0xffffffffu, far))
        for (int c = 0; c < a.bn; c += 32) {
          float v[32];
          tc::tmem_ld32(from + c, v);
          tc::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c + i < a.bn && isinf(v[i])) dst[c + i] = v[i];
        }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (*failed && threadIdx.x == 0) {
    set_device_error(a.err, kErrBounds);
    tc::drain(full, a.stages, *used);                       // leave no copy in flight behind
  }
  if (S > 1) cluster_sync();

  // this CTA's rows of the tile, summed over the cluster in the order of k
  {
    const int rows = BM / S, quads = a.bn / 4;
    const uint32_t base = tc::smem_u32(smem);
    for (int i = threadIdx.x; i < rows * quads; i += kLogitThreads) {
      const int r = split * rows + i / quads, c = i % quads * 4, t = m0 + r, e = n0 + c;
      if (t >= a.T || e >= a.E) continue;
      const uint32_t at = base + (uint32_t)(r * a.pitch + c) * 4;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f), p[8];   // (all on their way at once)
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if (s < S) p[s] = ld_cluster4(at, s);
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if (s < S) {
          v.x += p[s].x; v.y += p[s].y; v.z += p[s].z; v.w += p[s].w;
        }
      float o[4] = {v.x, v.y, v.z, v.w};
      float *dst = a.logits + (int64_t)t * a.E + e;
      const int n = min(4, a.E - e);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < n) {
          if (PACKED) o[j] *= __ldg(a.w_scale + e + j);
          if (a.bias) o[j] += __ldg(a.bias + e + j);
        }
      if ((a.E & 3) == 0) {
        *reinterpret_cast<float4 *>(dst) = make_float4(o[0], o[1], o[2], o[3]);
      } else {
        for (int j = 0; j < n; ++j) dst[j] = o[j];
      }
    }
  }
  if (S > 1) cluster_sync();        // nobody leaves while its sums are read
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, a.tmem_cols);
  }
}

}  // namespace rt
}  // namespace exl3

using namespace exl3;

namespace {

// fp16 [rows][cols], rows `stride` elements apart; boxes of box_rows x 64, 128-byte swizzle.
int map_rows(CUtensorMap *m, const void *base, int64_t rows, int cols, int64_t stride, int box_rows) {
  auto fn = exl3_tmap_encode_fn();
  if (!fn) return exl3_fail(EXL3_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, estr[2] = {1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return exl3_fail(EXL3_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return EXL3_OK;
}

constexpr int kGemvRows = 8;

template <bool PACKED>
int launch_logits(rt::LogitArgs a, cudaStream_t s) {
  if (a.T <= kGemvRows) {
    const int R = a.T <= 1 ? 1 : a.T <= 2 ? 2 : 4;
    const dim3 grid(a.E, (a.T + R - 1) / R), block(rt::kGemvThreads);
    return exl3_cuda_check(R == 1   ? launch_pdl(rt::logits_gemv_kernel<1, PACKED>, grid, block, 0, s, a)
                           : R == 2 ? launch_pdl(rt::logits_gemv_kernel<2, PACKED>, grid, block, 0, s, a)
                                    : launch_pdl(rt::logits_gemv_kernel<4, PACKED>, grid, block, 0, s, a),
                           "router logits launch");
  }
  const int sms = exl3_sm_count(), MT = (a.T + rt::BM - 1) / rt::BM, KB = (a.k + rt::BK - 1) / rt::BK;
  const int most = PACKED ? 128 : 256;                      // experts of one tile
  int NT = (a.E + most - 1) / most;
  // Clusters that run at once at one CTA per SM, by the parts that the SMs come in:
  // 76 of two CTAs, 36 of four, 15 of eight (of 152 SMs; one more cluster is a
  // second round: 48 tokens took 9.2 us as 16 clusters of eight and 5.1 as 8).
  // Smaller tiles of experts while clusters of four are to be had (32 experts at
  // least), then the largest split that fits.
  while ((int64_t)MT * 2 * NT <= sms * 36 / 152 && a.E / (2 * NT) >= 32) NT *= 2;
  const int64_t clusters = (int64_t)MT * NT;
  int S = clusters <= sms * 15 / 152 ? 8 : clusters <= sms * 36 / 152 ? 4 : clusters <= sms / 2 ? 2 : 1;
  while (S > KB) S /= 2;
  a.bn = ((a.E + NT - 1) / NT + 15) / 16 * 16;
  NT = (a.E + a.bn - 1) / a.bn;
  const int cols = PACKED ? 2 * a.bn : a.bn, stage = (rt::BM + cols) * rt::BK * 2;
  a.stages = std::min((KB + S - 1) / S, std::min(8, 200 * 1024 / stage));
  a.pitch = a.bn + 4;                                       // (a float4 apart: rows start in different banks)
  a.data_bytes = (int)((std::max<size_t>((size_t)a.stages * stage, (size_t)rt::BM * a.pitch * 4) + 15) / 16 * 16);
  a.tmem_cols = 32;                                         // (read 32 at a time: lo from bn on)
  while ((int)a.tmem_cols < cols + (PACKED && a.bn % 32 ? 16 : 0)) a.tmem_cols *= 2;
  // One CTA per SM whatever the ring needs: a CTA that waited for TMEM held by
  // another cluster's, which waits for its own members, could wait for ever.
  const size_t smem = std::max<size_t>(1024 + a.data_bytes + (2 * a.stages + 1) * 8 + 16, 120 * 1024);
  CUtensorMap mx, mw;
  int rc = map_rows(&mx, a.x, a.T, a.k, a.x_stride, rt::BM);
  if (rc) return rc;
  rc = map_rows(&mw, a.w, (int64_t)a.E * (PACKED ? 2 : 1), a.k, a.k, a.bn);
  if (rc) return rc;
  static std::atomic<size_t> given[kMaxDevices];
  auto kfn = rt::logits_tc_kernel<PACKED>;
  rc = exl3_cuda_check(exl3_ensure_smem(reinterpret_cast<const void *>(kfn), smem, given), "router logits attribute");
  if (rc) return rc;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = S;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(S, MT, NT);
  cfg.blockDim = dim3(rt::kLogitThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return exl3_cuda_check(cudaLaunchKernelEx(&cfg, kfn, mx, mw, a), "router logits launch");
}

}  // namespace

int exl3_launch_router_logits(const rt::LogitArgs &a, bool packed, cudaStream_t s) {
  return packed ? launch_logits<true>(a, s) : launch_logits<false>(a, s);
}

cudaError_t exl3_launch_router_pack(const float *w, int E, int k, __half *out, float *scale, cudaStream_t s) {
  rt::pack_kernel<<<E, 256, 0, s>>>(w, E, k, out, scale);
  return cudaGetLastError();
}
