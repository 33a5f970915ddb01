// adapter_tc.cu -- low-rank adapters on many rows, on the tensor cores:
//
//   out[t] = y[t] + scale (x[t] A^T) B^T
//
// A tile is up to 128 rows of one adapter, taken by a cluster of S CTAs:
//   1. each CTA forms h = x A^T over its share of k (tcgen05, 128 x R in TMEM);
//      x rows come by TMA gathers of four rows, so a tile's rows may lie anywhere;
//   2. each CTA adds up the cluster's sums for its share of the rows
//      (distributed shared memory, in the order of k), splits them into two fp16
//      parts and writes those into every CTA's shared memory as the next operand;
//   3. each CTA forms h B^T for its share of the n columns, 128 at a time, adds y
//      and writes out.
// One launch; x, y, A and B are read once, out is written once, h never leaves
// the SMs.  Up to 4 R / 3 operations per byte: HBM bounds it at every rank, most
// of it y and out in step 3, so that step keeps two chunks of y in flight per
// thread and reads and writes whole 32-byte sectors.  Up to rank 64 two CTAs
// share an SM, one's first steps under the other's last.
//
// h: each row is brought to [2^14, 2^15) by a power of two and then hi + lo, 22
// bits; the second product runs over both parts (twice the operations of a small
// K), so an fp32 out is as good as its sums.
#include "adapter.cuh"
#include "tc_ptx.cuh"

namespace exl3 {
namespace ad {

constexpr int kTcThreads = 320;                 // producer, issuer, eight warps for sums and output
constexpr int kEpiWarps = 8;
constexpr int kPanel = kTcRows * 128;           // bytes of 128 rows of 64 fp16
constexpr uint32_t kTmemCols = 256;             // two output accumulators; h first

struct TcArgs {
  Args a;
  int r16;                // ranks of the first product, a multiple of 16
  int panels;             // panels of 64 ranks
  int stages, b_stages;   // rings of step 1 and step 3
  int ring_bytes;         // the larger ring, or the sums
  int wide;               // y and out may be accessed 32 bytes at a time
};

// Four rows of a tensor map (its box is one row), 64 columns each.
__device__ __forceinline__ void tma_gather4(void *dst, const CUtensorMap *m, uint64_t *bar, int x, const int4 &rows) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
      "%5, %6, %7}], [%2];\n" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(tc::smem_u32(bar)), "r"(x), "r"(rows.x), "r"(rows.y), "r"(rows.z),
      "r"(rows.w)
      : "memory");
}

__device__ __forceinline__ void st_cluster16(uint32_t addr, const uint4 &v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async;\n" ::: "memory"); }

// 16 consecutive 32-bit TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// 64 bytes of y or out: two 32-byte accesses where the rows allow it.
struct Chunk {
  uint32_t w[16];
};
__device__ __forceinline__ void load_chunk(Chunk &c, const char *p, bool wide) {
  if (wide) {
#pragma unroll
    for (int i = 0; i < 16; i += 8)
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
                   : "=r"(c.w[i]), "=r"(c.w[i + 1]), "=r"(c.w[i + 2]), "=r"(c.w[i + 3]), "=r"(c.w[i + 4]),
                     "=r"(c.w[i + 5]), "=r"(c.w[i + 6]), "=r"(c.w[i + 7])
                   : "l"(p + i * 4)
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4 *>(p + i * 4);
      c.w[i] = v.x;
      c.w[i + 1] = v.y;
      c.w[i + 2] = v.z;
      c.w[i + 3] = v.w;
    }
  }
}
__device__ __forceinline__ void store_chunk(char *p, const Chunk &c, bool wide) {
  if (wide) {
#pragma unroll
    for (int i = 0; i < 16; i += 8)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p + i * 4), "r"(c.w[i]),
                   "r"(c.w[i + 1]), "r"(c.w[i + 2]), "r"(c.w[i + 3]), "r"(c.w[i + 4]), "r"(c.w[i + 5]), "r"(c.w[i + 6]),
                   "r"(c.w[i + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *reinterpret_cast<uint4 *>(p + i * 4) = make_uint4(c.w[i], c.w[i + 1], c.w[i + 2], c.w[i + 3]);
  }
}

// CTAS: of an SM.
template <bool F32, int CTAS>
__global__ void __launch_bounds__(kTcThreads, CTAS) adapter_tc_kernel(const __grid_constant__ CUtensorMap mx,
                                                                      const __grid_constant__ CUtensorMap ma,
                                                                      const __grid_constant__ CUtensorMap mb,
                                                                      const TcArgs g) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = tc::smem_u32(smem_raw);
  uint8_t *ring = smem_raw + (((raw + 1023u) & ~1023u) - raw);      // step 1's ring, then its sums, then step 3's ring
  uint8_t *hs = ring + g.ring_bytes;                                // [2][panels] panels: hi, lo
  float *back = reinterpret_cast<float *>(hs + 2 * g.panels * kPanel);   // [128]: scale 2^-p
  uint64_t *full = reinterpret_cast<uint64_t *>(back + kTcRows);
  uint64_t *empty = full + 8, *done = empty + 8, *b_full = done + 1, *b_empty = b_full + 8, *t_full = b_empty + 8,
           *t_empty = t_full + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(t_empty + 2);
  volatile int *failed = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const Args &a = g.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, S = gridDim.x, split = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 8; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
      tc::mbar_init(&b_full[s], 1);
      tc::mbar_init(&b_empty[s], 1);
    }
    tc::mbar_init(done, 1);
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(&t_full[s], 1);
      tc::mbar_init(&t_empty[s], kEpiWarps);
    }
    *failed = 0;
    tc::fence_mbar_init();
    tc::prefetch_tmap(&mx);
    tc::prefetch_tmap(&ma);
    tc::prefetch_tmap(&mb);
  }
  pdl_wait();
  const int tiles = plan_tiles(a, kPlanTcTiles);
  const int4 tile = a.tiles[blockIdx.y];
  const int rank = (int)blockIdx.y < tiles && tile.x >= 0 ? adapter_rank(a, tile.x) : 0;
  if (rank == 0) {                                                  // (the whole cluster)
    pdl_trigger();
    if ((int)blockIdx.y < tiles) copy_rows<F32>(a, tile, split, S, kTcThreads);
    return;
  }
  // TMEM only now: nobody ahead on the stream waits for it, and what comes next
  // may start once all of this kernel has its own
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();

  const int KB = a.k / 64, kb0 = KB * split / S, kb1 = KB * (split + 1) / S;
  const int NB = a.n / 128, nb0 = NB * split / S, nb1 = NB * (split + 1) / S;
  const int stage_bytes = kPanel + g.r16 * 128;

  // ---- step 1
  if (warp == 0) {
    // lane i gathers rows 4 i .. 4 i + 3 (past the last row: that one again)
    const int quads = (tile.z + 3) / 4;
    int4 rows;
    {
      const int *p = a.perm + tile.y;
      const int last = tile.z - 1, i = min(4 * lane, last);
      rows = make_int4(p[i], p[min(i + 1, last)], p[min(i + 2, last)], p[min(i + 3, last)]);
    }
    int st = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      bool ok = true;
      if (lane == 0) {
        ok = tc::mbar_wait(&empty[st], phase ^ 1);
        if (ok) tc::mbar_arrive_expect_tx(&full[st], quads * 512 + g.r16 * 128);
        else *failed = 1;
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      uint8_t *sx = ring + st * stage_bytes;
      if (lane < quads) tma_gather4(sx + lane * 512, &mx, &full[st], kb * 64, rows);
      if (lane == 0) tc::tma_load_3d(sx + kPanel, &ma, &full[st], kb * 64, 0, tile.x);
      if (++st == g.stages) { st = 0; phase ^= 1; }
    }
  } else if (warp == 1) {
    const uint32_t idesc = tc::idesc_f16(kTcRows, g.r16);
    int st = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!__all_sync(0xffffffffu, tc::mbar_wait(&full[st], phase))) {
        *failed = 1;
        break;
      }
      tc::tc_fence_after();
      const uint64_t ad = tc::sdesc_k_sw128(ring + st * stage_bytes);
      const uint64_t bd = tc::sdesc_k_sw128(ring + st * stage_bytes + kPanel);
      if (tc::elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) tc::mma_f16(tmem, ad + 2 * kk, bd + 2 * kk, idesc, (kb != kb0 || kk != 0) ? 1u : 0u);
        tc::mma_commit(&empty[st]);
      }
      __syncwarp();
      if (++st == g.stages) { st = 0; phase ^= 1; }
    }
    if (tc::elect_one()) tc::mma_commit(done);
    __syncwarp();
  }
  const int pitch = g.r16 + 4;                                      // floats between rows of sums
  const int quarter = warp & 3, half = (warp - 2) >> 2;             // of TMEM's lanes; of a tile's columns
  const int own = 32 * quarter + lane;                              // this thread's row of the tile
  if (warp >= 2) {
    if (!__all_sync(0xffffffffu, tc::mbar_wait(done, 0))) *failed = 1;
    tc::tc_fence_after();
    float *dst = reinterpret_cast<float *>(ring) + own * pitch;
    for (int c = 16 * half; c < g.r16; c += 32) {
      float v[16];
      if (kb0 < kb1) {
        tmem_ld16(tmem + ((uint32_t)(32 * quarter) << 16) + c, v);
        tc::tmem_ld_wait();
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0.0f;                   // (no share of k)
      }
#pragma unroll
      for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4 *>(dst + c + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
    tc::tc_fence_before();
  }
  cluster_arrive();
  cluster_wait();

  // ---- step 2: 16 threads to a row, eight ranks each
  if (warp >= 2) {
    const int per = kTcRows / S, t = threadIdx.x - 64, c = 8 * (t & 15);
    for (int r0 = t >> 4; r0 < per; r0 += 16) {                     // (per is a multiple of 16: whole half-warps)
      const int r = split * per + r0;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
      if (c < g.r16) {
        const uint32_t at = tc::smem_u32(ring) + (uint32_t)(r * pitch + c) * 4;
        for (int s = 0; s < S; ++s) {
          const uint32_t from = map_rank(at, s);
          const float4 p = ld_cluster4(from), q = ld_cluster4(from + 16);
          v[0] += p.x; v[1] += p.y; v[2] += p.z; v[3] += p.w;
          v[4] += q.x; v[5] += q.y; v[6] += q.z; v[7] += q.w;
        }
      }
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (c + i >= rank || r >= tile.z) v[i] = 0.0f;              // (rows past the last one: whatever was there)
        top = fmaxf(top, fabsf(v[i]));
      }
#pragma unroll
      for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int p = row_exponent(top);
      const float f = scalbnf(1.0f, p);
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float z0 = v[2 * i] * f, z1 = v[2 * i + 1] * f;
        const __half2 h = __floats2half2_rn(z0, z1);
        const __half2 l = __floats2half2_rn(z0 - __low2float(h), z1 - __high2float(h));
        hi[i] = *reinterpret_cast<const uint32_t *>(&h);
        lo[i] = *reinterpret_cast<const uint32_t *>(&l);
      }
      // 128-byte swizzle: the 16-byte piece of a row goes by the row's number too
      const uint32_t at = tc::smem_u32(hs) + (c >> 6) * kPanel + r * 128 + ((((c & 63) >> 3) ^ (r & 7)) << 4);
      const float b = __ldg(a.scale + tile.x) * scalbnf(1.0f, -p);
      for (int s = 0; s < S; ++s) {
        if (c < g.r16) {
          st_cluster16(map_rank(at, s), make_uint4(hi[0], hi[1], hi[2], hi[3]));
          st_cluster16(map_rank(at + g.panels * kPanel, s), make_uint4(lo[0], lo[1], lo[2], lo[3]));
        }
        if (c == 0) st_cluster(map_rank(tc::smem_u32(back + r), s), b);
      }
    }
  }
  fence_async();                                                    // the products and copies read and write past the caches of plain accesses
  cluster_arrive();
  cluster_wait();
  fence_async();

  // ---- step 3
  const int kr = (rank + 15) / 16;
  if (warp == 0) {
    if (lane == 0) {
      int st = 0;
      uint32_t phase = 0;
      const int b_bytes = g.panels * kPanel;
      for (int nb = nb0; nb < nb1; ++nb) {
        if (!tc::mbar_wait(&b_empty[st], phase ^ 1)) {
          *failed = 1;
          break;
        }
        tc::mbar_arrive_expect_tx(&b_full[st], b_bytes);
        for (int p = 0; p < g.panels; ++p)
          tc::tma_load_3d(ring + st * b_bytes + p * kPanel, &mb, &b_full[st], p * 64, nb * 128, tile.x);
        if (++st == g.b_stages) { st = 0; phase ^= 1; }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    tc::tc_fence_after();
    const uint32_t idesc = tc::idesc_f16(kTcRows, 128);
    const uint64_t hd = tc::sdesc_k_sw128(hs);
    int st = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    for (int nb = nb0; nb < nb1; ++nb) {
      const bool ok = tc::mbar_wait(&t_empty[acc], acc_phase ^ 1) && tc::mbar_wait(&b_full[st], phase);
      if (!__all_sync(0xffffffffu, ok)) {
        *failed = 1;
        break;
      }
      tc::tc_fence_after();
      const uint64_t bd = tc::sdesc_k_sw128(ring + st * g.panels * kPanel);
      if (tc::elect_one()) {
        for (int part = 0; part < 2; ++part)
          for (int kk = 0; kk < kr; ++kk) {
            const uint32_t in = (kk >> 2) * (kPanel >> 4) + (kk & 3) * 2;
            tc::mma_f16(tmem + acc * 128, hd + part * (g.panels * kPanel >> 4) + in, bd + in, idesc, part || kk ? 1u : 0u);
          }
        tc::mma_commit(&b_empty[st]);
        tc::mma_commit(&t_full[acc]);
      }
      __syncwarp();
      if (++st == g.b_stages) { st = 0; phase ^= 1; }
      if (++acc == 2) { acc = 0; acc_phase ^= 1; }
    }
  } else {
    constexpr int SIZE = F32 ? 4 : 2, COLS = 64 / SIZE, CHUNKS = 64 / COLS;   // columns of a chunk, chunks of a half tile
    const bool live = own < tile.z;
    const int64_t row = live ? a.perm[tile.y + own] : 0;
    const char *src = static_cast<const char *>(a.y) + (row * a.y_stride + half * 64) * SIZE;
    char *dst = static_cast<char *>(a.out) + (row * a.out_stride + half * 64) * SIZE;
    const float f = back[own];
    const bool wide = g.wide;
    Chunk next = {};
    if (live && nb0 < nb1) load_chunk(next, src + (int64_t)nb0 * 128 * SIZE, wide);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int nb = nb0; nb < nb1; ++nb) {
      bool stop = false;
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) {
        Chunk y = next;
        // the next chunk's y is on its way while this one's product is waited for
        const bool more = c + 1 < CHUNKS || nb + 1 < nb1;
        if (live && more)
          load_chunk(next, src + ((int64_t)(c + 1 < CHUNKS ? nb : nb + 1) * 128 + (c + 1) % CHUNKS * COLS) * SIZE, wide);
        if (c == 0) {
          stop = !__all_sync(0xffffffffu, tc::mbar_wait(&t_full[acc], acc_phase));
          if (stop) break;
          tc::tc_fence_after();
        }
        const uint32_t at = tmem + ((uint32_t)(32 * quarter) << 16) + acc * 128 + half * 64 + c * COLS;
        float v[COLS];
        if constexpr (F32) tmem_ld16(at, v);
        else tc::tmem_ld32(at, v);
        tc::tmem_ld_wait();
        if (c + 1 == CHUNKS) {
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&t_empty[acc]);
        }
        if (live) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (F32) {
              y.w[i] = __float_as_uint(fmaf(f, v[i], __uint_as_float(y.w[i])));
            } else {
              const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&y.w[i]));
              const __half2 o = __floats2half2_rn(fmaf(f, v[2 * i % COLS], t.x), fmaf(f, v[(2 * i + 1) % COLS], t.y));
              y.w[i] = *reinterpret_cast<const uint32_t *>(&o);
            }
          }
          store_chunk(dst + ((int64_t)nb * 128 + c * COLS) * SIZE, y, wide);
        }
      }
      if (stop) {
        *failed = 1;
        break;
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1; }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (*failed && threadIdx.x == 0) set_device_error(a.ctrl + kPlanErr, kErrBounds);
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace ad
}  // namespace exl3

using namespace exl3;

namespace {

int map_f16(CUtensorMap *m, const void *base, int dims, const cuuint64_t *size, const cuuint64_t *stride,
            const cuuint32_t *box) {
  auto fn = exl3_tmap_encode_fn();
  if (!fn) return exl3_fail(EXL3_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, dims, const_cast<void *>(base), size, stride, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return exl3_fail(EXL3_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return EXL3_OK;
}

template <bool F32, int CTAS>
int launch_tc(const CUtensorMap &mx, const CUtensorMap &ma, const CUtensorMap &mb, const ad::TcArgs &g, int S,
              size_t smem, cudaStream_t s) {
  auto kfn = ad::adapter_tc_kernel<F32, CTAS>;
  static std::atomic<size_t> given[kMaxDevices];
  int rc = exl3_cuda_check(exl3_ensure_smem(reinterpret_cast<const void *>(kfn), smem, given), "adapter attribute");
  if (rc) return rc;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = S;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(S, g.a.max_tiles);
  cfg.blockDim = dim3(ad::kTcThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return exl3_cuda_check(cudaLaunchKernelEx(&cfg, kfn, mx, ma, mb, g), "adapter launch");
}

}  // namespace

int exl3_launch_adapter_tc(const ad::Args &a, bool f32, cudaStream_t s) {
  ad::TcArgs g = {};
  g.a = a;
  g.r16 = (a.R + 15) / 16 * 16;
  g.panels = (a.R + 63) / 64;
  const int stage = ad::kPanel + g.r16 * 128;
  // Up to rank 64: rings of 72 KB, operands of 32 KB, two CTAs on an SM (and never
  // three, which TMEM would not hold).  Above: 128 KB and 64 KB, one.
  const int room = g.panels == 1 ? 72 * 1024 : 128 * 1024;
  g.stages = std::min(8, room / stage);
  g.b_stages = std::min(8, room / (g.panels * ad::kPanel));
  g.ring_bytes = room;
  const size_t smem = 1024 + g.ring_bytes + 2 * g.panels * ad::kPanel + ad::kTcRows * 4 + (4 * 8 + 5) * 8 + 16;
  const int size = f32 ? 4 : 2;
  const auto on32 = [&](const void *p, int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % 32 == 0 && stride * size % 32 == 0;
  };
  g.wide = on32(a.y, a.y_stride) && on32(a.out, a.out_stride);
  CUtensorMap mx, ma, mb;
  {
    const cuuint64_t dims[2] = {(cuuint64_t)a.k, (cuuint64_t)a.T}, stride[1] = {(cuuint64_t)a.x_stride * 2};
    const cuuint32_t box[2] = {64, 1};
    int rc = map_f16(&mx, a.x, 2, dims, stride, box);
    if (rc) return rc;
  }
  {
    const cuuint64_t dims[3] = {(cuuint64_t)a.k, (cuuint64_t)a.R, (cuuint64_t)a.N};
    const cuuint64_t stride[2] = {(cuuint64_t)a.k * 2, (cuuint64_t)a.k * a.R * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)g.r16, 1};
    int rc = map_f16(&ma, a.a, 3, dims, stride, box);
    if (rc) return rc;
  }
  {
    const cuuint64_t dims[3] = {(cuuint64_t)a.R, (cuuint64_t)a.n, (cuuint64_t)a.N};
    const cuuint64_t stride[2] = {(cuuint64_t)a.R * 2, (cuuint64_t)a.R * a.n * 2};
    const cuuint32_t box[3] = {64, 128, 1};
    int rc = map_f16(&mb, a.b, 3, dims, stride, box);
    if (rc) return rc;
  }
  // a cluster per tile: eight CTAs while that fills two rounds of SMs at most
  const int slots = exl3_sm_count() * (g.panels == 1 ? 2 : 1);
  int S = 8;
  while (S > 2 && (int64_t)a.max_tiles * S > 2 * slots) S /= 2;
  if (g.panels == 1) return f32 ? launch_tc<true, 2>(mx, ma, mb, g, S, smem, s) : launch_tc<false, 2>(mx, ma, mb, g, S, smem, s);
  return f32 ? launch_tc<true, 1>(mx, ma, mb, g, S, smem, s) : launch_tc<false, 1>(mx, ma, mb, g, S, smem, s);
}
