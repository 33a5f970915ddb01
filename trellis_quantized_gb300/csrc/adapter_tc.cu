// adapter_tc.cu -- low-rank adapters on many rows, on the tensor cores:
//
//   out[t] = y[t] + scale (x[t] A^T) B^T
//
// in tiles of up to 128 rows of one adapter, as two kernels:
//
// adapter_in_kernel   h = x A^T.  A cluster of S CTAs takes a tile; each forms h
//   over its share of k (tcgen05, 128 x R in TMEM; x comes by TMA gathers of four
//   rows, so a tile's rows may lie anywhere), then adds up the cluster's sums for
//   its share of the rows (distributed shared memory, in the order of k).
// adapter_out_kernel  out = y + h B^T.  The tiles' columns, 128 at a time, form one
//   line (weighted by a tile's rows) that persistent CTAs share in equal runs.
//
// x, y, A and B are read once and out is written once; h goes through L2.  Up to
// 4 R / 3 operations per byte: HBM bounds it at every rank, mostly by y and out.
// One launch (the cluster keeps h and splits the columns too) was measured at
// 228 us where this takes a third: 46 tiles are two rounds of clusters, one of
// them almost empty.
//
// h: each row is brought to [2^14, 2^15) by a power of two and then hi + lo, 22
// bits; the second product runs over both parts (twice the operations of a small
// K), so an fp32 out is as good as its sums.
//
// The accumulator is read in the layout of 16 x 256 bits: a lane gets two columns
// of every eight for rows g and g + 8.  The copy of B permutes its rows (as a
// tensor map of five dimensions) so that these are 16 neighbouring columns of out:
// four lanes access one 128-byte line of y or out, and no transposition is needed.
// (With a row to a lane, 32 lines an access, y and out ran at 3 TB/s.)
#include "adapter.cuh"
#include "tc_ptx.cuh"

namespace exl3 {
namespace ad {

constexpr int kPanel = kTcRows * 128;           // bytes of 128 rows of 64 fp16
constexpr int kInThreads = 192;                 // producer, issuer, four warps for the sums
constexpr int kOutThreads = 320;                // producer, issuer, eight warps for the output
constexpr int kEpiWarps = 8;
constexpr uint32_t kOutCols = 256;              // TMEM: two accumulators

struct InArgs {
  Args a;
  int r16;                // ranks of the product, a multiple of 16
  int stages, ring_bytes;
  uint32_t tmem_cols;
};

struct OutArgs {
  Args a;
  int panels;             // panels of 64 ranks
  int stages;
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

// 128 columns of B by 64 ranks from block z of 64 columns on, in the order that its map gives.
__device__ __forceinline__ void tma_load_5d(void *dst, const CUtensorMap *m, uint64_t *bar, int x, int z) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %4, %4, %5}], "
      "[%2];\n" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(tc::smem_u32(bar)), "r"(x), "r"(0), "r"(z)
      : "memory");
}

// 64 (or 32) accumulator columns of 16 lanes: register 4 j + i is column 8 j + 2 (lane % 4) + i % 2 of
// lane lane / 4 + 8 (i / 2).
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// 32 bytes of y or out: one access where the rows allow it.
struct Chunk {
  uint32_t w[8];
};
__device__ __forceinline__ void load_chunk(Chunk &c, const char *p, bool wide) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
                 : "=r"(c.w[0]), "=r"(c.w[1]), "=r"(c.w[2]), "=r"(c.w[3]), "=r"(c.w[4]), "=r"(c.w[5]), "=r"(c.w[6]),
                   "=r"(c.w[7])
                 : "l"(p)
                 : "memory");
  } else {
    const uint4 u = *reinterpret_cast<const uint4 *>(p), v = *reinterpret_cast<const uint4 *>(p + 16);
    c = {{u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w}};
  }
}
__device__ __forceinline__ void store_chunk(char *p, const Chunk &c, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p), "r"(c.w[0]), "r"(c.w[1]),
                 "r"(c.w[2]), "r"(c.w[3]), "r"(c.w[4]), "r"(c.w[5]), "r"(c.w[6]), "r"(c.w[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4 *>(p) = make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]);
    *reinterpret_cast<uint4 *>(p + 16) = make_uint4(c.w[4], c.w[5], c.w[6], c.w[7]);
  }
}

// ------------------------------------------------------------------- h = x A^T

__global__ void __launch_bounds__(kInThreads) adapter_in_kernel(const __grid_constant__ CUtensorMap mx,
                                                                const __grid_constant__ CUtensorMap mt,
                                                                const __grid_constant__ CUtensorMap ma,
                                                                const InArgs g) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = tc::smem_u32(smem_raw);
  uint8_t *ring = smem_raw + (((raw + 1023u) & ~1023u) - raw);      // operands, then the sums
  uint64_t *full = reinterpret_cast<uint64_t *>(ring + g.ring_bytes), *empty = full + 8, *done = empty + 8;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  volatile int *failed = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const Args &a = g.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, S = gridDim.x, split = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 8; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    tc::mbar_init(done, 1);
    *failed = 0;
    tc::fence_mbar_init();
    tc::prefetch_tmap(&mx);
    tc::prefetch_tmap(&mt);
    tc::prefetch_tmap(&ma);
  }
  pdl_wait();
  const int tiles = plan_tiles(a, kPlanTcTiles);
  const int4 tile = a.tiles[blockIdx.y];
  const int rank = (int)blockIdx.y < tiles && tile.x >= 0 ? adapter_rank(a, tile.x) : 0;
  if (rank == 0) {                                                  // (the whole cluster)
    pdl_trigger();
    return;
  }
  // TMEM only now: nobody ahead on the stream waits for it, and what comes next
  // may start once all of this kernel has its own
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, g.tmem_cols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();

  const int KB = a.k / 64, kb0 = KB * split / S, kb1 = KB * (split + 1) / S;
  const int stage_bytes = kPanel + g.r16 * 128;
  const int pitch = g.r16 + 4;                                      // floats between rows of sums
  if (warp == 0) {
    // lane i gathers rows 4 i .. 4 i + 3 (past the last row: that one again)
    const int quads = (tile.z + 3) / 4;
    int4 rows;
    {
      const int *p = a.perm + tile.y;
      const int last = tile.z - 1, i = min(4 * lane, last);
      rows = make_int4(p[i], p[min(i + 1, last)], p[min(i + 2, last)], p[min(i + 3, last)]);
    }
    // Rows that follow one another (a prompt's) come as one box, whose rows past the
    // tile are somebody else's: 32 gathers take an SM a microsecond, a box a tenth.
    const int at = __shfl_sync(0xffffffffu, rows.x, 0), n = min(4, tile.z - 4 * lane);
    const bool box = __all_sync(0xffffffffu, lane >= quads ||
                                                 (rows.x == at + 4 * lane && rows.y == rows.x + (n > 1) &&
                                                  rows.z == rows.y + (n > 2) && rows.w == rows.z + (n > 3)));
    int st = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      bool ok = true;
      if (lane == 0) {
        ok = tc::mbar_wait(&empty[st], phase ^ 1);
        if (ok) tc::mbar_arrive_expect_tx(&full[st], (box ? kPanel : quads * 512) + g.r16 * 128);
        else *failed = 1;
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      uint8_t *sx = ring + st * stage_bytes;
      if (box) {
        if (lane == 0) tc::tma_load_2d(sx, &mt, &full[st], kb * 64, at);
      } else if (lane < quads) tma_gather4(sx + lane * 512, &mx, &full[st], kb * 64, rows);
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
  } else {
    if (!__all_sync(0xffffffffu, tc::mbar_wait(done, 0))) *failed = 1;
    tc::tc_fence_after();
    const int row = 32 * (warp & 3) + lane;
    float *dst = reinterpret_cast<float *>(ring) + row * pitch;
    for (int c = 0; c < g.r16; c += 32) {
      float v[32];
      if (kb0 < kb1) {
        tc::tmem_ld32(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + c, v);
        tc::tmem_ld_wait();
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0.0f;                   // (no share of k)
      }
#pragma unroll
      for (int i = 0; i < 32; i += 4)
        if (c + i < g.r16) *reinterpret_cast<float4 *>(dst + c + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
    tc::tc_fence_before();
  }
  cluster_arrive();
  cluster_wait();

  // 16 threads to a row, eight ranks each (a half-warp stays whole: a CTA's rows are a multiple of 16)
  if (warp >= 2) {
    const int per = kTcRows / S, t = threadIdx.x - 64, c = 8 * (t & 15);
    for (int r0 = t >> 4; r0 < per; r0 += 8) {
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
        if (c + i >= rank) v[i] = 0.0f;
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
      if (r < tile.z) {                                             // (rows past the last one: whatever was there)
        const int64_t row = tile.y + r;
        if (c < a.R) {
          *reinterpret_cast<uint4 *>(a.h + row * a.R + c) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4 *>(a.h + ((int64_t)a.T + row) * a.R + c) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        if (c == 0) a.back[row] = __ldg(a.scale + tile.x) * scalbnf(1.0f, -p);
      }
    }
  }
  cluster_arrive();
  cluster_wait();                                                   // nobody leaves while its sums are read
  if (*failed && threadIdx.x == 0) set_device_error(a.err, kErrBounds);
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, g.tmem_cols);
  }
}

// --------------------------------------------------------------- out = y + h B^T

// A CTA's run of the line: columns [nb0, nb1) (in 128s) of each tile from
// `first` on.  A tile's place is tile.w * NB, a column block as wide as
// its tile costs.
struct Run {
  int64_t lo, hi;
  int first, tiles, NB;
  __device__ __forceinline__ bool part(const Args &a, int i, int4 &tile, int &nb0, int &nb1) const {
    if (i >= tiles) return false;
    tile = a.tiles[i];
    const int64_t at = (int64_t)tile.w * NB;
    if (at >= hi) return false;
    const int cost = tile.z + kTileCost;
    nb0 = (int)(max((int64_t)0, lo - at + cost - 1) / cost);
    nb1 = (int)min((int64_t)NB, (hi - at + cost - 1) / cost);
    return true;
  }
};

template <bool F32, int CTAS>
__global__ void __launch_bounds__(kOutThreads, CTAS) adapter_out_kernel(const __grid_constant__ CUtensorMap mh,
                                                                        const __grid_constant__ CUtensorMap mb,
                                                                        const OutArgs g) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = tc::smem_u32(smem_raw);
  uint8_t *hs = smem_raw + (((raw + 1023u) & ~1023u) - raw);        // [2][panels]: hi, lo
  uint8_t *ring = hs + 2 * g.panels * kPanel;                       // B
  uint64_t *full = reinterpret_cast<uint64_t *>(ring + g.stages * g.panels * kPanel);
  uint64_t *empty = full + 8, *h_full = empty + 8, *h_empty = h_full + 1, *t_full = h_empty + 1, *t_empty = t_full + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(t_empty + 2);
  volatile int *failed = reinterpret_cast<volatile int *>(tmem_slot + 1);
  volatile int *first = failed + 1;
  const Args &a = g.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 8; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    tc::mbar_init(h_full, 1);
    tc::mbar_init(h_empty, 1);
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(&t_full[s], 1);
      tc::mbar_init(&t_empty[s], kEpiWarps);
    }
    *failed = 0;
    *first = 0x7fffffff;
    tc::fence_mbar_init();
    tc::prefetch_tmap(&mh);
    tc::prefetch_tmap(&mb);
  }
  pdl_wait();
  if (warp == 1) {                                                  // (after the wait, as above)
    tc::tmem_alloc(tmem_slot, kOutCols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();
  Run run;
  run.tiles = plan_tiles(a, kPlanTcTiles);
  run.NB = a.n / 128;
  {
    const int64_t total = (int64_t)a.ctrl[kPlanCost] * run.NB;
    run.lo = total * blockIdx.x / gridDim.x;
    run.hi = total * (blockIdx.x + 1) / gridDim.x;
    // the tile that holds the run's first place
    for (int i = threadIdx.x; i < run.tiles; i += kOutThreads) {
      const int4 t = a.tiles[i];
      const int64_t at = (int64_t)t.w * run.NB;
      if (at <= run.lo && run.lo < at + (int64_t)(t.z + kTileCost) * run.NB) *first = i;
    }
    __syncthreads();
    run.first = *first;
  }

  int4 tile;
  int nb0, nb1;
  if (warp == 0) {
    if (lane == 0) {
      const int bytes = g.panels * kPanel;
      int st = 0;
      uint32_t phase = 0, h_phase = 0;
      bool ok = true;
      for (int i = run.first; ok && run.part(a, i, tile, nb0, nb1); ++i) {
        if (tile.x < 0 || nb0 >= nb1 || adapter_rank(a, tile.x) == 0) continue;
        ok = tc::mbar_wait(h_empty, h_phase ^ 1);
        if (!ok) break;
        h_phase ^= 1;
        tc::mbar_arrive_expect_tx(h_full, 2 * bytes);
        for (int p = 0; p < 2 * g.panels; ++p)
          tc::tma_load_3d(hs + p * kPanel, &mh, h_full, p % g.panels * 64, tile.y, p / g.panels);
        for (int nb = nb0; nb < nb1; ++nb) {
          ok = tc::mbar_wait(&empty[st], phase ^ 1);
          if (!ok) break;
          tc::mbar_arrive_expect_tx(&full[st], bytes);
          for (int p = 0; p < g.panels; ++p)
            tma_load_5d(ring + st * bytes + p * kPanel, &mb, &full[st], p * 64, tile.x * (a.n / 64) + 2 * nb);
          if (++st == g.stages) { st = 0; phase ^= 1; }
        }
      }
      if (!ok) *failed = 1;
    }
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t idesc = tc::idesc_f16(kTcRows, 128);
    const uint64_t hd = tc::sdesc_k_sw128(hs);
    int st = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0, h_phase = 0;
    bool ok = true;
    for (int i = run.first; ok && run.part(a, i, tile, nb0, nb1); ++i) {
      if (tile.x < 0 || nb0 >= nb1) continue;
      const int kr = (adapter_rank(a, tile.x) + 15) / 16;
      if (kr == 0) continue;
      ok = __all_sync(0xffffffffu, tc::mbar_wait(h_full, h_phase));
      h_phase ^= 1;
      for (int nb = nb0; ok && nb < nb1; ++nb) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&t_empty[acc], acc_phase ^ 1) && tc::mbar_wait(&full[st], phase));
        if (!ok) break;
        tc::tc_fence_after();
        const uint64_t bd = tc::sdesc_k_sw128(ring + st * g.panels * kPanel);
        if (tc::elect_one()) {
          for (int part = 0; part < 2; ++part)
            for (int kk = 0; kk < kr; ++kk) {
              const uint32_t in = (kk >> 2) * (kPanel >> 4) + (kk & 3) * 2;
              tc::mma_f16(tmem + acc * 128, hd + part * (g.panels * kPanel >> 4) + in, bd + in, idesc,
                          part || kk ? 1u : 0u);
            }
          tc::mma_commit(&empty[st]);
          tc::mma_commit(&t_full[acc]);
          if (nb + 1 == nb1) tc::mma_commit(h_empty);
        }
        __syncwarp();
        if (++st == g.stages) { st = 0; phase ^= 1; }
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
    }
    if (!ok) *failed = 1;
  } else {
    // warps 2-9: 32 rows by 64 columns each, 16 rows at a time; lane: rows g and
    // g + 8, 16 columns (fp32: eight, in two goes)
    constexpr int SIZE = F32 ? 4 : 2, COLS = 32 / SIZE, GOES = 16 / COLS, CHUNKS = 2 * GOES;
    const int quarter = warp & 3, half = (warp - 2) >> 2, gr = lane >> 2, col = half * 64 + 16 * (lane & 3);
    const bool wide = g.wide;
    const char *src = static_cast<const char *>(a.y) + col * SIZE;
    char *dst = static_cast<char *>(a.out) + col * SIZE;
    const int64_t y_bytes = a.y_stride * SIZE, out_bytes = a.out_stride * SIZE;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int i = run.first; ok && run.part(a, i, tile, nb0, nb1); ++i) {
      if (nb0 >= nb1) continue;
      const bool copy = tile.x < 0 || adapter_rank(a, tile.x) == 0;
      if (copy && a.out == a.y) continue;
      int rows[4];                                                  // of m: 8 m + g; -1: none
      float f[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int r = 32 * quarter + 8 * m + gr;
        rows[m] = r < tile.z ? a.perm[tile.y + r] : -1;
        f[m] = r < tile.z && !copy ? a.back[tile.y + r] : 0.0f;
      }
      Chunk y[2][2];
      // chunk c of a block: rows of m = c / GOES, columns COLS (c % GOES) on
      const auto load = [&](int nb, int c) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (rows[2 * (c / GOES) + h] >= 0)
            load_chunk(y[c & 1][h], src + rows[2 * (c / GOES) + h] * y_bytes + (nb * 128 + c % GOES * COLS) * SIZE, wide);
      };
      load(nb0, 0);
      load(nb0, 1);
      for (int nb = nb0; nb < nb1; ++nb) {
        if (!copy) {
          ok = __all_sync(0xffffffffu, tc::mbar_wait(&t_full[acc], acc_phase));
          if (!ok) break;
          tc::tc_fence_after();
        }
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
          float v[2 * COLS];
          if (!copy) {
            tmem_ld_rows(tmem + ((uint32_t)(32 * quarter + 16 * (c / GOES)) << 16) + acc * 128 + half * 64 + c % GOES * 32, v);
            tc::tmem_ld_wait();
            if (c + 1 == CHUNKS) {
              tc::tc_fence_before();
              __syncwarp();
              if (lane == 0) tc::mbar_arrive(&t_empty[acc]);
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int m = 2 * (c / GOES) + h;
            if (rows[m] < 0) continue;
            Chunk &t = y[c & 1][h];
            if (!copy) {
#pragma unroll
              for (int j = 0; j < COLS / 2; ++j) {
                const float d0 = v[4 * j + 2 * h], d1 = v[4 * j + 2 * h + 1];
                if (F32) {
                  t.w[(2 * j) % 8] = __float_as_uint(fmaf(f[m], d0, __uint_as_float(t.w[(2 * j) % 8])));
                  t.w[(2 * j + 1) % 8] = __float_as_uint(fmaf(f[m], d1, __uint_as_float(t.w[(2 * j + 1) % 8])));
                } else {
                  const float2 z = __half22float2(*reinterpret_cast<const __half2 *>(&t.w[j]));
                  const __half2 o = __floats2half2_rn(fmaf(f[m], d0, z.x), fmaf(f[m], d1, z.y));
                  t.w[j] = *reinterpret_cast<const uint32_t *>(&o);
                }
              }
            }
            store_chunk(dst + rows[m] * out_bytes + (nb * 128 + c % GOES * COLS) * SIZE, t, wide);
          }
          if (c + 2 < CHUNKS) load(nb, c + 2);
          else if (nb + 1 < nb1) load(nb + 1, c + 2 - CHUNKS);
        }
        if (!copy && ++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
    }
    if (!ok) *failed = 1;
  }
  tc::tc_fence_before();
  __syncthreads();
  if (*failed && threadIdx.x == 0) set_device_error(a.err, kErrBounds);
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kOutCols);
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
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, dims, const_cast<void *>(base), size, stride, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return exl3_fail(EXL3_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return EXL3_OK;
}

int launch_in(const ad::Args &a, cudaStream_t s) {
  ad::InArgs g = {};
  g.a = a;
  g.r16 = (a.R + 15) / 16 * 16;
  const int stage = ad::kPanel + g.r16 * 128;
  // a ring of 72 KB: at most three CTAs on an SM, whose 128 TMEM columns each fit
  // (a CTA that waited for TMEM while its cluster waits for it could wait for ever)
  g.stages = 72 * 1024 / stage;
  g.ring_bytes = 72 * 1024;
  g.tmem_cols = 32;
  while ((int)g.tmem_cols < g.r16) g.tmem_cols *= 2;
  const size_t smem = 1024 + g.ring_bytes + 17 * 8 + 8;
  CUtensorMap mx, mt, ma;      // x for gathers of rows and for boxes; A
  {
    const cuuint64_t dims[2] = {(cuuint64_t)a.k, (cuuint64_t)a.T}, stride[1] = {(cuuint64_t)a.x_stride * 2};
    const cuuint32_t row[2] = {64, 1}, box[2] = {64, ad::kTcRows};
    int rc = map_f16(&mx, a.x, 2, dims, stride, row);
    if (rc) return rc;
    rc = map_f16(&mt, a.x, 2, dims, stride, box);
    if (rc) return rc;
  }
  {
    const cuuint64_t dims[3] = {(cuuint64_t)a.k, (cuuint64_t)a.R, (cuuint64_t)a.N};
    const cuuint64_t stride[2] = {(cuuint64_t)a.k * 2, (cuuint64_t)a.k * a.R * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)g.r16, 1};
    int rc = map_f16(&ma, a.a, 3, dims, stride, box);
    if (rc) return rc;
  }
  static std::atomic<size_t> given[kMaxDevices];
  int rc = exl3_cuda_check(exl3_ensure_smem(reinterpret_cast<const void *>(ad::adapter_in_kernel), smem, given),
                           "adapter attribute");
  if (rc) return rc;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 8;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(8, a.max_tiles);
  cfg.blockDim = dim3(ad::kInThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return exl3_cuda_check(cudaLaunchKernelEx(&cfg, ad::adapter_in_kernel, mx, mt, ma, g), "adapter launch");
}

template <bool F32, int CTAS>
int launch_out(const ad::OutArgs &g, cudaStream_t s) {
  const ad::Args &a = g.a;
  CUtensorMap mh, mb;
  {
    const cuuint64_t dims[3] = {(cuuint64_t)a.R, (cuuint64_t)a.T, 2};
    const cuuint64_t stride[2] = {(cuuint64_t)a.R * 2, (cuuint64_t)a.T * a.R * 2};
    const cuuint32_t box[3] = {64, 128, 1};
    int rc = map_f16(&mh, a.h, 3, dims, stride, box);
    if (rc) return rc;
  }
  {
    // column 16 t + 2 j + b of 64 goes to row 8 j + 2 t + b of the operand
    const cuuint64_t R = a.R, dims[5] = {R, 2, 4, 8, (cuuint64_t)a.n / 64 * a.N};
    const cuuint64_t stride[4] = {R * 2, R * 32, R * 4, R * 128};
    const cuuint32_t box[5] = {64, 2, 4, 8, 2};
    int rc = map_f16(&mb, a.b, 5, dims, stride, box);
    if (rc) return rc;
  }
  const size_t smem = 1024 + (2 + g.stages) * (size_t)g.panels * ad::kPanel + 22 * 8 + 16;
  auto kfn = ad::adapter_out_kernel<F32, CTAS>;
  static std::atomic<size_t> given[kMaxDevices];
  int rc = exl3_cuda_check(exl3_ensure_smem(reinterpret_cast<const void *>(kfn), smem, given), "adapter attribute");
  if (rc) return rc;
  return exl3_cuda_check(launch_pdl(kfn, dim3(exl3_sm_count() * CTAS), dim3(ad::kOutThreads), smem, s, mh, mb, g),
                         "adapter launch");
}

}  // namespace

int exl3_launch_adapter_tc(const ad::Args &a, bool f32, cudaStream_t s) {
  int rc = launch_in(a, s);
  if (rc) return rc;
  ad::OutArgs g = {};
  g.a = a;
  g.panels = (a.R + 63) / 64;
  // Up to rank 64 two CTAs on an SM (operands of 32 KB, a ring of 64), above it one
  g.stages = g.panels == 1 ? 4 : 3;
  const int size = f32 ? 4 : 2;
  const auto on32 = [&](const void *p, int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % 32 == 0 && stride * size % 32 == 0;
  };
  g.wide = on32(a.y, a.y_stride) && on32(a.out, a.out_stride);
  if (g.panels == 1) return f32 ? launch_out<true, 2>(g, s) : launch_out<false, 2>(g, s);
  return f32 ? launch_out<true, 1>(g, s) : launch_out<false, 1>(g, s);
}
