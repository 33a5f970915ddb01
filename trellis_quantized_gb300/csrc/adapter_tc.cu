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
// Four prompts of 6301 tokens, rank 16, 5120 -> 17408, take 98 us: 19 and 79, the
// second 439 MB of y and out at 0.8 of the copy rate.  One launch (the cluster keeps h
// and splits the columns too) took 228: 50 tiles are two rounds of clusters, one of
// them almost empty.
//
// h: each row is brought to [2^14, 2^15) by a power of two and then hi + lo, 22
// bits; the second product runs over both parts (twice the operations of a small
// K), so an fp32 out is as good as its sums.
//
// The accumulator is read in the layout of 16 x 256 bits: a lane gets two columns
// of every eight for rows g and g + 8.  The copy of B permutes its rows (as a
// tensor map of five dimensions) so that these are 32 neighbouring bytes of out:
// four lanes write one 128-byte line, and no transposition is needed.
#include "adapter.cuh"
#include "tc_ptx.cuh"

namespace exl3 {
namespace ad {

constexpr int kPanel = kTcRows * 128;           // bytes of 128 rows of 64 fp16
constexpr int kInThreads = 192;                 // producer, issuer, four warps for the sums
constexpr int kEpiWarps = 8;
constexpr int kOutThreads = (3 + kEpiWarps) * 32;   // producers of h and B, and of y; issuer; output
constexpr uint32_t kOutCols = 256;              // TMEM: two accumulators
constexpr int kBStages = 4, kYPlaces = 8;       // at most: blocks of B, pieces of y

struct InArgs {
  Args a;
  int r16;                // ranks of the product, a multiple of 16
  int stages, ring_bytes;
  uint32_t tmem_cols;
};

struct OutArgs {
  Args a;
  int panels;             // panels of 64 ranks
  int stages, y_stages;   // blocks of B; pieces of y
  int wide;               // out may be written 32 bytes at a time
};

// Rings of the output kernel: 224 KB hold h, blocks of B (as far ahead as y, behind
// whose copies theirs queue: two blocks and ten pieces took 109 us on the prompts
// above) and pieces of y.  The places for pieces are a multiple of a block's pieces, so
// that a place always serves the same four warps: a warp that did not see each of its
// phases could not tell them apart.
struct Rings {
  int stages, y_stages;
};
constexpr Rings out_rings(int panels, bool f32) {
  return {panels == 1 ? 4 : f32 ? 3 : 2, panels == 1 ? 8 : f32 ? 4 : 6};
}
constexpr size_t out_smem(int panels, Rings r) {
  return 1024 + ((2 + r.stages) * (size_t)panels + r.y_stages) * kPanel + (6 + 2 * kBStages + 2 * kYPlaces) * 8 + 16;
}
constexpr bool rings_fit(int panels, bool f32) {
  const Rings r = out_rings(panels, f32);
  return r.y_stages % (f32 ? 4 : 2) == 0 && r.y_stages <= kYPlaces && r.stages <= kBStages &&
         out_smem(panels, r) <= 227 * 1024;
}
static_assert(rings_fit(1, false) && rings_fit(1, true) && rings_fit(2, false) && rings_fit(2, true),
              "whole blocks of pieces, a barrier for every place, the shared memory of a CTA");

// Four rows of a tensor map (its box is one row), 64 columns each.
__device__ __forceinline__ void tma_gather4(void *dst, const CUtensorMap *m, uint64_t *bar, int x, const int4 &rows) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
      "%5, %6, %7}], [%2];\n" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(tc::smem_u32(bar)), "r"(x), "r"(rows.x), "r"(rows.y), "r"(rows.z),
      "r"(rows.w)
      : "memory");
}

// 128 columns of B by 64 ranks, from place z on in the order that its map gives.
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

// 32 bytes of out: one store where the rows allow it.
struct Chunk {
  uint32_t w[8];
};
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

// The rows of a tile as one warp's copies of 128-byte pieces see them, 32 at a time:
// one box where they follow one another (a prompt's; rows of the box past the tile
// are somebody else's), else gathers of four, lane i rows 4 i .. 4 i + 3 (past the
// last row: that one again).  32 gathers take an SM a microsecond, a box of as many
// rows a tenth.  One elected lane starts the boxes and a vote skips the gathers: copies
// under conditions that the compiler cannot tell to be one lane's took the warp 1100
// cycles a piece, 600 of them for a branch that no lane took.
struct TileRows {
  int4 rows;
  int quads, total;
  int first[4];           // rows of the boxes
  unsigned boxes;         // a bit for each that is one
  bool gather;            // this lane's rows
  __device__ __forceinline__ void load(const Args &a, const int4 &tile, int lane) {
    const int *p = a.perm + tile.y;
    const int last = tile.z - 1, i = min(4 * lane, last), n = min(4, tile.z - 4 * lane);
    rows = make_int4(p[i], p[min(i + 1, last)], p[min(i + 2, last)], p[min(i + 3, last)]);
    quads = (tile.z + 3) / 4;
    const int start = __shfl_sync(0xffffffffu, rows.x, lane & 24);
    const bool next = rows.x == start + 4 * (lane & 7) && rows.y == rows.x + (n > 1) && rows.z == rows.y + (n > 2) &&
                      rows.w == rows.z + (n > 3);
    const unsigned apart = __ballot_sync(0xffffffffu, lane < quads && !next);
    boxes = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      first[b] = __shfl_sync(0xffffffffu, rows.x, 8 * b);
      // (fewer than twelve rows: three gathers at most)
      if (!(apart >> (8 * b) & 0xffu) && tile.z - 32 * b >= 12) boxes |= 1u << b;
    }
    gather = lane < quads && !(boxes >> (lane >> 3) & 1u);
    total = __popc(boxes) * 4096 + __popc(__ballot_sync(0xffffffffu, gather)) * 512;
  }
  // Bytes that a piece's copies bring.
  __device__ __forceinline__ int bytes() const { return total; }
  // The piece at column x: `box_map` has boxes of 32 rows, `row_map` of one.
  __device__ __forceinline__ void copy(uint8_t *dst, const CUtensorMap *box_map, const CUtensorMap *row_map,
                                       uint64_t *bar, int x, int lane) const {
    if (tc::elect_one()) {
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (boxes >> b & 1u) tc::tma_load_2d(dst + b * 4096, box_map, bar, x, first[b]);
    }
    if (__any_sync(0xffffffffu, gather)) {
      if (gather) tma_gather4(dst + lane * 512, row_map, bar, x, rows);
      __syncwarp();
    }
  }
};

// ------------------------------------------------------------------- h = x A^T

// S: CTAs of a cluster, shares of k.
template <int S>
__global__ void __launch_bounds__(kInThreads) adapter_in_kernel(const __grid_constant__ CUtensorMap mx,
                                                                const __grid_constant__ CUtensorMap mt,
                                                                const __grid_constant__ CUtensorMap ma,
                                                                const InArgs g) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = tc::smem_u32(smem_raw);
  uint8_t *ring = smem_raw + (((raw + 1023u) & ~1023u) - raw);      // operands, then the sums
  uint64_t *full = reinterpret_cast<uint64_t *>(ring + g.ring_bytes), *empty = full + 8, *done = empty + 8;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  volatile int *failed = reinterpret_cast<volatile int *>(tmem_slot + 1), *used = failed + 1;   // (uses of the ring)
  const Args &a = g.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, split = blockIdx.x;

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
  int4 tile = make_int4(-1, 0, 0, 0);
  if ((int)blockIdx.y < tiles) tile = a.tiles[blockIdx.y];          // (else it may lie behind another call's plan)
  const bool some = tile.x >= 0;
  TileRows rows;
  if (some && warp == 0) rows.load(a, tile, lane);                  // (beside the rank's load)
  const int rank = some ? adapter_rank(a, tile.x) : 0;
  if (rank == 0) {                                                  // (the whole cluster)
    pdl_trigger();
    return;
  }
  const int KB = a.k / 64, kb0 = KB * split / S, kb1 = KB * (split + 1) / S;
  if (threadIdx.x == 0) *used = kb1 - kb0;
  const int stage_bytes = kPanel + g.r16 * 128;
  const int pitch = g.r16 + 4;                                      // floats between rows of sums
  const auto bring = [&](int st, int kb) {                          // (warp 0)
    uint8_t *sx = ring + st * stage_bytes;
    if (tc::elect_one()) {
      tc::mbar_arrive_expect_tx(&full[st], rows.bytes() + g.r16 * 128);
      tc::tma_load_3d(sx + kPanel, &ma, &full[st], kb * 64, 0, tile.x);
    }
    __syncwarp();
    rows.copy(sx, &mt, &mx, &full[st], kb * 64, lane);
  };
  const int ahead = min(kb1, kb0 + g.stages);
  __syncwarp();
  if (warp == 0)                                                    // the ring's first round
    for (int kb = kb0; kb < ahead; ++kb) bring(kb - kb0, kb);
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

  if (warp == 0) {
    int st = 0;
    uint32_t phase = 0;
    for (int kb = ahead; kb < kb1; ++kb) {
      const bool ok = __all_sync(0xffffffffu, lane != 0 || tc::mbar_wait(&empty[st], phase));
      if (!ok) {
        *failed = 1;
        *used = kb - kb0;
        break;
      }
      bring(st, kb);
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
        for (int kk = 0; kk < 4; ++kk)
          tc::mma_f16(tmem, ad + 2 * kk, bd + 2 * kk, idesc, (kb != kb0 || kk != 0) ? 1u : 0u);
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

  // `per_row` threads to a row, eight ranks each (a warp stays whole: a CTA's rows are a multiple of 16)
  if (warp >= 2) {
    constexpr int per = kTcRows / S;
    int per_row = 2;
    while (per_row * 8 < g.r16) per_row *= 2;
    const int t = threadIdx.x - 64, c = 8 * (t & (per_row - 1));
    for (int r0 = t / per_row; r0 < per; r0 += 128 / per_row) {
      const int r = split * per + r0;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
      if (c < rank && r < tile.z) {
        const uint32_t at = tc::smem_u32(ring) + (uint32_t)(r * pitch + c) * 4;
        float4 p[S], q[S];                                // (all on their way at once)
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const uint32_t from = map_rank(at, s);
          p[s] = ld_cluster4(from);
          q[s] = ld_cluster4(from + 16);
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
          v[0] += p[s].x; v[1] += p[s].y; v[2] += p[s].z; v[3] += p[s].w;
          v[4] += q[s].x; v[5] += q[s].y; v[6] += q[s].z; v[7] += q[s].w;
        }
      }
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (c + i >= rank) v[i] = 0.0f;
        top = fmaxf(top, fabsf(v[i]));
      }
#pragma unroll
      for (int o = 8; o; o >>= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, top, o);
        if (o < per_row) top = fmaxf(top, other);
      }
      const int p = row_exponent(top);
      const float f = scalbnf(1.0f, p);
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        __half2 h, l;
        split_h(v[2 * i] * f, isinf(top), h.x, l.x);
        split_h(v[2 * i + 1] * f, isinf(top), h.y, l.y);
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
  if (*failed && threadIdx.x == 0) {
    set_device_error(a.err, kErrBounds);
    tc::drain(full, g.stages, *used);                               // leave no copy in flight behind
  }
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

// A tile whose rows keep y.
__device__ __forceinline__ bool copies(const Args &a, const int4 &tile) {
  return tile.x < 0 || adapter_rank(a, tile.x) == 0;
}

// Warp 0 brings h and B, warp 1 issues the products, warps 2 to 9 add y and write
// out, warp 10 brings y: pieces of 128 rows by 128 bytes, a ring of 64 to
// 128 KB of them (loads into registers, 64 KB of them in flight, ran at 2.2 TB/s).
template <bool F32>
__global__ void __launch_bounds__(kOutThreads, 1) adapter_out_kernel(const __grid_constant__ CUtensorMap mh,
                                                                     const __grid_constant__ CUtensorMap mb,
                                                                     const __grid_constant__ CUtensorMap my,
                                                                     const __grid_constant__ CUtensorMap mr,
                                                                     const OutArgs g) {
  constexpr int SIZE = F32 ? 4 : 2, PIECES = F32 ? 4 : 2, PCOLS = 128 / SIZE;   // pieces of 128 columns
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = tc::smem_u32(smem_raw);
  uint8_t *hs = smem_raw + (((raw + 1023u) & ~1023u) - raw);        // [2][panels]: hi, lo
  uint8_t *ring = hs + 2 * g.panels * kPanel;                       // B
  uint8_t *ys = ring + g.stages * g.panels * kPanel;                // y
  uint64_t *full = reinterpret_cast<uint64_t *>(ys + g.y_stages * kPanel), *empty = full + kBStages;
  uint64_t *y_full = empty + kBStages, *y_empty = y_full + kYPlaces;
  uint64_t *h_full = y_empty + kYPlaces, *h_empty = h_full + 1, *t_full = h_empty + 1, *t_empty = t_full + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(t_empty + 2);
  volatile int *failed = reinterpret_cast<volatile int *>(tmem_slot + 1);
  volatile int *first = failed + 1;
  const Args &a = g.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kBStages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kYPlaces; ++s) {
      tc::mbar_init(&y_full[s], 1);
      tc::mbar_init(&y_empty[s], 4);
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
    tc::prefetch_tmap(&my);
    tc::prefetch_tmap(&mr);
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
  int nb0, nb1, used = 0, h_used = 0;                               // (of B's or y's ring, and of h's place)
  bool ok = true;
  if (warp == 0) {
    if (lane == 0) {
      const int bytes = g.panels * kPanel;
      int st = 0;
      uint32_t phase = 0, h_phase = 0;
      for (int i = run.first; ok && run.part(a, i, tile, nb0, nb1); ++i) {
        if (nb0 >= nb1 || copies(a, tile)) continue;
        ok = tc::mbar_wait(h_empty, h_phase ^ 1);
        if (!ok) break;
        h_phase ^= 1;
        tc::mbar_arrive_expect_tx(h_full, 2 * bytes);
        for (int p = 0; p < 2 * g.panels; ++p)
          tc::tma_load_3d(hs + p * kPanel, &mh, h_full, p % g.panels * 64, tile.y, p / g.panels);
        ++h_used;
        for (int nb = nb0; nb < nb1; ++nb) {
          ok = tc::mbar_wait(&empty[st], phase ^ 1);
          if (!ok) break;
          tc::mbar_arrive_expect_tx(&full[st], bytes);
          for (int p = 0; p < g.panels; ++p)
            tma_load_5d(ring + st * bytes + p * kPanel, &mb, &full[st], p * 64, (tile.x * run.NB + nb) * (F32 ? 4 : 2));
          ++used;
          if (++st == g.stages) { st = 0; phase ^= 1; }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t idesc = tc::idesc_f16(kTcRows, 128);
    const uint64_t hd = tc::sdesc_k_sw128(hs);
    int st = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0, h_phase = 0;
    for (int i = run.first; ok && run.part(a, i, tile, nb0, nb1); ++i) {
      if (nb0 >= nb1 || copies(a, tile)) continue;
      const int kr = (adapter_rank(a, tile.x) + 15) / 16;
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
          if (nb + 1 == nb1) tc::mma_commit(h_empty);
          tc::mma_commit(&t_full[acc]);                             // (last: what waits for it ends the kernel)
        }
        __syncwarp();
        if (++st == g.stages) { st = 0; phase ^= 1; }
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
    }
  } else if (warp == 2 + kEpiWarps) {
    int st = 0;
    uint32_t phase = 0;
    for (int i = run.first; ok && run.part(a, i, tile, nb0, nb1); ++i) {
      if (nb0 >= nb1 || (a.out == a.y && copies(a, tile))) continue;
      TileRows rows;
      rows.load(a, tile, lane);
      for (int p = nb0 * PIECES; p < nb1 * PIECES; ++p) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&y_empty[st], phase ^ 1));
        if (!ok) break;
        if (tc::elect_one()) tc::mbar_arrive_expect_tx(&y_full[st], rows.bytes());
        __syncwarp();
        rows.copy(ys + st * kPanel, &my, &mr, &y_full[st], p * PCOLS, lane);
        ++used;
        if (++st == g.y_stages) { st = 0; phase ^= 1; }
      }
    }
  } else {
    // 32 rows by 64 columns per block and warp, 16 rows at a time; a lane: rows g
    // and g + 8, 16 neighbouring columns (fp32: eight, in two pieces)
    constexpr int COLS = 32 / SIZE, GOES = PIECES / 2;
    const int quarter = warp & 3, half = (warp - 2) >> 2, gr = lane >> 2, t = lane & 3;
    const bool wide = g.wide;
    char *dst = static_cast<char *>(a.out) + (half * 64 + COLS * t) * SIZE;
    const int64_t out_bytes = a.out_stride * SIZE;
    int acc = 0, st = half * GOES;                                  // this half's first piece
    uint32_t acc_phase = 0, phase = 0;
    for (int i = run.first; ok && run.part(a, i, tile, nb0, nb1); ++i) {
      if (nb0 >= nb1) continue;
      const bool copy = copies(a, tile);
      if (copy && a.out == a.y) continue;
      int rows[4];                                                  // of m: 8 m + g; -1: none
      float f[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int r = 32 * quarter + 8 * m + gr;
        rows[m] = r < tile.z ? a.perm[tile.y + r] : -1;
        f[m] = r < tile.z && !copy ? a.back[tile.y + r] : 0.0f;
      }
      for (int nb = nb0; nb < nb1; ++nb) {
        if (!copy) {
          ok = __all_sync(0xffffffffu, tc::mbar_wait(&t_full[acc], acc_phase));
          if (!ok) break;
          tc::tc_fence_after();
        }
#pragma unroll
        for (int go = 0; go < GOES; ++go) {
          float v[2][2 * COLS];
          if (!copy) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
              tmem_ld_rows(tmem + ((uint32_t)(32 * quarter + 16 * m) << 16) + acc * 128 + half * 64 + go * 32, v[m]);
            tc::tmem_ld_wait();
            if (go + 1 == GOES) {
              tc::tc_fence_before();
              __syncwarp();
              if (lane == 0) tc::mbar_arrive(&t_empty[acc]);
            }
          }
          ok = __all_sync(0xffffffffu, tc::mbar_wait(&y_full[st], phase));
          if (!ok) break;
          const uint8_t *piece = ys + st * kPanel;
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            // 128-byte swizzle; a row's 16-byte places 2 t and 2 t + 1
            const int r = 32 * quarter + 8 * m + gr;
            const uint8_t *row = piece + r * 128;
            const uint4 lo = *reinterpret_cast<const uint4 *>(row + (((2 * t) ^ (r & 7)) << 4));
            const uint4 hi = *reinterpret_cast<const uint4 *>(row + (((2 * t + 1) ^ (r & 7)) << 4));
            Chunk c = {{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}};
            if (!copy) {
#pragma unroll
              for (int j = 0; j < COLS / 2; ++j) {
                const float d0 = v[m / 2][4 * j + 2 * (m & 1)], d1 = v[m / 2][4 * j + 2 * (m & 1) + 1];
                if (F32) {
                  c.w[(2 * j) % 8] = __float_as_uint(fmaf(f[m], d0, __uint_as_float(c.w[(2 * j) % 8])));
                  c.w[(2 * j + 1) % 8] = __float_as_uint(fmaf(f[m], d1, __uint_as_float(c.w[(2 * j + 1) % 8])));
                } else {
                  const float2 z = __half22float2(*reinterpret_cast<const __half2 *>(&c.w[j]));
                  const __half2 o = __floats2half2_rn(fmaf(f[m], d0, z.x), fmaf(f[m], d1, z.y));
                  c.w[j] = *reinterpret_cast<const uint32_t *>(&o);
                }
              }
            }
            if (rows[m] >= 0) store_chunk(dst + rows[m] * out_bytes + (nb * 128 + go * 32) * SIZE, c, wide);
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&y_empty[st]);
          const int step = go + 1 < GOES ? 1 : PIECES - GOES + 1;    // over the other half's pieces
          st += step;
          if (st >= g.y_stages) { st -= g.y_stages; phase ^= 1; }
        }
        if (!ok) break;
        if (!copy && ++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
    }
  }
  if (!ok) *failed = 1;
  tc::tc_fence_before();
  __syncthreads();
  if (*failed) {                                                    // leave no copy in flight behind
    if (threadIdx.x == 0) {
      set_device_error(a.err, kErrBounds);
      tc::drain(full, g.stages, used);
      tc::drain(h_full, 1, h_used);
    } else if (warp == 2 + kEpiWarps && lane == 0) {
      tc::drain(y_full, g.y_stages, used);
    }
  }
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kOutCols);
  }
}

}  // namespace ad
}  // namespace exl3

using namespace exl3;

namespace {

int map_rows(CUtensorMap *m, const void *base, int dims, const cuuint64_t *size, const cuuint64_t *stride,
             const cuuint32_t *box, bool f32) {
  auto fn = exl3_tmap_encode_fn();
  if (!fn) return exl3_fail(EXL3_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, dims,
                  const_cast<void *>(base), size, stride, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return exl3_fail(EXL3_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return EXL3_OK;
}

int map_f16(CUtensorMap *m, const void *base, int dims, const cuuint64_t *size, const cuuint64_t *stride,
            const cuuint32_t *box) {
  return map_rows(m, base, dims, size, stride, box, false);
}

template <int S>
int launch_clusters(const CUtensorMap &mx, const CUtensorMap &mt, const CUtensorMap &ma, const ad::InArgs &g,
                    size_t smem, cudaStream_t s) {
  auto kfn = ad::adapter_in_kernel<S>;
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
  cfg.blockDim = dim3(ad::kInThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return exl3_cuda_check(cudaLaunchKernelEx(&cfg, kfn, mx, mt, ma, g), "adapter launch");
}

int launch_in(const ad::Args &a, cudaStream_t s) {
  ad::InArgs g = {};
  g.a = a;
  g.r16 = (a.R + 15) / 16 * 16;
  const int stage = ad::kPanel + g.r16 * 128;
  // Three CTAs on an SM, two above rank 64: never more than TMEM has columns for
  // (a CTA that waited for TMEM while its cluster waits for it could wait for ever).
  // Few tiles leave a CTA an SM: as deep a ring as fits.
  const bool few = a.max_tiles <= exl3_sm_count() * 15 / 152;
  g.ring_bytes = (few ? 192 : a.R <= 64 ? 72 : 104) * 1024;
  g.stages = std::min(8, g.ring_bytes / stage);
  g.tmem_cols = 32;
  while ((int)g.tmem_cols < g.r16) g.tmem_cols *= 2;
  const size_t smem = 1024 + g.ring_bytes + 17 * 8 + 16;
  CUtensorMap mx, mt, ma;      // x for gathers of rows and for boxes; A
  {
    const cuuint64_t dims[2] = {(cuuint64_t)a.k, (cuuint64_t)a.T}, stride[1] = {(cuuint64_t)a.x_stride * 2};
    const cuuint32_t row[2] = {64, 1}, box[2] = {64, 32};
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
  // The largest split whose clusters all run at once (as for the router's product:
  // 15, 36 or 76 clusters of eight, four or two at one CTA per SM)
  const int sms = exl3_sm_count() * (a.R <= 64 ? 3 : 2);
  if (a.max_tiles <= sms * 15 / 152) return launch_clusters<8>(mx, mt, ma, g, smem, s);
  if (a.max_tiles <= sms * 36 / 152) return launch_clusters<4>(mx, mt, ma, g, smem, s);
  return launch_clusters<2>(mx, mt, ma, g, smem, s);
}

template <bool F32>
int launch_out(const ad::OutArgs &g, cudaStream_t s) {
  const ad::Args &a = g.a;
  CUtensorMap mh, mb, my, mr;
  {
    const cuuint64_t dims[3] = {(cuuint64_t)a.R, (cuuint64_t)a.T, 2};
    const cuuint64_t stride[2] = {(cuuint64_t)a.R * 2, (cuuint64_t)a.T * a.R * 2};
    const cuuint32_t box[3] = {64, 128, 1};
    int rc = map_f16(&mh, a.h, 3, dims, stride, box);
    if (rc) return rc;
  }
  {
    // fp16: column 16 t + 2 j + b of 64 goes to row 8 j + 2 t + b of the operand,
    // fp32: column 8 t + 2 j + b of 32 (32 bytes a lane either way)
    const cuuint64_t R = a.R, J = F32 ? 4 : 8;
    const cuuint64_t dims[5] = {R, 2, 4, J, (cuuint64_t)a.n / (8 * J) * a.N};
    const cuuint64_t stride[4] = {R * 2, R * 2 * J * 2, R * 4, R * 8 * J * 2};
    const cuuint32_t box[5] = {64, 2, 4, (cuuint32_t)J, F32 ? 4u : 2u};
    int rc = map_f16(&mb, a.b, 5, dims, stride, box);
    if (rc) return rc;
  }
  {
    const cuuint64_t dims[2] = {(cuuint64_t)a.n, (cuuint64_t)a.T}, stride[1] = {(cuuint64_t)a.y_stride * (F32 ? 4 : 2)};
    const cuuint32_t box[2] = {F32 ? 32u : 64u, 32}, row[2] = {F32 ? 32u : 64u, 1};
    int rc = map_rows(&my, a.y, 2, dims, stride, box, F32);
    if (rc) return rc;
    rc = map_rows(&mr, a.y, 2, dims, stride, row, F32);
    if (rc) return rc;
  }
  const size_t smem = ad::out_smem(g.panels, {g.stages, g.y_stages});
  auto kfn = ad::adapter_out_kernel<F32>;
  static std::atomic<size_t> given[kMaxDevices];
  int rc = exl3_cuda_check(exl3_ensure_smem(reinterpret_cast<const void *>(kfn), smem, given), "adapter attribute");
  if (rc) return rc;
  return exl3_cuda_check(launch_pdl(kfn, dim3(exl3_sm_count()), dim3(ad::kOutThreads), smem, s, mh, mb, my, mr, g),
                         "adapter launch");
}

}  // namespace

int exl3_launch_adapter_tc(const ad::Args &a, bool f32, cudaStream_t s) {
  int rc = launch_in(a, s);
  if (rc) return rc;
  ad::OutArgs g = {};
  g.a = a;
  g.panels = (a.R + 63) / 64;
  const ad::Rings r = ad::out_rings(g.panels, f32);
  g.stages = r.stages;
  g.y_stages = r.y_stages;
  g.wide = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && a.out_stride * (f32 ? 4 : 2) % 32 == 0;
  return f32 ? launch_out<true>(g, s) : launch_out<false>(g, s);
}
