// adapter.cuh -- arguments and the plan's layout shared by the adapter kernels
// (adapter_plan.cu, adapter_step.cu, adapter_tc.cu).
#pragma once

#include <algorithm>

#include "exl3_common.cuh"

namespace exl3 {
namespace ad {

constexpr int kStepRows = 16;      // rows of a tile: few tokens
constexpr int kTcRows = 128;       // rows of a tile: tensor-core kernel
constexpr int kMaxRank = 128;
constexpr int kMaxCount = 4096;    // adapters of a plan

// Words of a plan's control block (offset 0, 256 bytes; the error word first):
// tiles of both sizes, the large tiles' cost, then what the plan was made for.
constexpr int kPlanErr = 0, kPlanStepTiles = 1, kPlanTcTiles = 2, kPlanCost = 3, kPlanT = 4, kPlanB = 5, kPlanN = 6;
// A large tile's cost per column block, in rows, besides its rows: a block of B
// and a product are taken whatever the rows.
constexpr int kTileCost = 96;

// A plan: control block, each sequence's place in the order, the rows in the
// order of their adapters (rows without one last), and the tiles of both sizes
// (adapter or -1, first place, rows, cost of the tiles before it).  Only what is known on the host goes
// into the sizes.
struct PlanLayout {
  size_t base, perm, step_tiles, tc_tiles, total;
  int max_step_tiles, max_tc_tiles;
};

inline PlanLayout plan_layout(int T, int batch, int count) {
  PlanLayout p;
  const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  // every adapter in use, and the rows without one, end in at most one part-filled tile
  const int64_t used = std::min({(int64_t)count, (int64_t)batch, (int64_t)T}) + 1;
  p.max_step_tiles = (int)std::min<int64_t>(T, T / kStepRows + used);
  p.max_tc_tiles = (int)std::min<int64_t>(T, T / kTcRows + used);
  p.base = 256;
  p.perm = up(p.base + (size_t)batch * 4);
  p.step_tiles = up(p.perm + (size_t)T * 4);
  p.tc_tiles = up(p.step_tiles + (size_t)p.max_step_tiles * 16);
  p.total = up(p.tc_tiles + (size_t)p.max_tc_tiles * 16);
  return p;
}

struct PlanArgs {
  const int32_t *q_start, *adapter;    // [B + 1], [B]
  int T, B, N;
  int *ctrl, *base, *perm;
  int4 *step_tiles, *tc_tiles;
  int max_step_tiles, max_tc_tiles;
};

struct Args {
  const __half *x;                     // [T][k]
  const void *y;                       // [T][n] fp16 or fp32
  void *out;
  int64_t x_stride, y_stride, out_stride;
  const __half *a, *b;                 // [N][R][k], [N][n][R]
  const float *scale;                  // [N]
  const int32_t *rank;                 // [N] or null: all R
  int N, R, k, n, T;
  int B;
  const int *ctrl;                     // the plan's control block
  const int *perm;
  const int4 *tiles;
  int max_tiles;
  int *err;
  // tensor cores: h of the rows in the plan's order, two parts, and scale 2^-p
  __half *h;                           // [2][T][R]
  float *back;                         // [T]
};

// Tiles of a plan (word `which` of its control block); none, and an error, if
// it was made for another call.
__device__ __forceinline__ int plan_tiles(const Args &a, int which) {
  const int4 made = *reinterpret_cast<const int4 *>(a.ctrl + kPlanT);
  const int tiles = a.ctrl[which];
  if (made.x == a.T && made.y == a.B && made.z == a.N) return min(tiles, a.max_tiles);
  if (threadIdx.x == 0) set_device_error(a.err, kErrBounds);
  return 0;
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;\n" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;\n" ::: "memory"); }

// A shared-memory address of this CTA as CTA `rank` of the cluster sees its own.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_cluster4(uint32_t addr, const float4 &v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// An adapter's rank, held to the pool's.
__device__ __forceinline__ int adapter_rank(const Args &a, int id) {
  return a.rank ? min(max(__ldg(a.rank + id), 0), a.R) : a.R;
}

// Rows without an adapter: out = y (if they are two buffers).
template <bool F32>
__device__ __forceinline__ void copy_rows(const Args &a, const int4 &tile, int split, int S, int threads) {
  if (a.out == a.y) return;
  constexpr int PER = F32 ? 4 : 8, SIZE = F32 ? 4 : 2;
  const int quads = a.n / PER;
  for (int r = 0; r < tile.z; ++r) {
    const int64_t row = a.perm[tile.y + r];
    const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const char *>(a.y) + row * a.y_stride * SIZE);
    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<char *>(a.out) + row * a.out_stride * SIZE);
    for (int i = split * threads + threadIdx.x; i < quads; i += S * threads) dst[i] = src[i];
  }
}

// The power of two that brings a row's largest |h| into [2^14, 2^15), as its
// exponent; 0 for a row of zeros or one with infinities or NaN.
__device__ __forceinline__ int row_exponent(float top) {
  if (!(top > 0.0f) || !isfinite(top)) return 0;
  return min(14 - ilogbf(top), 126);
}

// z (an h times its row's power of two) as hi + lo.  `far`: the row's largest is
// infinite; its infinities and NaN decide every output then, so the finite ones,
// which may lie above fp16's range, become zeros, and nothing is left for lo.
__device__ __forceinline__ void split_h(float z, bool far, __half &hi, __half &lo) {
  if (far && isfinite(z)) z = 0.0f;
  hi = __float2half_rn(z);
  lo = __float2half_rn(far ? 0.0f : z - __half2float(hi));
}

}  // namespace ad
}  // namespace exl3
