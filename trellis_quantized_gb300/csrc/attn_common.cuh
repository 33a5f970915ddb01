// attn_common.cuh -- arguments and work division shared by the attention
// kernels (attn_step.cu, attn_tc.cu).
//
// A unit of work is (sequence, row tile, key head): the rows of a tile are
// the sequence's new tokens times the G query heads of one key head, row r
// being token r / G and head r % G, so that all rows of a unit read the same
// keys and values.  A unit's keys are cut into blocks of KB; every unit has
// at least one block (a unit whose rows see nothing still has its zeros to
// write).  The blocks of all units, in order of (sequence, tile, key head),
// form one line that the CTAs share in equal runs: no host knowledge of the
// lengths, no idle CTA behind a long sequence.  A unit cut by a run's border
// leaves one partial result per CTA in the workspace and the CTA that
// arrives last adds them in the order of the line.
#pragma once

#include "exl3_common.cuh"

namespace exl3 {
namespace attn {

struct Args {
  const __half *q;
  int64_t q_stride;          // elements between tokens
  int T, Hq, Hkv, G;
  const int *q_start, *kv_len, *table;
  int B, max_pages, page_size, num_pages;
  int box;                   // rows of one TMA copy: gcd(page_size, KB)
  int head_first;            // tensor map order: (d, head, token, page), else (d, token, head, page)
  float scale_log2;          // scale * log2(e)
  int causal, window;        // window 0: none
  void *y;                   // [T][Hq][D]
  int f32out;
  float *lse;                // [T][Hq] or null
  float *part_o;             // partial results: [grid][2][rows][D] fp32
  float *part_lse;           // [grid][2][rows], log2 of the sum
  int *counters;             // [grid] arrival counters, zero between calls
  int *err;
};

// One sequence: first row, new tokens, tokens in the cache.
struct Seq {
  int t0, nq, len;
};

__device__ __forceinline__ Seq load_seq(const Args &a, int b, bool report) {
  const int s0 = __ldg(a.q_start + b), s1 = __ldg(a.q_start + b + 1), l = __ldg(a.kv_len + b);
  const int cap = a.max_pages * a.page_size;
  Seq s;
  s.t0 = min(max(s0, 0), a.T);
  const int e = min(max(s1, s.t0), a.T);
  s.nq = e - s.t0;
  s.len = min(max(l, 0), cap);
  if (report && (s.t0 != s0 || e != s1 || s.len != l || s.len < s.nq)) set_device_error(a.err, kErrBounds);
  return s;
}

// Keys [lo, hi) that rows r0 .. r0 + rows - 1 of a sequence see between them.
__device__ __forceinline__ void tile_range(const Args &a, const Seq &s, int r0, int rows, int &lo, int &hi) {
  const int base = s.len - s.nq;                       // cache index of the sequence's first new token
  const int p0 = base + r0 / a.G, p1 = base + (r0 + rows - 1) / a.G;
  hi = a.causal ? min(max(p1 + 1, 0), s.len) : s.len;
  lo = a.window ? max(0, max(p0, 0) - a.window + 1) : 0;
  if (lo > hi) lo = hi;
}

// exp2 by the hardware's approximation (2 ulp; subnormal results are zero).
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float neg_inf() { return __int_as_float((int)0xff800000u); }

// Four neighbouring elements of the output, rounded once if it is fp16.
__device__ __forceinline__ void store4(const Args &a, int64_t i, const float4 &v) {
  if (a.f32out) {
    *reinterpret_cast<float4 *>(static_cast<float *>(a.y) + i) = v;
  } else {
    __half2 h[2] = {__floats2half2_rn(v.x, v.y), __floats2half2_rn(v.z, v.w)};
    *reinterpret_cast<uint2 *>(static_cast<__half *>(a.y) + i) = *reinterpret_cast<uint2 *>(h);
  }
}

// Rows of the call that belong to no sequence: y = 0, lse = -infinity.
template <int D>
__device__ __forceinline__ void clear_padding(const Args &a, int nthreads) {
  const int first = min(max(__ldg(a.q_start), 0), a.T), end = min(max(__ldg(a.q_start + a.B), first), a.T);
  const int n = first + a.T - end;
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int64_t t = i < first ? i : end + (i - first);
    const int bytes = a.f32out ? 4 : 2;
    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<char *>(a.y) + t * a.Hq * D * bytes);
    for (int j = threadIdx.x; j < a.Hq * D * bytes / 16; j += nthreads) dst[j] = make_uint4(0, 0, 0, 0);
    if (a.lse)
      for (int j = threadIdx.x; j < a.Hq; j += nthreads) a.lse[t * a.Hq + j] = neg_inf();
  }
}

// Keys [lo, hi) that row r sees.
__device__ __forceinline__ void row_range(const Args &a, const Seq &s, int r, int &lo, int &hi) {
  const int p = s.len - s.nq + r / a.G;
  hi = a.causal ? min(max(p + 1, 0), s.len) : s.len;
  lo = a.window ? max(0, max(p, 0) - a.window + 1) : 0;
  if (lo > hi) lo = hi;
}

template <int KB>
__device__ __forceinline__ int range_blocks(int lo, int hi) {
  return lo >= hi ? 1 : (hi + KB - 1) / KB - lo / KB;
}

// Blocks of one sequence in the line.
template <int ROWS, int KB>
__device__ long long seq_blocks(const Args &a, const Seq &s) {
  const int rows = s.nq * a.G;
  long long n = 0;
  for (int r0 = 0; r0 < rows; r0 += ROWS) {
    int lo, hi;
    tile_range(a, s, r0, min(ROWS, rows - r0), lo, hi);
    n += range_blocks<KB>(lo, hi);
  }
  return n * a.Hkv;
}

// A place in the line: block `blk` of the unit (b, tile at r0, head h).
struct Walk {
  int b, r0, rows, h;
  int lo, hi;          // keys of the unit
  int nblk;            // its blocks
  Seq s;

  template <int ROWS, int KB>
  __device__ __forceinline__ void set_tile(const Args &a) {
    rows = min(ROWS, s.nq * a.G - r0);
    tile_range(a, s, r0, rows, lo, hi);
    nblk = range_blocks<KB>(lo, hi);
  }

  // The unit after this one (the caller knows that there is one).
  template <int ROWS, int KB>
  __device__ __forceinline__ void next(const Args &a) {
    if (++h < a.Hkv) return;
    h = 0;
    r0 += ROWS;
    while (r0 >= s.nq * a.G) {
      r0 = 0;
      if (++b >= a.B) {
        rows = 0;
        return;
      }
      s = load_seq(a, b, false);
    }
    set_tile<ROWS, KB>(a);
  }
};

// What every CTA works out for itself at its start.
struct Share {
  long long total;     // blocks in the line
  long long per;       // blocks per CTA
  int b;               // sequence that holds the CTA's first block
  long long off;       // that block's index within the sequence's blocks
};

// Scan of the sequences' block counts by the whole CTA; `sh` needs
// NT / 32 + 1 entries and a Share of its own.  CTA 0 also reports lengths
// that contradict one another.
template <int ROWS, int KB, int NT>
__device__ void make_share(const Args &a, int min_per, Share *out, long long *warp_sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int NW = NT / 32;
  const int chunk = (a.B + NT - 1) / NT;
  const int b0 = min(a.B, tid * chunk), b1 = min(a.B, b0 + chunk);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += seq_blocks<ROWS, KB>(a, load_seq(a, b, blockIdx.x == 0));
  long long inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
  }
  long long per = (total + gridDim.x - 1) / gridDim.x;
  if (per < min_per) per = min_per;
  const long long start = per * blockIdx.x;
  long long ex = before + inc - mine;
  if (tid == 0) {
    out->total = total;
    out->per = per;
    out->b = a.B;
  }
  __syncthreads();
  if (start < total && start >= ex && start < ex + mine) {
    for (int b = b0; b < b1; ++b) {
      const long long n = seq_blocks<ROWS, KB>(a, load_seq(a, b, false));
      if (start < ex + n) {
        out->b = b;
        out->off = start - ex;
        break;
      }
      ex += n;
    }
  }
  __syncthreads();
}

// The unit that holds block `off` of sequence w.b; *blk: the block within it.
template <int ROWS, int KB>
__device__ void seek(const Args &a, Walk &w, int b, long long off, int *blk) {
  w.b = b;
  w.h = 0;
  w.r0 = 0;
  w.s = load_seq(a, b, false);
  w.set_tile<ROWS, KB>(a);
  while (off >= (long long)w.nblk * a.Hkv && w.r0 + ROWS < w.s.nq * a.G) {
    off -= (long long)w.nblk * a.Hkv;
    w.r0 += ROWS;
    w.set_tile<ROWS, KB>(a);
  }
  w.h = (int)(off / w.nblk);
  *blk = (int)(off % w.nblk);
}

}  // namespace attn
}  // namespace exl3
