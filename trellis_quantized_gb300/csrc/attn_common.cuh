// attn_common.cuh -- arguments and work division shared by the attention
// kernels (attn_step.cu, attn_tc.cu).
//
// A unit of work is (sequence, tile of new tokens, key head): its rows are
// those tokens times the G query heads of the key head, row r being token
// r / G and head r % G, so that all rows of a unit read the same keys and
// values.  A unit's keys are cut into blocks of KB; every unit has
// at least one block (a unit whose rows see nothing still has its zeros to
// write).  The blocks of all units, in order of (sequence, tile, key head),
// form one line (with a few places more for each unit's start and end) that
// the CTAs share in equal runs: no host knowledge of the lengths, no idle CTA
// behind a long sequence.  A unit cut by a run's border leaves one partial
// result per CTA in the workspace, which a second kernel joins in the order of
// the line (attn_join.cu).
#pragma once

#include "exl3_common.cuh"

namespace exl3 {
namespace attn {

struct Args {
  const __half *q;
  int64_t q_stride;          // elements between tokens
  int T, Hq, Hkv, G;
  unsigned g_inv;            // ceil(2^32 / G), G > 1: r / G for a unit's rows
  int unit_tok;              // tokens of a unit
  int tile_tok;              // tokens of one of its row tiles (attn_tc)
  const int *q_start, *kv_len, *table;
  int B, max_pages, page_size, num_pages;
  int box_log2;              // tokens of one TMA copy: the largest power of two in page_size, at most a block's
  int head_first;            // tensor map order: (d, head, token, page), else (d, token, head, page)
  float scale_log2;          // scale * log2(e)
  int causal, window;        // window 0: none
  void *y;                   // [T][Hq][D]
  int f32out, y_aligned32;
  float *lse;                // [T][Hq] or null
  float *part_o;             // partial results: [grid][2][rows][D] fp32
  float2 *part_ml;           // [grid][2][rows]: maximum of the scaled scores (log2), sum of 2^(score - maximum)
  struct Cut *cuts;          // [grid] the unit that begins in a CTA and ends in a later one
  int *err;
};

// A unit in parts: its first part is slot 1 of the CTA that the record
// belongs to, the others slot 0 of the CTAs up to `last`.
struct __align__(16) Cut {
  int rows;                  // 0: no such unit
  int last;
  int t, h;                  // first token (row of the call) and key head
};
static_assert(sizeof(Cut) == 16, "read as one int4");

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

// r / G for a row of a unit (r < 2^16).
__device__ __forceinline__ int row_token(const Args &a, int r) {
  return a.G == 1 ? r : (int)__umulhi((unsigned)r, a.g_inv);
}

// Keys [lo, hi) that the tokens i0 .. i0 + n - 1 of a sequence see between
// them.
__device__ __forceinline__ void token_range(const Args &a, const Seq &s, int i0, int n, int &lo, int &hi) {
  const int p0 = s.len - s.nq + i0, p1 = p0 + n - 1;   // cache indexes
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

// ln of the sum of weights, from their maximum (log2) and the sum of 2^(score -
// maximum).
__device__ __forceinline__ float natural_lse(float m2, float l) {
  return l == 0.0f ? neg_inf() : (m2 + log2f(l)) * 0.69314718055994530942f;
}

// Four neighbouring elements of the output, rounded once if it is fp16.
__device__ __forceinline__ void store4(const Args &a, int64_t i, const float4 &v) {
  if (a.f32out) {
    *reinterpret_cast<float4 *>(static_cast<float *>(a.y) + i) = v;
  } else {
    __half2 h[2] = {__floats2half2_rn(v.x, v.y), __floats2half2_rn(v.z, v.w)};
    *reinterpret_cast<uint2 *>(static_cast<__half *>(a.y) + i) = *reinterpret_cast<uint2 *>(h);
  }
}

// Output row (token, query head) of row r of a unit whose first token is row
// t of the call.
__device__ __forceinline__ int64_t out_head(const Args &a, int t, int h, int r) {
  const int tok = row_token(a, r);
  return (int64_t)(t + tok) * a.Hq + h * a.G + r - tok * a.G;
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

template <int KB>
__device__ __forceinline__ int range_blocks(int lo, int hi) {
  return lo >= hi ? 1 : (hi + KB - 1) / KB - lo / KB;
}

// The work of one unit on the line: its blocks, and OV more for its start
// and end (reading q, joining and writing y), during which no block is done.
template <int KB, int OV>
__device__ __forceinline__ int tile_cost(const Args &a, const Seq &s, int i0) {
  int lo, hi;
  token_range(a, s, i0, min(a.unit_tok, s.nq - i0), lo, hi);
  return range_blocks<KB>(lo, hi) + OV;
}

// What every CTA works out for itself at its start.
struct Share {
  long long total;     // length of the line
  long long per;       // each CTA's part of it
  int b, i0;           // tile that holds the CTA's first place (b = B: none)
  int off;             // that place within the tile's units
};

// The costs of up to 32 sequences, lane i that of sequence b + i (0 past
// `end`).  Sequences of many tiles are summed by the whole warp.
template <int KB, int OV>
__device__ long long warp_costs(const Args &a, int b, int end, bool report, Seq &s) {
  const int lane = threadIdx.x & 31;
  s = Seq{0, 0, 0};
  if (b + lane < end) s = load_seq(a, b + lane, report);
  const bool many = s.nq > 4 * a.unit_tok;
  long long n = 0;
  if (!many)
    for (int i0 = 0; i0 < s.nq; i0 += a.unit_tok) n += tile_cost<KB, OV>(a, s, i0);
  unsigned todo = __ballot_sync(0xffffffffu, many);
  while (todo) {
    const int i = __ffs(todo) - 1;
    todo &= todo - 1;
    const Seq q = {__shfl_sync(0xffffffffu, s.t0, i), __shfl_sync(0xffffffffu, s.nq, i),
                   __shfl_sync(0xffffffffu, s.len, i)};
    long long c = 0;
    for (int i0 = lane * a.unit_tok; i0 < q.nq; i0 += 32 * a.unit_tok) c += tile_cost<KB, OV>(a, q, i0);
#pragma unroll
    for (int d = 16; d; d >>= 1) c += __shfl_xor_sync(0xffffffffu, c, d);
    if (lane == i) n = c;
  }
  return n * a.Hkv;
}

__device__ __forceinline__ long long warp_scan(long long v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// The tile that holds place `start`, searched by a whole warp from sequence b
// on (whose units begin at place `at`); false if it is not below `end`.  `n`
// and `s`: the costs and sequences b .. b + 31, if the caller has them.
template <int KB, int OV>
__device__ __forceinline__ bool find_tile(const Args &a, int b, int end, long long at, long long start, long long n,
                                          Seq s, bool known, Share &out) {
  const int lane = threadIdx.x & 31;
  for (; b < end; b += 32) {
    if (!known) n = warp_costs<KB, OV>(a, b, end, false, s);
    known = false;
    const long long inc = at + warp_scan(n);
    const unsigned hit = __ballot_sync(0xffffffffu, start < inc && start >= inc - n);
    at = __shfl_sync(0xffffffffu, inc, 31);
    if (!hit) continue;
    const int i = __ffs(hit) - 1;
    const Seq q = {0, __shfl_sync(0xffffffffu, s.nq, i), __shfl_sync(0xffffffffu, s.len, i)};
    long long tile_at = __shfl_sync(0xffffffffu, inc - n, i);
    for (int g0 = 0; g0 < q.nq; g0 += 32 * a.unit_tok) {
      const int i0 = g0 + lane * a.unit_tok;
      const long long c = i0 < q.nq ? (long long)tile_cost<KB, OV>(a, q, i0) * a.Hkv : 0;
      const long long e = tile_at + warp_scan(c);
      const unsigned tile = __ballot_sync(0xffffffffu, start < e && start >= e - c);
      if (tile) {
        const int k = __ffs(tile) - 1;
        out.b = b + i;
        out.i0 = g0 + k * a.unit_tok;
        out.off = __shfl_sync(0xffffffffu, (int)(start - (e - c)), k);
        return true;
      }
      tile_at = __shfl_sync(0xffffffffu, e, 31);
    }
    return false;
  }
  return false;
}

// Cuts the line into the CTAs' parts and finds this CTA's first tile.  Up to
// 32 sequences: every warp works it out for itself, without a barrier (code
// that all warps share; the start of a launch waits for its instructions).
// More: each warp sums a run of sequences, the warp whose run holds the place
// looks for it.  `sums` has NT / 32 entries.  CTA 0 also reports lengths that
// contradict one another.
template <int KB, int OV, int NT>
__device__ __forceinline__ Share make_share(const Args &a, int min_per, Share *shared, long long *sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int NW = NT / 32;
  const bool few = a.B <= 32;
  const int chunk = few ? 32 : (a.B + NW - 1) / NW;
  const int b0 = few ? 0 : min(a.B, warp * chunk), b1 = min(a.B, b0 + chunk);
  long long n = 0, mine = 0;
  Seq s = {0, 0, 0};
  for (int b = b0; b < b1; b += 32) {
    n = warp_costs<KB, OV>(a, b, b1, blockIdx.x == 0 && (!few || warp == 0), s);
    mine += n;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, d);
  long long before = 0;
  Share out;
  out.total = mine;
  if (!few) {
    if (lane == 0) sums[warp] = mine;
    if (threadIdx.x == 0) shared->b = a.B;
    __syncthreads();
    out.total = 0;
    for (int w = 0; w < NW; ++w) {
      if (w < warp) before += sums[w];
      out.total += sums[w];
    }
  }
  const long long up = out.total + gridDim.x - 1;
  out.per = up >> 31 ? up / gridDim.x : (long long)((unsigned)up / gridDim.x);
  if (out.per < min_per) out.per = min_per;
  const long long start = out.per * blockIdx.x;
  out.b = a.B;
  out.i0 = out.off = 0;
  bool found = false;
  if (start >= before && start < before + mine) found = find_tile<KB, OV>(a, b0, b1, before, start, n, s, chunk <= 32, out);
  if (!few) {
    if (found && lane == 0) *shared = out;
    __syncthreads();
    const int b = shared->b;
    if (b < a.B) {
      out.b = b;
      out.i0 = shared->i0;
      out.off = shared->off;
    }
  }
  return out;
}

// One CTA's part of the line, unit by unit: tokens i0 .. i0 + ntok - 1 of
// sequence b (`rows` rows) against key head h, blocks blk .. blk + nseg - 1 of
// the nblk blocks that hold keys [lo, hi).
template <int KB, int OV>
struct Walk {
  int b, i0, ntok, rows, h;
  int lo, hi, nblk;
  int blk, nseg;
  Seq s;
  long long at;        // place of the unit on the line
  int x;               // first place within the unit
  int left;            // places left, this unit's included

  __device__ __forceinline__ void set_tile(const Args &a) {
    ntok = min(a.unit_tok, s.nq - i0);
    rows = ntok * a.G;
    token_range(a, s, i0, ntok, lo, hi);
    nblk = range_blocks<KB>(lo, hi);
  }

  // The unit's places from OV on are its blocks.
  __device__ __forceinline__ void set_segment() {
    const int end = min(nblk + OV, x + left);
    blk = max(0, x - OV);
    nseg = max(0, end - OV) - blk;
    if (nseg <= 0) left = 0;           // (only places without blocks: the next CTA has the unit)
  }

  __device__ __forceinline__ void begin(const Args &a, const Share &sh) {
    left = 0;
    const long long start = sh.per * blockIdx.x;
    if (start >= sh.total || sh.b >= a.B) return;
    left = (int)min(sh.per, sh.total - start);
    b = sh.b;
    i0 = sh.i0;
    s = load_seq(a, b, false);
    set_tile(a);
    h = sh.off / (nblk + OV);
    x = sh.off - h * (nblk + OV);
    at = start - x;
    set_segment();
  }

  __device__ __forceinline__ void next(const Args &a) {
    const int used = min(nblk + OV, x + left) - x;
    left -= used;
    if (left <= 0) return;
    at += nblk + OV;
    x = 0;
    if (++h >= a.Hkv) {
      h = 0;
      i0 += a.unit_tok;
      while (i0 >= s.nq) {
        i0 = 0;
        if (++b >= a.B) {
          left = 0;
          return;
        }
        s = load_seq(a, b, false);
      }
      set_tile(a);
    }
    set_segment();
  }

  __device__ __forceinline__ bool whole() const { return nseg == nblk; }
  // Where a part goes: a unit's first part to slot 1, one that continues a
  // unit (at most one per CTA, its first) to slot 0.
  __device__ __forceinline__ int slot() const { return blk == 0 ? 1 : 0; }
  // The record of the unit that this CTA leaves unfinished.
  __device__ __forceinline__ Cut cut(const Share &sh) const {
    return Cut{rows, (int)((at + OV + nblk - 1) / sh.per), s.t0 + i0, h};
  }
};

// The pages of a unit's blocks, followed block by block by a warp whose lane i
// looks up box i of the block (the division is left to the start of a unit).
template <int KB>
struct PageWalk {
  int64_t row;       // the sequence's first entry in the page table
  int lo, hi;        // keys that are looked at
  int key, index, off;

  template <class W>
  __device__ __forceinline__ void begin(const Args &a, const W &w) {
    row = (int64_t)w.b * a.max_pages;
    lo = w.lo;
    hi = w.hi;
    key = (w.lo / KB + w.blk) * KB + ((int)(threadIdx.x & 31) << a.box_log2);
    index = key / a.page_size;
    off = key - index * a.page_size;
  }
  // This block's page (-1: not needed) and the offset in it; on to the next.
  __device__ __forceinline__ void next(const Args &a, int &page, int &offset) {
    page = -1;
    offset = off;
    const int lane = threadIdx.x & 31;
    if (lane < (KB >> a.box_log2) && key + (1 << a.box_log2) > lo && key < hi) page = __ldg(a.table + row + index);
    key += KB;
    off += KB;
    while (off >= a.page_size) {
      off -= a.page_size;
      ++index;
    }
  }
};

}  // namespace attn
}  // namespace exl3
