// attn_step.cu -- attention of few rows over a paged cache (decode steps and
// short verifications): at most 16 rows (tokens x query heads of one key
// head) share a pass over their keys and values.
//
//   s_ij = scale q_i . k_j,  m = running max, l = running sum of exp(s - m),
//   o <- o exp(m_old - m) + exp(s - m) v,  y = o / l
//
// Bound by memory: every live key and value is read once (4 D bytes per token
// and key head) against 4 D flops per row.  So the pass is built around the
// reads: one warp keeps a ring of TMA copies in flight (64 tokens of K and V
// per stage, pages looked up one block ahead), four warps each take 16 of a
// block's keys with a softmax of their own, and nothing in the loop makes
// the warps wait for one another; they are joined once per unit.  The
// products run on mma.sync (16 rows x 8 keys, and 16 rows x 8 elements of v):
// the tcgen05 instructions need 64 or 128 rows of which a step would fill 5
// or 8, and at one 16 x 8 x 16 product per 256 bytes of cache the legacy path
// has 5x the rate that the memory can feed.  P moves from accumulator to
// operand registers without leaving the thread.
//
// Measured (40 query on 8 key heads of 128): one sequence of 131,001 tokens,
// 537 MB, 87 to 89 us with the join, 83 without; 64 sequences of up to 8,000
// tokens, 875 MB, 143 to 148 us and 135.  Two CTAs on an SM with three stages each have 192 KB
// of loads in flight; what is left to the memory's rate is the start (lengths,
// pages, the first bytes) and the end of the longest part.
#include <cudaTypedefs.h>

#include "attn_common.cuh"
#include "tc_ptx.cuh"

int exl3_attn_step_grid(int D);

namespace exl3 {
namespace attn {

constexpr int kStepRows = 16, kStepKeys = 64;
constexpr int kStepCost = 1;            // a unit's start and end, in blocks
// Weights are 2^kStepTop at the maximum (off again in the sum that leaves the
// kernel): fp16 then holds those down to 2^-29 of the largest in full and the
// rest to 2^-40 of it, which counts where one key outweighs a long history.
constexpr float kStepTop = 15.0f;
constexpr int kStepThreads = 160;       // four consumer warps and the producer

template <int D>
struct StepCfg {
  static constexpr int STAGES = 3;
  static constexpr int CTAS = D == 64 ? 3 : D == 128 ? 2 : 1;      // per SM
  static constexpr int PANEL = kStepKeys * 128;                    // 64 columns of a block
  static constexpr int OPERAND = kStepKeys * D * 2;                // K or V of a block
  static constexpr int STAGE = 2 * OPERAND;
  static constexpr int QPITCH = D + 8;                             // halves; rows 16 bytes apart in banks
  static constexpr int MPITCH = D + 8;                             // floats
  static constexpr int OFF_Q = STAGES * STAGE;
  static constexpr int OFF_M = OFF_Q + kStepRows * QPITCH * 2;
  static constexpr int SMEM = OFF_M + 2 * 8 * MPITCH * 4 + 1024 /*alignment*/;
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_half2(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// 4-D tiled TMA load (innermost coordinate first).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *m, uint64_t *bar, int x, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(tc::smem_u32(bar)), "r"(x), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

template <int D>
__global__ void __launch_bounds__(kStepThreads, StepCfg<D>::CTAS)
    attn_step_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Args a) {
  using C = StepCfg<D>;
  constexpr int ST = C::STAGES, NP = D / 64;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[ST], empty[ST];
  __shared__ Share share_mem;
  __shared__ long long warp_sums[kStepThreads / 32];
  __shared__ float sm_m[4][kStepRows], sm_l[4][kStepRows];
  __shared__ int abort_word;
  const uint32_t raw = tc::smem_u32(smem_raw);
  uint8_t *smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const uint32_t sbase = tc::smem_u32(smem);
  volatile int *abort_flag = &abort_word;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < ST; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 4);
    }
    abort_word = 0;
    tc::fence_mbar_init();
    tc::prefetch_tmap(&tmK);
    tc::prefetch_tmap(&tmV);
  }
  __syncthreads();
  pdl_trigger();
  pdl_wait();
  const Share share = make_share<kStepKeys, kStepCost, kStepThreads>(a, 1 + kStepCost, &share_mem, warp_sums);
  clear_padding<D>(a, kStepThreads);
  Walk<kStepKeys, kStepCost> w;
  w.begin(a, share);
  if (tid == 0) {
    a.cuts[blockIdx.x].rows = 0;           // (the thread that may fill the record in below)
    share_mem = share;                     // (out of the registers; who still reads it, reads the same)
  }

  if (warp == 4) {
    // ------------------------------------------------------------ producer
    // the pages of a block's boxes, lane i box i (at most 4), looked up while
    // the block before is under way
    int it = 0;
    bool stop = false;
    int page = -1, off = 0;
    PageWalk<kStepKeys> pages;
    if (w.left > 0) {
      pages.begin(a, w);
      pages.next(a, page, off);
    }
    while (w.left > 0 && !stop) {
      auto ahead = w;
      ahead.next(a);
      for (int i = 0; i < w.nseg; ++i, ++it) {
        const int key0 = (w.lo / kStepKeys + w.blk + i) * kStepKeys;
        const int k_lo = max(w.lo, key0), k_hi = min(w.hi, key0 + kStepKeys), box = 1 << a.box_log2;
        const int box0 = (k_lo - key0) >> a.box_log2;
        const int nbox = k_hi > k_lo ? ((k_hi - key0 + box - 1) >> a.box_log2) - box0 : 0;
        // one copy per lane: (box, panel, K or V); at most 4 boxes x 4 panels x 2
        const bool mine = lane < nbox * NP * 2;
        const int bx = box0 + lane / (NP * 2), panel = (lane >> 1) % NP, isv = lane & 1;
        int my_page = __shfl_sync(0xffffffffu, page, bx & 31);
        const int my_off = __shfl_sync(0xffffffffu, off, bx & 31);
        if (mine && (unsigned)my_page >= (unsigned)a.num_pages) {
          set_device_error(a.err, kErrBounds);
          my_page = a.num_pages;             // past the map's end: reads as zeros
        }
        if (i + 1 < w.nseg) {
          pages.next(a, page, off);
        } else if (ahead.left > 0) {
          pages.begin(a, ahead);
          pages.next(a, page, off);
        }
        const int s = it % ST;
        if (it >= ST) {
          const bool ok = __all_sync(0xffffffffu, tc::mbar_wait(&empty[s], ((it / ST) & 1) ^ 1));
          if (!ok || *abort_flag) {
            if (lane == 0 && !ok) set_device_error(a.err, kErrBounds);
            *abort_flag = 1;
            stop = true;
            break;
          }
        }
        if (lane == 0) {
          const uint32_t bytes = (uint32_t)((nbox << a.box_log2) * 128 * NP * 2);
          if (bytes) tc::mbar_arrive_expect_tx(&full[s], bytes);
          else tc::mbar_arrive(&full[s]);
        }
        __syncwarp();
        if (mine) {
          const uint32_t dst = sbase + s * C::STAGE + isv * C::OPERAND + panel * C::PANEL + (bx << a.box_log2) * 128;
          if (a.head_first) tma_load_4d(dst, isv ? &tmV : &tmK, &full[s], panel * 64, w.h, my_off, my_page);
          else tma_load_4d(dst, isv ? &tmV : &tmK, &full[s], panel * 64, my_off, w.h, my_page);
        }
        __syncwarp();
      }
      w = ahead;
    }
    if (stop) {                            // leave no copy in flight behind
      for (int j = max(0, it - ST); j < it; ++j) tc::mbar_wait(&full[j % ST], (j / ST) & 1);
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  __half *sq = reinterpret_cast<__half *>(smem + C::OFF_Q);
  float *mb = reinterpret_cast<float *>(smem + C::OFF_M);
  const uint32_t sq_addr = tc::smem_u32(sq);
  const int q4 = lane & 3, rl = lane >> 2;
  // ldmatrix lanes: K as (keys 0-7 | 8-15) x (two 16-byte chunks), V as
  // (keys 0-7, keys 8-15) x (two chunks), Q as (rows 0-7, rows 8-15) x chunks
  const int kkey = warp * 16 + ((lane >> 4) & 1) * 8 + (lane & 7), kchunk = (lane >> 3) & 1;
  const int vkey = warp * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), vchunk = (lane >> 4) & 1;
  const uint32_t kbase = kkey * 128, vbase = vkey * 128;
  const uint32_t qbase = sq_addr + (((lane >> 3) & 1) * 8 + (lane & 7)) * C::QPITCH * 2 + ((lane >> 4) & 1) * 16;
  int it = 0;
  for (; w.left > 0; w.next(a)) {
    const bool whole = w.whole();
    // ---- the unit's rows of q (rows past the unit's are zero)
    for (int i = tid; i < kStepRows * (D / 8); i += 128) {
      const int r = i / (D / 8), c8 = i % (D / 8);
      uint4 u = make_uint4(0, 0, 0, 0);
      if (r < w.rows) {
        const int tok = row_token(a, r);
        u = *reinterpret_cast<const uint4 *>(a.q + (int64_t)(w.s.t0 + w.i0 + tok) * a.q_stride +
                                             (int64_t)(w.h * a.G + r - tok * a.G) * D + c8 * 8);
      }
      *reinterpret_cast<uint4 *>(sq + r * C::QPITCH + c8 * 8) = u;
    }
    consumer_sync();
    constexpr bool QREG = D <= 128;        // 256-wide heads read q from shared memory in every block
    uint32_t qf[QREG ? D / 16 : 1][4];
    if constexpr (QREG) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) ldmatrix4(qbase + k * 32, qf[k]);
    }
    const bool two = w.rows > 8;
    int lo0 = 0, hi0 = 0, lo1 = 0, hi1 = 0;
    if (rl < w.rows) token_range(a, w.s, w.i0 + row_token(a, rl), 1, lo0, hi0);
    if (rl + 8 < w.rows) token_range(a, w.s, w.i0 + row_token(a, rl + 8), 1, lo1, hi1);
    // keys that every row sees need no mask
    int all_lo, all_hi, tmp;
    token_range(a, w.s, w.i0, 1, tmp, all_hi);
    token_range(a, w.s, w.i0 + w.ntok - 1, 1, all_lo, tmp);

    float m0 = neg_inf(), m1 = neg_inf(), l0 = 0.0f, l1 = 0.0f;
    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;

    for (int i = 0; i < w.nseg; ++i, ++it) {
      const int s = it % ST;
      if (!*abort_flag && !tc::mbar_wait(&full[s], (it / ST) & 1)) {
        set_device_error(a.err, kErrBounds);
        *abort_flag = 1;
      }
      __syncwarp();
      const int key0 = (w.lo / kStepKeys + w.blk + i) * kStepKeys + warp * 16;
      if (key0 < w.hi && key0 + 16 > w.lo) {         // (else no row sees any of this warp's keys)
        const uint32_t ks = sbase + s * C::STAGE, vs = ks + C::OPERAND;
        // ---- s = q k^T, two tiles of 8 keys
        float sc[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t kf[4];
          const int ch = 2 * k + kchunk;
          ldmatrix4(ks + (ch >> 3) * C::PANEL + kbase + (((ch & 7) ^ (kkey & 7)) << 4), kf);
          if constexpr (QREG) {
            mma16816(sc[0], qf[k], kf[0], kf[1]);
            mma16816(sc[1], qf[k], kf[2], kf[3]);
          } else {
            uint32_t qk[4];
            ldmatrix4(qbase + k * 32, qk);
            mma16816(sc[0], qk, kf[0], kf[1]);
            mma16816(sc[1], qk, kf[2], kf[3]);
          }
        }
        const bool edge = key0 < all_lo || key0 + 16 > all_hi;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) sc[n][j] *= a.scale_log2;
        if (edge) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int key = key0 + n * 8 + 2 * q4 + j;
              if (key < lo0 || key >= hi0) sc[n][j] = neg_inf();
              if (key < lo1 || key >= hi1) sc[n][2 + j] = neg_inf();
            }
        }
        // ---- running maximum and sum
        float x0 = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
        float x1 = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
        const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
        const float base0 = n0 == neg_inf() ? 0.0f : n0, base1 = n1 == neg_inf() ? 0.0f : n1;
        if (__any_sync(0xffffffffu, n0 != m0 || n1 != m1)) {
          const float f0 = exp2_approx(m0 - base0), f1 = exp2_approx(m1 - base1);
          l0 *= f0;
          l1 *= f1;
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            o[n][0] *= f0;
            o[n][1] *= f0;
            o[n][2] *= f1;
            o[n][3] *= f1;
          }
          m0 = n0;
          m1 = n1;
        }
        float p[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          // (two steps: at large scores the base itself cannot take the 15)
          p[n][0] = exp2_approx((sc[n][0] - base0) + kStepTop);
          p[n][1] = exp2_approx((sc[n][1] - base0) + kStepTop);
          p[n][2] = two ? exp2_approx((sc[n][2] - base1) + kStepTop) : 0.0f;
          p[n][3] = two ? exp2_approx((sc[n][3] - base1) + kStepTop) : 0.0f;
        }
        l0 += (p[0][0] + p[0][1]) + (p[1][0] + p[1][1]);
        l1 += (p[0][2] + p[0][3]) + (p[1][2] + p[1][3]);
        // weights in [0, 2^15], rounded to fp16 for the second product
        const uint32_t pf[4] = {pack_half2(p[0][0], p[0][1]), pack_half2(p[0][2], p[0][3]),
                                pack_half2(p[1][0], p[1][1]), pack_half2(p[1][2], p[1][3])};
        // ---- o += p v; keys that no row sees may hold anything: 0 * NaN
        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
        if (edge) {
          const auto seen = [&](int key) { return key >= w.lo && key < w.hi; };
          const int k0 = key0 + 2 * q4;
          keep0 = (seen(k0) ? 0x0000ffffu : 0u) | (seen(k0 + 1) ? 0xffff0000u : 0u);
          keep1 = (seen(k0 + 8) ? 0x0000ffffu : 0u) | (seen(k0 + 9) ? 0xffff0000u : 0u);
        }
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
          uint32_t vf[4];
          const int ch = 2 * n + vchunk;
          ldmatrix4_trans(vs + (ch >> 3) * C::PANEL + vbase + (((ch & 7) ^ (vkey & 7)) << 4), vf);
          mma16816(o[2 * n], pf, vf[0] & keep0, vf[1] & keep1);
          mma16816(o[2 * n + 1], pf, vf[2] & keep0, vf[3] & keep1);
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&empty[s]);
    }

    // ---- join the four warps
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    if (q4 == 0) {
      sm_m[warp][rl] = m0;
      sm_m[warp][rl + 8] = m1;
      sm_l[warp][rl] = l0;
      sm_l[warp][rl + 8] = l1;
    }
    consumer_sync();
#pragma unroll 1
    for (int part = 0; part < (two ? 2 : 1); ++part) {
      const int row = part * 8 + rl;
      const float mx = fmaxf(fmaxf(sm_m[0][row], sm_m[1][row]), fmaxf(sm_m[2][row], sm_m[3][row]));
      const float f = mx == neg_inf() ? 0.0f : exp2_approx((part ? m1 : m0) - mx);
      float *dst = mb + ((warp & 1) * 8 + rl) * C::MPITCH + 2 * q4;
      if (warp >= 2) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
          *reinterpret_cast<float2 *>(dst + n * 8) =
              make_float2((part ? o[n][2] : o[n][0]) * f, (part ? o[n][3] : o[n][1]) * f);
      }
      consumer_sync();
      if (warp < 2) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          float2 v = *reinterpret_cast<float2 *>(dst + n * 8);
          v.x = fmaf(part ? o[n][2] : o[n][0], f, v.x);
          v.y = fmaf(part ? o[n][3] : o[n][1], f, v.y);
          *reinterpret_cast<float2 *>(dst + n * 8) = v;
        }
      }
      consumer_sync();
      for (int i = tid; i < 8 * (D / 4); i += 128) {
        const int r8 = i / (D / 4), c4 = (i % (D / 4)) * 4, r = part * 8 + r8;
        if (r >= w.rows) continue;
        const float mr = fmaxf(fmaxf(sm_m[0][r], sm_m[1][r]), fmaxf(sm_m[2][r], sm_m[3][r]));
        float l = 0.0f;
#pragma unroll
        for (int x = 0; x < 4; ++x)          // (a warp whose scores are all NaN has no maximum, but a sum)
          l = fmaf(sm_l[x][r], sm_m[x][r] == neg_inf() ? 0.0f : exp2_approx(sm_m[x][r] - mr), l);
        const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);    // (NaN stays)
        l *= 1.0f / (1 << (int)kStepTop);
        const float4 u = *reinterpret_cast<const float4 *>(mb + r8 * C::MPITCH + c4);
        const float4 v = *reinterpret_cast<const float4 *>(mb + (8 + r8) * C::MPITCH + c4);
        const float4 res = make_float4((u.x + v.x) * inv, (u.y + v.y) * inv, (u.z + v.z) * inv, (u.w + v.w) * inv);
        if (whole) {
          const int64_t head = out_head(a, w.s.t0 + w.i0, w.h, r);
          store4(a, head * D + c4, res);
          if (a.lse && c4 == 0) a.lse[head] = natural_lse(mr, l);
        } else {
          const int64_t pr = ((int64_t)blockIdx.x * 2 + w.slot()) * kStepRows + r;
          *reinterpret_cast<float4 *>(a.part_o + pr * D + c4) = res;
          if (c4 == 0) a.part_ml[pr] = make_float2(mr, l);
        }
      }
      consumer_sync();
    }
    if (tid == 0 && !whole && w.slot() == 1) a.cuts[blockIdx.x] = w.cut(share_mem);
  }
}

template <int D>
cudaError_t launch_step(const CUtensorMap &mk, const CUtensorMap &mv, const Args &a, cudaStream_t s) {
  static std::atomic<size_t> per_dev[kMaxDevices];
  cudaError_t e = exl3_ensure_smem(reinterpret_cast<const void *>(attn_step_kernel<D>), StepCfg<D>::SMEM, per_dev);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_step_kernel<D>, dim3(exl3_attn_step_grid(D)), dim3(kStepThreads), StepCfg<D>::SMEM, s, mk,
                    mv, a);
}

}  // namespace attn
}  // namespace exl3

int exl3_attn_step_rows() { return exl3::attn::kStepRows; }
int exl3_attn_step_keys() { return exl3::attn::kStepKeys; }

// CTAs of a launch: all that the SMs hold at once.
int exl3_attn_step_grid(int D) {
  using namespace exl3::attn;
  return exl3_sm_count() * (D == 64 ? StepCfg<64>::CTAS : D == 128 ? StepCfg<128>::CTAS : StepCfg<256>::CTAS);
}

cudaError_t exl3_launch_attn_step(const CUtensorMap &mk, const CUtensorMap &mv, const exl3::attn::Args &a, int D,
                                  cudaStream_t s) {
  using namespace exl3::attn;
  switch (D) {
    case 64: return launch_step<64>(mk, mv, a, s);
    case 128: return launch_step<128>(mk, mv, a, s);
    default: return launch_step<256>(mk, mv, a, s);
  }
}
