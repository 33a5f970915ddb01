// attn_tc.cu -- attention of chunks of new tokens over a paged cache on the
// 5th-generation tensor cores.
//
//   S = Q K^T,  P = exp2(S scale_log2 - base),  O += P V,  y = O / sum(P)
//
// A unit holds up to 256 rows (D <= 128) or 128 rows (D = 256) of one key
// head and walks over its keys in blocks of 128: 4 D operations per row and
// key against 4 D bytes per key, so from about 280 rows per byte-bound key on
// the tensor cores are the limit.  Both products are tcgen05.mma: Q and K
// from shared memory into a TMEM slot of 128 x 128 fp32 scores; the softmax
// warps read the slot (a thread per row), write the fp16 weights over its
// first half, and the second product takes them from there (A operand in
// TMEM) with V as it lies in the cache (an MN-major operand: no transposition
// anywhere) into O, which stays in TMEM for the whole unit.
//
// Two slots keep the tensor cores busy while the exponentials run: a unit of
// more than 128 rows has two row tiles with a slot and a softmax warpgroup
// each, and the MMAs of one tile run during the softmax of the other; a unit
// of one tile gives its blocks to the slots in turn, and the scores of the
// next block are computed during the softmax of this one.
//
// The running maximum moves only when it has grown by more than a factor of
// 2^8 (in the weights; fp16 holds 2^15): then O is read, scaled and written
// back, which is rare after the first blocks.  Sums, maxima, S and O are
// fp32; the weights are rounded to fp16 once.
//
// Blocks in which some row sees not all keys are masked; their V rows that no
// row of the unit sees are zeroed in shared memory first, since 0 * NaN would
// not be 0.
#include <cudaTypedefs.h>

#include "attn_common.cuh"
#include "tc_ptx.cuh"

int exl3_attn_tc_grid();

namespace exl3 {
namespace attn {

constexpr int kTcKeys = 128;
constexpr int kTcCost = 3;         // a unit's start and end, in blocks
constexpr float kLazy = 8.0f;      // log2 of the growth that moves the maximum

#ifndef OPS_OF
#define OPS_OF(D) ((D) == 256 ? 2 : 1)
#endif
template <int D>
struct TcCfg {
  static constexpr int NQ = D == 256 ? 1 : 2;            // row tiles of a unit
  static constexpr int ROWS = NQ * 128;
  // The ring's stages are parts of an operand, so that a part's place is free
  // again as soon as its MMAs are done.
  static constexpr int OPS = OPS_OF(D);                  // parts of one operand
  static constexpr int KPANELS = D / 64 / OPS;           // K part: 128 keys x this many 64-column panels
  static constexpr int VPART_KEYS = kTcKeys / OPS;       // V part: these keys x D columns
  static constexpr int STAGE = kTcKeys * D * 2 / OPS;
  static constexpr int ST = 163840 / STAGE;              // 160 KB
  static constexpr int QTILE = 128 * D * 2;
  static constexpr int QPANEL = 128 * 128;               // 64 columns of 128 rows
  static constexpr int OFF_RING = NQ * QTILE;
  static constexpr int SMEM = OFF_RING + ST * STAGE + 1024 /*alignment*/;
  static constexpr int SM_WARPS = 4 * NQ;                // softmax warps
  // softmax warpgroups, then one warpgroup with the MMA issuer and the
  // producer; registers move from the latter to the former (the sum over the
  // warpgroups is what the launch allots: 3 x 168 or 2 x 248)
  static constexpr int THREADS = (SM_WARPS + 4) * 32;
  static constexpr int REGS_SM = NQ == 2 ? 208 : 248, REGS_IO = NQ == 2 ? 88 : 248;
  static constexpr uint32_t TM_S = 0, TM_O = 256;        // TMEM columns
  static constexpr uint32_t IDESC_S = tc::idesc_f16(128, kTcKeys);
  static constexpr uint32_t IDESC_O = tc::idesc_f16(128, D) | (1u << 16);   // B (V) is MN-major
};

// D[tmem] (+)= A[tmem] * B[smem]: the weights are the A operand.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// MN-major operand, 128-byte swizzle: rows of 64 elements (128 bytes) along
// N, 8-row atoms of 1024 bytes along K, the next 64 elements `panel` bytes on.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t addr, uint32_t panel) {
  uint64_t d = 0;
  d |= (addr >> 4) & 0x3FFFull;
  d |= (uint64_t)((panel >> 4) & 0x3FFF) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ uint64_t sdesc_k_sw128(uint32_t addr) {
  return ((addr >> 4) & 0x3FFFull) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)2 << 61);
}

__device__ __forceinline__ void tmem_st32u(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]),
      "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]),
      "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

__device__ __forceinline__ void tma_load_4d_at(uint32_t dst, const CUtensorMap *m, uint64_t *bar, int x, int c1,
                                               int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(tc::smem_u32(bar)), "r"(x), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d_at(uint32_t dst, const CUtensorMap *m, uint64_t *bar, int x, int c1,
                                               int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
      "[%2];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(tc::smem_u32(bar)), "r"(x), "r"(c1), "r"(c2)
      : "memory");
}

__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void set_registers(bool more) {
  if (more) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// How often each of the two slots has been given scores.
struct Uses {
  int u0 = 0, u1 = 0;
  __device__ __forceinline__ int get(int s) const { return s ? u1 : u0; }
  __device__ __forceinline__ void add(int s, int n) {
    if (s) u1 += n;
    else u0 += n;
  }
};

// Order of a unit's operands in the ring, that of their use: with two row
// tiles K0 V0 K1 V1 ..., with one (whose next scores come before this block's
// weights) K0 K1 V0 K2 V1 ... V(n-1).  The o-th operand's block:
__device__ __forceinline__ int operand(bool two, int n, int o, bool &isv) {
  if (two) {
    isv = o & 1;
    return o >> 1;
  }
  isv = o > 0 && (o % 2 == 0 || o == 2 * n - 1);
  return o == 2 * n - 1 ? n - 1 : isv ? o / 2 - 1 : (o + 1) / 2;
}

// ... and the place of block j's K or V among them.
__device__ __forceinline__ int k_place(bool two, int j) { return two ? 2 * j : max(0, 2 * j - 1); }
__device__ __forceinline__ int v_place(bool two, int n, int j) { return two || j == n - 1 ? 2 * j + 1 : 2 * j + 2; }

template <int D>
__global__ void __launch_bounds__(TcCfg<D>::THREADS, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const Args a) {
  using C = TcCfg<D>;
  constexpr int ST = C::ST, OPS = C::OPS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[ST], empty[ST], s_full[2], p_full[2], pv_done[2], q_full[2], q_empty[2];
  __shared__ Share share;
  __shared__ long long warp_sums[C::THREADS / 32];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  const uint32_t raw = tc::smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  const uint32_t ring = sbase + C::OFF_RING;
  volatile int *abort_flag = &abort_word;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < ST; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(&s_full[s], 1);
      tc::mbar_init(&p_full[s], 4);
      tc::mbar_init(&pv_done[s], 1);
      tc::mbar_init(&q_full[s], 1);
      tc::mbar_init(&q_empty[s], 1);
    }
    abort_word = 0;
    tc::fence_mbar_init();
    tc::prefetch_tmap(&tmQ);
    tc::prefetch_tmap(&tmK);
    tc::prefetch_tmap(&tmV);
  }
  if (warp == C::SM_WARPS) {
    tc::tmem_alloc(&tmem_slot, 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_trigger();
  pdl_wait();
  make_share<kTcKeys, kTcCost, C::THREADS>(a, 1 + kTcCost, &share, warp_sums);
  clear_padding<D>(a, C::THREADS);

  // A wait that runs out records the error; every later wait then returns at
  // once, so that all roles run through their loops and the CTA ends.
  const auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
    if (tc::mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!*abort_flag) {
      if (tc::mbar_try_wait(bar, parity)) return true;
      if (clock64() - t0 > tc::kWaitLimit) {
        set_device_error(a.err, kErrBounds);
        *abort_flag = 1;
      }
    }
    return false;
  };

  Walk<kTcKeys, kTcCost> w;
  w.begin(a, share);
  if (tid == 0) a.cuts[blockIdx.x].rows = 0;           // (the thread that may fill the record in below)

  // (every warp of a warpgroup moves its registers, at the head of its role)
  if (warp == C::SM_WARPS + 1) {
    // ============================================================ producer
    if constexpr (C::REGS_IO < C::REGS_SM) set_registers<C::REGS_IO>(false);
    int it = 0, qn0 = 0, qn1 = 0;
    bool stop = false;
    // the pages of a block's boxes, lane i box i (at most 8), looked up while
    // the block before is under way; K and V of a unit are asked for in the
    // order of their use, which may have block j + 1's K before block j's V,
    // so the pages of two blocks are held
    int page[2], off[2], next_page = -1, next_off = 0;
    PageWalk<kTcKeys> pages;
    if (w.left > 0) {
      pages.begin(a, w);
      pages.next(a, next_page, next_off);
    }
    while (w.left > 0 && !stop) {
      auto ahead = w;
      ahead.next(a);
      const int n = w.nseg;
      const bool two = C::NQ == 2 && w.ntok > a.tile_tok;
      for (int o = 0; o < 2 * n && !stop; ++o) {
        bool isv;
        const int j = operand(two, n, o, isv);
        if (!isv) {
          page[1] = page[0];
          off[1] = off[0];
          page[0] = next_page;
          off[0] = next_off;
          if (j + 1 < n) {
            pages.next(a, next_page, next_off);
          } else if (ahead.left > 0) {
            pages.begin(a, ahead);
            pages.next(a, next_page, next_off);
          }
        }
        // block j is the newest whose K was asked for, or the one before it
        const int newest = two ? j : min(n - 1, o == 0 ? 0 : (o + 1) / 2);
        const int old = isv && j < newest;
        const int key0 = (w.lo / kTcKeys + w.blk + j) * kTcKeys;
#pragma unroll 1
        for (int p = 0; p < OPS && !stop; ++p, ++it) {
          // the boxes of this part that some row sees
          const int nkeys = isv ? C::VPART_KEYS : kTcKeys, npan = isv ? D / 64 : C::KPANELS;
          const int base = key0 + (isv ? p * C::VPART_KEYS : 0);
          const int k_lo = max(w.lo, base), k_hi = min(w.hi, base + nkeys);
          const int box = 1 << a.box_log2;
          const int box0 = k_hi > k_lo ? (k_lo - base) >> a.box_log2 : 0;
          const int nbox = k_hi > k_lo ? ((k_hi - base + box - 1) >> a.box_log2) - box0 : 0;
          const int first = (isv ? (p * C::VPART_KEYS) >> a.box_log2 : 0) + box0;   // of the block's boxes
          const int s = it % ST;
          if (it >= ST) stop = !__all_sync(0xffffffffu, wait(&empty[s], ((it / ST) & 1) ^ 1));
          if (stop) break;
          const uint32_t bytes = (uint32_t)((nbox << a.box_log2) * 128 * npan);
          if (lane == 0) {
            if (bytes) tc::mbar_arrive_expect_tx(&full[s], bytes);
            else tc::mbar_arrive(&full[s]);
          }
          __syncwarp();
          // one lane asks for the boxes: everything here is uniform, and
          // copies asked for by several lanes would be issued one by one too
          for (int bx = 0; bx < nbox; ++bx) {
            int my_page = __shfl_sync(0xffffffffu, old ? page[1] : page[0], first + bx);
            const int my_off = __shfl_sync(0xffffffffu, old ? off[1] : off[0], first + bx);
            if ((unsigned)my_page >= (unsigned)a.num_pages) {
              if (lane == 0) set_device_error(a.err, kErrBounds);
              my_page = a.num_pages;         // past the map's end: reads as zeros
            }
            const uint32_t dst = ring + s * C::STAGE + ((box0 + bx) << a.box_log2) * 128;
            const int c1 = a.head_first ? w.h : my_off, c2 = a.head_first ? my_off : w.h;
            if (tc::elect_one()) {
              if (isv) {
#pragma unroll
                for (int q = 0; q < D / 64; ++q)
                  tma_load_4d_at(dst + q * (C::VPART_KEYS * 128), &tmV, &full[s], q * 64, c1, c2, my_page);
              } else {
#pragma unroll
                for (int q = 0; q < C::KPANELS; ++q)
                  tma_load_4d_at(dst + q * (kTcKeys * 128), &tmK, &full[s], (p * C::KPANELS + q) * 64, c1, c2, my_page);
              }
            }
            __syncwarp();
          }
        }
        if (o == 0 && !stop) {
          // the unit's q, as soon as the last unit's scores are done with its
          // place: G heads of tile_tok tokens are the tile's rows in order
          // (tokens past the unit's are rows that nobody writes)
#pragma unroll 1
          for (int t = 0; t < (two ? 2 : 1); ++t) {
            const int u = t ? qn1++ : qn0++;
            if (u > 0) stop = !__all_sync(0xffffffffu, wait(&q_empty[t], (u - 1) & 1));
            if (stop) break;
            if (lane == 0) tc::mbar_arrive_expect_tx(&q_full[t], (uint32_t)(a.tile_tok * a.G * D * 2));
            __syncwarp();
            if (tc::elect_one()) {
#pragma unroll
              for (int q = 0; q < D / 64; ++q)
                tma_load_3d_at(sbase + t * C::QTILE + q * C::QPANEL, &tmQ, &q_full[t], q * 64, w.h * a.G,
                               w.s.t0 + w.i0 + t * a.tile_tok);
            }
            __syncwarp();
          }
        }
      }
      w = ahead;
    }
    if (stop) {                              // leave no copy in flight behind
      for (int i = max(0, it - ST); i < it; ++i) tc::mbar_wait(&full[i % ST], (i / ST) & 1);
      // (a phase that q was not asked for in has no copy either)
      if (qn0 > 0) tc::mbar_wait(&q_full[0], (qn0 - 1) & 1);
      if (qn1 > 0) tc::mbar_wait(&q_full[1], (qn1 - 1) & 1);
    }
  } else if (warp == C::SM_WARPS) {
    // ========================================================== MMA issuer
    if constexpr (C::REGS_IO < C::REGS_SM) set_registers<C::REGS_IO>(false);
    int it = 0;
    Uses use;
    // Scores of a block into a slot; `free_k`: nobody reads these K parts
    // after, `free_q`: nor this tile's q.
    const auto issue_s = [&](int t, int slot, int kit, bool free_k, bool free_q) {
      // the slot's last weights have to be consumed first
      if (use.get(slot) > 0) wait(&pv_done[slot], (use.get(slot) - 1) & 1);
#pragma unroll
      for (int p = 0; p < OPS; ++p) {
        const int st = (kit + p) % ST;
        wait(&full[st], ((kit + p) / ST) & 1);
        __syncwarp();
        tc::tc_fence_after();
        if (tc::elect_one()) {
          const uint64_t ad = sdesc_k_sw128(sbase + t * C::QTILE + p * C::KPANELS * C::QPANEL);
          const uint64_t bd = sdesc_k_sw128(ring + st * C::STAGE);
#pragma unroll
          for (int kk = 0; kk < C::KPANELS * 4; ++kk) {
            const int o = (kk / 4) * (C::QPANEL >> 4) + (kk % 4) * 2;
            tc::mma_f16(tmem + C::TM_S + slot * 128, ad + o, bd + o, C::IDESC_S, (p | kk) ? 1u : 0u);
          }
          if (p == OPS - 1) tc::mma_commit(&s_full[slot]);
          if (free_k) tc::mma_commit(&empty[st]);
          if (p == OPS - 1 && free_q) tc::mma_commit(&q_empty[t]);
        }
        __syncwarp();
      }
      use.add(slot, 1);
    };
    // O += weights of a slot times a block's V.
    const auto issue_pv = [&](int t, int slot, int vit, bool first, bool free_v) {
      wait(&p_full[slot], (use.get(slot) - 1) & 1);
#pragma unroll
      for (int p = 0; p < OPS; ++p) {
        const int st = (vit + p) % ST;
        wait(&full[st], ((vit + p) / ST) & 1);
        __syncwarp();
        tc::tc_fence_after();
        if (tc::elect_one()) {
          const uint64_t bd = sdesc_mn_sw128(ring + st * C::STAGE, C::VPART_KEYS * 128);
#pragma unroll
          for (int kk = 0; kk < C::VPART_KEYS / 16; ++kk)
            mma_f16_ts(tmem + C::TM_O + t * D, tmem + C::TM_S + slot * 128 + (p * C::VPART_KEYS / 16 + kk) * 8,
                       bd + kk * (2048 >> 4), C::IDESC_O, (!first || p || kk) ? 1u : 0u);
          if (p == OPS - 1) tc::mma_commit(&pv_done[slot]);
          if (free_v) tc::mma_commit(&empty[st]);
        }
        __syncwarp();
      }
    };
    int qphase0 = 0, qphase1 = 0;
    for (; w.left > 0; w.next(a)) {
      const int n = w.nseg;
      const bool two = C::NQ == 2 && w.ntok > a.tile_tok;
      const auto kit = [&](int j) { return it + OPS * k_place(two, j); };
      const auto vit = [&](int j) { return it + OPS * v_place(two, n, j); };
      wait(&q_full[0], qphase0++ & 1);
      if (two) {
        issue_s(0, 0, kit(0), false, n == 1);
        wait(&q_full[1], qphase1++ & 1);
        issue_s(1, 1, kit(0), true, n == 1);
        for (int j = 0; j < n; ++j) {
          issue_pv(0, 0, vit(j), j == 0, false);
          if (j + 1 < n) issue_s(0, 0, kit(j + 1), false, j + 2 == n);
          issue_pv(1, 1, vit(j), j == 0, true);
          if (j + 1 < n) issue_s(1, 1, kit(j + 1), true, j + 2 == n);
        }
      } else {
        issue_s(0, 0, kit(0), true, n == 1);
        for (int j = 0; j < n; ++j) {
          if (j + 1 < n) issue_s(0, (j + 1) & 1, kit(j + 1), true, j + 2 == n);
          issue_pv(0, j & 1, vit(j), j == 0, true);
        }
      }
      it += 2 * OPS * n;
    }
  } else if (warp < C::SM_WARPS) {
    // ============================================================= softmax
    if constexpr (C::REGS_IO < C::REGS_SM) set_registers<C::REGS_SM>(true);
    const int t = warp / 4;                  // row tile
    const int wl = warp & 3;
    const uint32_t lanes = (uint32_t)(wl * 32) << 16;
    const int row = wl * 32 + lane;          // within the tile
    const int ltid = tid - t * 128;
    int it = 0;
    Uses use;
    for (; w.left > 0; w.next(a)) {
      const int n = w.nseg;
      const bool two = C::NQ == 2 && w.ntok > a.tile_tok;
      if (t == 1 && !two) {
        // a unit of one tile uses both slots: follow the second one's phases
        for (int j = 1; j < n; j += 2) wait(&s_full[1], use.u1++ & 1);
        use.u0 += (n + 1) / 2;
        it += 2 * OPS * n;
        continue;
      }
      // this tile's tokens and rows, and the keys that this thread's row sees
      const int i0 = w.i0 + t * a.tile_tok, ntok = min(a.tile_tok, w.ntok - t * a.tile_tok);
      const int rows = ntok * a.G;
      int lo = 0, hi = 0, all_lo, all_hi, tmp;
      if (row < rows) token_range(a, w.s, i0 + row_token(a, row), 1, lo, hi);
      token_range(a, w.s, i0, 1, tmp, all_hi);
      token_range(a, w.s, i0 + ntok - 1, 1, all_lo, tmp);

      float m = neg_inf(), l = 0.0f;         // the exponent's base (in scores) and the sum of weights
      int last_slot = 0, last_use = 0;
      for (int j = 0; j < n; ++j) {
        const int slot = two ? t : (j & 1);
        const int u = use.get(slot);
        use.add(slot, 1);
        const int key0 = (w.lo / kTcKeys + w.blk + j) * kTcKeys;
        wait(&s_full[slot], u & 1);
        __syncwarp();
        tc::tc_fence_after();
        float s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float v[32];
          tc::tmem_ld32(tmem + C::TM_S + slot * 128 + lanes + 32 * c, v);
#pragma unroll
          for (int i = 0; i < 32; ++i) s[32 * c + i] = v[i];
        }
        tc::tmem_ld_wait();
        if (key0 < all_lo || key0 + kTcKeys > all_hi) {
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (key0 + i < lo || key0 + i >= hi) s[i] = neg_inf();
        }
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = s[i];
#pragma unroll
        for (int i = 8; i < 128; ++i) x[i & 7] = fmaxf(x[i & 7], s[i]);
        const float mx = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
        const bool grow = m != neg_inf() && (mx - m) * a.scale_log2 > kLazy;
        if (__any_sync(0xffffffffu, grow)) {
          // O so far has to be complete before it is scaled
          wait(&pv_done[last_slot], last_use & 1);
          __syncwarp();
          tc::tc_fence_after();
          const float f = grow ? exp2_approx((m - mx) * a.scale_log2) : 1.0f;
          l *= f;
          if (grow) m = mx;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float v[32];
            tc::tmem_ld32(tmem + C::TM_O + t * D + lanes + 32 * c, v);
            tc::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= f;
            tc::tmem_st32(tmem + C::TM_O + t * D + lanes + 32 * c, v);
          }
          tc::tmem_st_wait();
        }
        if (m == neg_inf()) m = mx;          // a row's first keys: O and the sum are zero
        const float base = m == neg_inf() ? 0.0f : m * a.scale_log2;
        const float2 sc2 = make_float2(a.scale_log2, a.scale_log2), nb2 = make_float2(-base, -base);
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 e = __ffma2_rn(make_float2(s[64 * c + 2 * i], s[64 * c + 2 * i + 1]), sc2, nb2);
            const float2 p = make_float2(exp2_approx(e.x), exp2_approx(e.y));
            sum[i & 1] = __fadd2_rn(sum[i & 1], p);
            const __half2 h = __floats2half2_rn(p.x, p.y);
            pk[i] = *reinterpret_cast<const uint32_t *>(&h);
          }
          tmem_st32u(tmem + C::TM_S + slot * 128 + lanes + 32 * c, pk);
        }
        if (key0 < w.lo || key0 + kTcKeys > w.hi) {
          // V rows that no row of the unit sees: zeros.  The last block's
          // product has to be over before `full` of this block's V is looked
          // at: until then the ring may be a whole turn behind it.
          if (j > 0) wait(&pv_done[last_slot], last_use & 1);
          const int vi = it + OPS * v_place(two, n, j) + ltid / C::VPART_KEYS;
          wait(&full[vi % ST], (vi / ST) & 1);
          const int key = key0 + ltid;
          if (key < w.lo || key >= w.hi) {
            const uint32_t dst = ring + (vi % ST) * C::STAGE + (ltid % C::VPART_KEYS) * 128;
#pragma unroll
            for (int p = 0; p < D / 64; ++p)
#pragma unroll
              for (int c = 0; c < 8; ++c)
                asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(dst + p * C::VPART_KEYS * 128 + c * 16),
                             "r"(0)
                             : "memory");
          }
          fence_async_shared();
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        tc::tmem_st_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&p_full[slot]);
        last_slot = slot;
        last_use = u;
      }
      if (two) use.add(1 - t, n);
      it += 2 * OPS * n;

      // ---- O complete: y, or this CTA's part of it
      wait(&pv_done[last_slot], last_use & 1);
      __syncwarp();
      tc::tc_fence_after();
      const bool whole = w.whole();
      const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);      // (NaN stays)
      const float lse2 = l == 0.0f ? neg_inf() : m * a.scale_log2 + log2f(l);
      // (parts of a cut unit: the rows of its tiles one after the other)
      const int64_t head = out_head(a, w.s.t0 + i0, w.h, row);
      const int64_t pr = ((int64_t)blockIdx.x * 2 + w.slot()) * C::ROWS + t * a.tile_tok * a.G + row;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float v[32];
        tc::tmem_ld32(tmem + C::TM_O + t * D + lanes + 32 * c, v);
        tc::tmem_ld_wait();
        if (row < rows) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] *= inv;
          if (whole && !a.f32out) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              __half2 h[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) h[k] = __floats2half2_rn(v[i + 2 * k], v[i + 2 * k + 1]);
              *reinterpret_cast<uint4 *>(static_cast<__half *>(a.y) + head * D + 32 * c + i) =
                  *reinterpret_cast<uint4 *>(h);
            }
          } else {
            float *dst = whole ? static_cast<float *>(a.y) + head * D : a.part_o + pr * D;
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4 *>(dst + 32 * c + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          }
        }
      }
      if (row < rows) {
        if (!whole) a.part_lse[pr] = lse2;
        else if (a.lse) a.lse[head] = lse2 * 0.69314718055994530942f;
      }
      tc::tc_fence_before();
      if (tid == 0 && !whole && w.slot() == 1) a.cuts[blockIdx.x] = w.cut(share);
    }
  } else {
    if constexpr (C::REGS_IO < C::REGS_SM) set_registers<C::REGS_IO>(false);
  }

  tc::tc_fence_before();
  __syncthreads();
  if (warp == C::SM_WARPS) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch_tc(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const Args &a, cudaStream_t s) {
  static std::atomic<size_t> per_dev[kMaxDevices];
  cudaError_t e = exl3_ensure_smem(reinterpret_cast<const void *>(attn_tc_kernel<D>), TcCfg<D>::SMEM, per_dev);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_tc_kernel<D>, dim3(exl3_attn_tc_grid()), dim3(TcCfg<D>::THREADS), TcCfg<D>::SMEM, s, mq, mk,
                    mv, a);
}

}  // namespace attn
}  // namespace exl3

int exl3_attn_tc_rows(int D) { return D == 256 ? 128 : 256; }
// Keys that one tensor copy must not straddle: a block, or a part of its V.
int exl3_attn_tc_keys(int D) { return exl3::attn::kTcKeys / OPS_OF(D); }
int exl3_attn_tc_grid() { return exl3_sm_count(); }

cudaError_t exl3_launch_attn_tc(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                                const exl3::attn::Args &a, int D, cudaStream_t s) {
  using namespace exl3::attn;
  switch (D) {
    case 64: return launch_tc<64>(mq, mk, mv, a, s);
    case 128: return launch_tc<128>(mq, mk, mv, a, s);
    default: return launch_tc<256>(mq, mk, mv, a, s);
  }
}
