// attn_tc.cu -- attention of chunks of new tokens over a paged cache on the
// 5th-generation tensor cores.
//
//   S = Q K^T,  P = exp2((S - m) scale_log2 + 7),  O += P V,  y = O / sum(P)
//
// A unit holds up to 256 rows (D <= 128) or 128 rows (D = 256) of one key
// head and walks over its keys in blocks of 64: 4 D operations per row and
// key against 4 D bytes per key, so from about 280 rows per key read from
// memory the tensor cores are the limit.  Both products are tcgen05.mma: Q and
// K from shared memory into a TMEM slot of 128 x 64 fp32 scores; the softmax
// warps read the slot (a thread per row), write the fp16 weights over its
// first half, and the second product takes them from there (A operand in
// TMEM) with V as it lies in the cache (an MN-major operand: no transposition
// anywhere) into O, which stays in TMEM for the whole unit.  With 256-wide
// heads q is an A operand in TMEM too: its 64 KB of shared memory go to the
// rings and a score product reads K alone (16 on 2 heads, 2,047 tokens behind
// 63,000, by graph replay: 1.66 to 1.76 ms with q in shared memory, 1.59 to 1.7
// so, boards and their temperature differ).
//
// Every row tile of 128 has two slots that its blocks take in turn and a
// softmax warpgroup: the scores of block j + 1 are computed while the weights
// of block j are, and only the softmax of a tile is a chain.  (Blocks of 128
// keys leave room for one slot per tile; then the next scores wait for the
// product that reads the weights, and softmax, both products and four barriers
// follow one another: 1.34 PFLOP/s on 4096 tokens behind 64,000 at D = 128,
// against 1.46.)  64-wide score products read 6 KB of shared memory each, 48
// cycles where the arithmetic takes 32, which caps the pair of products at 80 %
// of the tensor cores' rate.  At that rate the chip is also held by its power
// limit when the launch is repeated: 8,192 tokens take 529 us after a rest and
// 565 us at the 1942 MHz that are left after seconds.
//
// Each MMA warp spends about as long on barriers, descriptors and commits as
// its products take, so score products have two warps (a tile or a slot each)
// and weight products one per tile.
//
// The running maximum m moves only when it has grown by more than a factor of
// 2^8 (in the weights; fp16 holds 2^15): then O is read, scaled and written
// back, which is rare after the first blocks.  Sums, maxima, S and O are
// fp32; the weights are rounded to fp16 once, the type of V, which the second
// product's operands have to share.  m is taken off before the scale
// is multiplied on, so that the exponent of the largest key is exactly
// 7 whatever the scores' size: as fma(S, scale_log2, -m scale_log2) it would add
// the rounding error of the product, which from 2^28 on passes the range of
// fp16 (that form took 1.3 % less on 8,192 tokens).
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

constexpr int kTcKeys = 64;
constexpr int kTcCost = 7;         // a unit's start and end, in blocks
constexpr float kLazy = 8.0f;      // log2 of the growth that moves the maximum
// Weights are 2^kTop at the maximum (off again in the sum that leaves the
// kernel), so 2^15 at most, and fp16 holds those down to 2^-21 of the largest
// in full and the rest to 2^-32 of it.
constexpr float kTop = 7.0f;

template <int D>
struct TcCfg {
  static constexpr int NQ = D == 256 ? 1 : 2;            // row tiles of a unit
  static constexpr int ROWS = NQ * 128;
  // K and V have a ring each, written by one warp and read by one: a stage is
  // a block's K (64-column panels of 64 keys) or V; up to 160 KB in all.
  static constexpr int PANEL = kTcKeys * 128;            // bytes
  static constexpr int STAGE = kTcKeys * D * 2;
  static constexpr int KST = D == 64 ? 8 : D == 128 ? 5 : 4, VST = D == 64 ? 8 : D == 128 ? 5 : 3;
  // With one tile of 256-wide heads there is room for q in TMEM.
  static constexpr bool QTM = D == 256;
  static constexpr int QTILE = 128 * D * 2;
  static constexpr int QPANEL = 128 * 128;               // 64 columns of 128 rows
  static constexpr int OFF_K = QTM ? 0 : NQ * QTILE, OFF_V = OFF_K + KST * STAGE;
  static constexpr int SMEM = OFF_V + VST * STAGE + 1024 /*alignment*/;
  static constexpr int SM_WARPS = 4 * NQ;                // softmax warps
  // softmax warpgroups, then two warpgroups with the MMA issuers and the
  // producers; registers move from the latter to the former (the sum over the
  // warpgroups is what the launch allots: 4 x 128, or 3 x 168)
  static constexpr int THREADS = (SM_WARPS + 8) * 32;
  static constexpr int REGS_SM = NQ == 2 ? 168 : 216, REGS_IO = NQ == 2 ? 88 : 144;
  static constexpr uint32_t TM_S = 0, TM_Q = 128, TM_O = 256;   // TMEM columns: slots of 64, two per tile; q; O
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

__device__ __forceinline__ bool try_wait_plain(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(tc::smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// 32 bytes in one store, or in two where only 16-byte alignment is known.
__device__ __forceinline__ void store32(void *dst, const uint32_t (&v)[8], bool aligned) {
  if (!aligned) {
    reinterpret_cast<uint4 *>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4 *>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    return;
  }
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

template <int N>
__device__ __forceinline__ void set_registers(bool more) {
  if (more) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A producer warp: brings every block's K (or V) to its ring.  K and V have a
// warp each: the arithmetic, barriers and issue of one operand take a warp
// about half as long as its MMAs take the tensor cores, and a chain of both
// in one warp held the rest up.
template <int D, bool V, class Wait>
__device__ __forceinline__ void produce(const Args &a, Walk<kTcKeys, kTcCost> w, const CUtensorMap *tmQ,
                                        const CUtensorMap *tm, uint32_t sbase, uint64_t *full, uint64_t *empty,
                                        uint64_t *q_full, uint64_t *q_empty, const Wait &wait) {
  using C = TcCfg<D>;
  constexpr int ST = V ? C::VST : C::KST;
  const int lane = threadIdx.x & 31, box = 1 << a.box_log2;
  int it = 0, qn0 = 0, qn1 = 0;
  bool stop = false;
  // the pages of a block's boxes, lane i box i (at most 4), looked up while
  // the block before is under way (a unit's first block waits for its look-up:
  // the ring is blocks ahead of the MMAs, registers are short)
  int page = -1, off = 0;
  PageWalk<kTcKeys> pages;
  for (; w.left > 0 && !stop; w.next(a)) {
    pages.begin(a, w);
    pages.next(a, page, off);
    const int n = w.nseg;
    const bool two = C::NQ == 2 && w.ntok > a.tile_tok;
    for (int j = 0; j < n && !stop; ++j) {
      const int key0 = (w.lo / kTcKeys + w.blk + j) * kTcKeys;
      int my_page = page;
      const int my_off = off;
      if (j + 1 < n) pages.next(a, page, off);
      const int lo = max(w.lo - key0, 0), hi = min(w.hi - key0, kTcKeys);     // keys of the block that some row sees
      if (lane >= (lo >> a.box_log2) && lane << a.box_log2 < hi && (unsigned)my_page >= (unsigned)a.num_pages) {
        set_device_error(a.err, kErrBounds);
        my_page = a.num_pages;                 // past the map's end: reads as zeros
      }
      // every lane holds the boxes' pages before the wait, so that after it one
      // lane has nothing to do but ask
      int pg[4], c1[4], c2[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        pg[b] = __shfl_sync(0xffffffffu, my_page, b);
        const int po = __shfl_sync(0xffffffffu, my_off, b);
        c1[b] = a.head_first ? w.h : po;
        c2[b] = a.head_first ? po : w.h;
      }
      const int item = it + j, st = item % ST;
      const int b0 = lo >> a.box_log2, b1 = (hi + box - 1) >> a.box_log2;      // the boxes that some row sees
      const uint32_t dst = sbase + (V ? C::OFF_V : C::OFF_K) + st * C::STAGE;
      if (item >= ST) stop = !__all_sync(0xffffffffu, wait(&empty[st], ((item / ST) & 1) ^ 1));
      if (stop) break;
      if (tc::elect_one()) {
        if (b1 > b0) tc::mbar_arrive_expect_tx(&full[st], (uint32_t)(((b1 - b0) << a.box_log2) * D * 2));
        else tc::mbar_arrive(&full[st]);
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (b >= b0 && b < b1) {
#pragma unroll
            for (int q = 0; q < D / 64; ++q)
              tma_load_4d_at(dst + (b << a.box_log2) * 128 + q * C::PANEL, tm, &full[st], q * 64, c1[b], c2[b], pg[b]);
          }
      }
      __syncwarp();
      if (!V && !C::QTM && j == 0 && !stop) {
        // the unit's q, as soon as the last unit's scores are done with its
        // place: G heads of tile_tok tokens are the tile's rows in order
        // (tokens past the unit's are rows that nobody writes)
#pragma unroll 1
        for (int t = 0; t < (two ? 2 : 1); ++t) {
          const int u = t ? qn1 : qn0;
          if (u > 0) stop = !__all_sync(0xffffffffu, wait(&q_empty[t], (u - 1) & 1));
          if (stop) break;
          if (t) ++qn1;
          else ++qn0;
          if (tc::elect_one()) {
            tc::mbar_arrive_expect_tx(&q_full[t], (uint32_t)(a.tile_tok * a.G * D * 2));
#pragma unroll
            for (int q = 0; q < D / 64; ++q)
              tma_load_3d_at(sbase + t * C::QTILE + q * C::QPANEL, tmQ, &q_full[t], q * 64, w.h * a.G,
                             w.s.t0 + w.i0 + t * a.tile_tok);
          }
          __syncwarp();
        }
      }
    }
    it += n;
  }
  // After a wait that ran out nobody consumes any more: give the copies in
  // flight their time before the CTA's memory goes to another.
  if (stop) __nanosleep(1000000);
}

template <int D>
__global__ void __launch_bounds__(TcCfg<D>::THREADS, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const Args a) {
  using C = TcCfg<D>;
  constexpr int KST = C::KST, VST = C::VST;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t k_full[KST], k_empty[KST], v_full[VST], v_empty[VST], s_full[4], p_full[4], pv_done[4], q_full[2],
      q_empty[2];
  __shared__ Share share_mem;
  __shared__ long long warp_sums[C::THREADS / 32];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  const uint32_t raw = tc::smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  volatile int *abort_flag = &abort_word;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < KST; ++s) {
      tc::mbar_init(&k_full[s], 1);
      tc::mbar_init(&k_empty[s], 2);
    }
    for (int s = 0; s < VST; ++s) {
      tc::mbar_init(&v_full[s], 1);
      tc::mbar_init(&v_empty[s], C::NQ);
    }
    for (int s = 0; s < 4; ++s) {
      tc::mbar_init(&s_full[s], 1);
      tc::mbar_init(&p_full[s], 4);
      tc::mbar_init(&pv_done[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(&q_full[s], C::QTM ? 4 : 1);
      tc::mbar_init(&q_empty[s], C::QTM ? 2 : 1);
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
  const Share share = make_share<kTcKeys, kTcCost, C::THREADS>(a, 1 + kTcCost, &share_mem, warp_sums);
  clear_padding<D>(a, C::THREADS);

  // A wait that runs out records the error; every later wait then returns at
  // once, so that all roles run through their loops and the CTA ends.
  // (Waits without a suspend-time hint: with one, waking up costs 4 % of a
  // long chunk; spinning on test_wait costs as much in issue slots.)
  const auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
    if (try_wait_plain(bar, parity)) return true;
    const long long t0 = clock64();
    while (!*abort_flag) {
      if (try_wait_plain(bar, parity)) return true;
      if (clock64() - t0 > tc::kWaitLimit) {
        set_device_error(a.err, kErrBounds);
        *abort_flag = 1;
      }
    }
    return false;
  };

  Walk<kTcKeys, kTcCost> w;
  w.begin(a, share);
  if (tid == 0) {
    a.cuts[blockIdx.x].rows = 0;           // (the thread that may fill the record in below)
    share_mem = share;                     // (out of the registers; who still reads it, reads the same)
  }

  // (This branch first: with the softmax ahead of it in the code, the prompt of
  // 8,192 tokens took 596 us instead of 522.  Why is not known; the 64- and
  // 128-wide kernels spill 336 bytes, all on account of the softmax loop, and
  // are as sensitive to branches in it that are never taken.)
  if (warp >= C::SM_WARPS) {
    set_registers<C::REGS_IO>(false);
    if (warp == C::SM_WARPS || warp == C::SM_WARPS + 1) {
      // ======================================================== MMAs: scores
      // Two warps: one per tile, or (one tile) one per slot, so that the waits,
      // commits and descriptors of one are covered by the MMAs of the other.  A
      // tile's blocks are counted through all its units: block c takes slot
      // c % 2 of the tile, and is the slot's use c / 2.
      const int me = warp - C::SM_WARPS, t = C::NQ == 2 ? me : 0;
      int it = 0, units = 0, c0 = 0;
      for (; w.left > 0; w.next(a)) {
        const int n = w.nseg;
        const bool live = t == 0 || w.ntok > a.tile_tok;          // this unit has the tile
        if (live) wait(&q_full[t], units++ & 1);
        // (q in TMEM: in a unit of one block only one of the two warps has scores
        // to compute, so the next q is announced once both have seen this one's)
        __syncwarp();
        if (C::QTM && tc::elect_one()) tc::mbar_arrive(&q_empty[0]);
        for (int j = 0; j < n; ++j) {
          const int st = (it + j) % KST, c = c0 + j, slot = 2 * t + (c & 1);
          const bool mine = C::NQ == 2 ? live : (c & 1) == me;
          // the slot's last weights have to be consumed first
          if (mine && c >= 2) wait(&pv_done[slot], ((c >> 1) - 1) & 1);
          wait(&k_full[st], ((it + j) / KST) & 1);
          __syncwarp();
          tc::tc_fence_after();
          if (tc::elect_one()) {
            if (mine) {
              const uint64_t ad = sdesc_k_sw128(sbase + t * C::QTILE);
              const uint64_t bd = sdesc_k_sw128(sbase + C::OFF_K + st * C::STAGE);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t bk = bd + (kk / 4) * (C::PANEL >> 4) + (kk % 4) * 2;
                if constexpr (C::QTM)
                  mma_f16_ts(tmem + C::TM_S + slot * 64, tmem + C::TM_Q + kk * 8, bk, C::IDESC_S, kk ? 1u : 0u);
                else
                  tc::mma_f16(tmem + C::TM_S + slot * 64, ad + (kk / 4) * (C::QPANEL >> 4) + (kk % 4) * 2, bk, C::IDESC_S,
                              kk ? 1u : 0u);
              }
              tc::mma_commit(&s_full[slot]);
              tc::mma_commit(&k_empty[st]);
            } else {
              tc::mbar_arrive(&k_empty[st]);
            }
            // this warp's last scores of the unit: q is free when they are done
            if (!C::QTM && live && j == n - 1) tc::mma_commit(&q_empty[t]);
          }
          __syncwarp();
        }
        it += n;
        if (live) c0 += n;
      }
    } else if (warp == C::SM_WARPS + 2 || (C::NQ == 2 && warp == C::SM_WARPS + 3)) {
      // ================================================ MMAs: weighted values
      const int t = warp - C::SM_WARPS - 2;
      int it = 0, c0 = 0;
      for (; w.left > 0; w.next(a)) {
        const int n = w.nseg;
        const bool live = t == 0 || w.ntok > a.tile_tok;
        for (int j = 0; j < n; ++j) {
          const int st = (it + j) % VST, c = c0 + j, slot = 2 * t + (c & 1);
          if (live) wait(&p_full[slot], (c >> 1) & 1);
          wait(&v_full[st], ((it + j) / VST) & 1);
          const int key0 = (w.lo / kTcKeys + w.blk + j) * kTcKeys;
          if (live && (key0 < w.lo || key0 + kTcKeys > w.hi)) {
            // V rows that no row of the unit sees may hold anything: zeros (the
            // other tile's warp may be writing the same)
            for (int i = lane; i < kTcKeys * (D / 8); i += 32) {
              const int r = i & (kTcKeys - 1), q = i / kTcKeys;      // row, 16-byte column
              if (key0 + r < w.lo || key0 + r >= w.hi)
                asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(
                                 sbase + C::OFF_V + st * C::STAGE + (q >> 3) * C::PANEL + r * 128 + (q & 7) * 16),
                             "r"(0)
                             : "memory");
            }
            fence_async_shared();
          }
          __syncwarp();
          tc::tc_fence_after();
          if (tc::elect_one()) {
            if (live) {
              const uint64_t bd = sdesc_mn_sw128(sbase + C::OFF_V + st * C::STAGE, C::PANEL);
#pragma unroll
              for (int kk = 0; kk < kTcKeys / 16; ++kk)
                mma_f16_ts(tmem + C::TM_O + t * D, tmem + C::TM_S + slot * 64 + kk * 8, bd + kk * (2048 >> 4), C::IDESC_O,
                           (j | kk) ? 1u : 0u);
              tc::mma_commit(&pv_done[slot]);
              tc::mma_commit(&v_empty[st]);
            } else {
              tc::mbar_arrive(&v_empty[st]);
            }
          }
          __syncwarp();
        }
        it += n;
        if (live) c0 += n;
      }
    } else if (warp == C::SM_WARPS + 4) {
      // =========================================================== producers
      produce<D, false>(a, w, &tmQ, &tmK, sbase, k_full, k_empty, q_full, q_empty, wait);
    } else if (warp == C::SM_WARPS + 5) {
      produce<D, true>(a, w, &tmQ, &tmV, sbase, v_full, v_empty, q_full, q_empty, wait);
    }
  } else {
    // ============================================================= softmax
    set_registers<C::REGS_SM>(true);
    const int t = warp / 4;                  // row tile
    const int wl = warp & 3;
    const uint32_t lanes = (uint32_t)(wl * 32) << 16;
    const int row = wl * 32 + lane;          // within the tile
    const float lazy = fminf(kLazy / a.scale_log2, 1e38f);
    int c = 0;                               // blocks of this tile so far
    int brought = 0;                         // units whose q is in TMEM
    // q of a unit to TMEM (256-wide heads): a thread brings its row, as the
    // fp16 pairs that an A operand's columns hold.  The place is free when the
    // scores of the unit before have all been read; the barrier may go on to
    // its next phase only when both score warps have seen the last.
    const auto bring_q = [&](const auto &u) {
      if (u.left <= 0) return;
      const int tok = row_token(a, row);
      const uint4 *src = reinterpret_cast<const uint4 *>(a.q + (int64_t)(u.s.t0 + u.i0 + tok) * a.q_stride +
                                                         (int64_t)(u.h * a.G + row - tok * a.G) * D);
#pragma unroll
      for (int q = 0; q < D / 64; ++q) {
        uint32_t v[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 x = row < u.rows ? src[8 * q + i] : make_uint4(0, 0, 0, 0);
          v[4 * i] = x.x;
          v[4 * i + 1] = x.y;
          v[4 * i + 2] = x.z;
          v[4 * i + 3] = x.w;
        }
        tmem_st32u(tmem + C::TM_Q + lanes + 32 * q, v);
      }
      tc::tmem_st_wait();
      tc::tc_fence_before();
      if (brought > 0) wait(&q_empty[0], (brought - 1) & 1);
      ++brought;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&q_full[0]);
    };
    if constexpr (C::QTM) bring_q(w);
    for (; w.left > 0; w.next(a)) {
      const int n = w.nseg;
      const bool two = C::NQ == 2 && w.ntok > a.tile_tok;
      if (t == 1 && !two) continue;
      // this tile's tokens and rows, and the keys that this thread's row sees
      const int i0 = w.i0 + t * a.tile_tok, ntok = min(a.tile_tok, w.ntok - t * a.tile_tok);
      const int rows = ntok * a.G;
      int lo = 0, hi = 0, all_lo, all_hi, tmp;
      if (row < rows) token_range(a, w.s, i0 + row_token(a, row), 1, lo, hi);
      token_range(a, w.s, i0, 1, tmp, all_hi);
      token_range(a, w.s, i0 + ntok - 1, 1, all_lo, tmp);

      float m = neg_inf(), l = 0.0f;         // the exponents' base (in scores) and the sum of weights
      float base = 0.0f;                     // m, or 0 before the row's first keys
      for (int j = 0; j < n; ++j, ++c) {
        const int slot = 2 * t + (c & 1);
        const uint32_t tm_s = tmem + C::TM_S + slot * 64 + lanes;
        const int key0 = (w.lo / kTcKeys + w.blk + j) * kTcKeys;
        wait(&s_full[slot], (c >> 1) & 1);
        __syncwarp();
        tc::tc_fence_after();
        float s[64];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float v[32];
          tc::tmem_ld32(tm_s + 32 * q, v);
#pragma unroll
          for (int i = 0; i < 32; ++i) s[32 * q + i] = v[i];
        }
        tc::tmem_ld_wait();
        if (key0 < all_lo || key0 + kTcKeys > all_hi) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (key0 + i < lo || key0 + i >= hi) s[i] = neg_inf();
        }
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = s[i];
#pragma unroll
        for (int i = 4; i < 64; ++i) x[i & 3] = fmaxf(x[i & 3], s[i]);
        const float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        // (the sum is rounded down: no weight's exponent passes kLazy)
        const bool grow = mx > __fadd_rd(m, lazy);
        if (__any_sync(0xffffffffu, grow)) {
          const bool scaled = grow && m != neg_inf();      // (before a row's first keys O and the sum are zero)
          if (__any_sync(0xffffffffu, scaled)) {
            // O so far has to be complete before it is scaled
            wait(&pv_done[slot ^ 1], ((c - 1) >> 1) & 1);
            __syncwarp();
            tc::tc_fence_after();
            const float f = scaled ? exp2_approx((m - mx) * a.scale_log2) : 1.0f;
            l *= f;
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              float v[32];
              tc::tmem_ld32(tmem + C::TM_O + t * D + lanes + 32 * q, v);
              tc::tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] *= f;
              tc::tmem_st32(tmem + C::TM_O + t * D + lanes + 32 * q, v);
            }
            tc::tmem_st_wait();
          }
          if (grow) m = mx;
          base = m == neg_inf() ? 0.0f : m;
        }
        const float2 sc2 = make_float2(a.scale_log2, a.scale_log2), nb2 = make_float2(-base, -base);
        const float2 top2 = make_float2(kTop, kTop);
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float2 e = __ffma2_rn(__fadd2_rn(make_float2(s[2 * i], s[2 * i + 1]), nb2), sc2, top2);
          const float2 p = make_float2(exp2_approx(e.x), exp2_approx(e.y));
          sum[i & 1] = __fadd2_rn(sum[i & 1], p);
          const __half2 h = __floats2half2_rn(p.x, p.y);
          pk[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        tmem_st32u(tm_s, pk);
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        tc::tmem_st_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&p_full[slot]);
      }

      if constexpr (C::QTM) {
        // (this unit's scores are all there, so its q is no longer read)
        auto ahead = w;
        ahead.next(a);
        bring_q(ahead);
      }
      // ---- O complete: y, or this CTA's part of it
      wait(&pv_done[2 * t + ((c - 1) & 1)], ((c - 1) >> 1) & 1);
      __syncwarp();
      tc::tc_fence_after();
      const bool whole = w.whole();
      const bool aligned = !whole || a.y_aligned32;
      const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);      // (NaN stays)
      const float m2 = m * a.scale_log2;
      l *= 1.0f / (1 << (int)kTop);
      // (parts of a cut unit: the rows of its tiles one after the other)
      const int64_t head = out_head(a, w.s.t0 + i0, w.h, row);
      const int64_t pr = ((int64_t)blockIdx.x * 2 + w.slot()) * C::ROWS + t * a.tile_tok * a.G + row;
      if (row < rows) {
        if (!whole) a.part_ml[pr] = make_float2(m2, l);
        else if (a.lse) a.lse[head] = natural_lse(m2, l);
      }
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        float v[32];
        tc::tmem_ld32(tmem + C::TM_O + t * D + lanes + 32 * q, v);
        tc::tmem_ld_wait();
        if (row < rows) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] *= inv;
          // (32-byte stores: a row's sectors are written whole)
          if (whole && !a.f32out) {
            __half *dst = static_cast<__half *>(a.y) + head * D + 32 * q;
#pragma unroll
            for (int i = 0; i < 32; i += 16) {
              uint32_t h[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const __half2 x = __floats2half2_rn(v[i + 2 * k], v[i + 2 * k + 1]);
                h[k] = *reinterpret_cast<const uint32_t *>(&x);
              }
              store32(dst + i, h, aligned);
            }
          } else {
            float *dst = (whole ? static_cast<float *>(a.y) + head * D : a.part_o + pr * D) + 32 * q;
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint32_t h[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) h[k] = __float_as_uint(v[i + k]);
              store32(dst + i, h, aligned);
            }
          }
        }
      }
      tc::tc_fence_before();
      if (tid == 0 && !whole && w.slot() == 1) a.cuts[blockIdx.x] = w.cut(share_mem);
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  if (warp == C::SM_WARPS) {
    if (*abort_flag) __nanosleep(1000000);   // (MMAs that nobody waited for)
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
// Keys that one tensor copy must not straddle.
int exl3_attn_tc_keys() { return exl3::attn::kTcKeys; }
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
