// route.cu -- routing to experts: from a token's logits to the ids and weights
// that the grouped experts take.
//
//   s_e = softmax_e(l) or 1 / (1 + exp(-l_e));  c_e = s_e + bias_e
//   groups of consecutive experts are ranked by their largest c or by the sum
//   of their two largest, the best `kept` stay; the topk largest c of those are
//   chosen (equal values: the lower id); weights are the chosen s, divided by
//   their sum if asked, times `scale`.
//
// A warp takes a token; lane l holds experts l, l + 32, ... as keys that order as
// their values do (the float's bits, made monotone).  A pick is one warp reduction
// (redux: the largest key), a ballot (its lane) and a subtraction and a maximum
// over the owner's keys.  Softmax and the sigmoid
// are monotone, so without a bias and without sums of two the keys are the
// logits themselves: exact, and no exponential before the topk chosen ones.
//
// Otherwise values are computed in 32 bits, and every comparison that decides
// something (neighbouring picks, the last group kept and the first left out) is
// tested against a bound on their error.  A row with one that is closer than
// that, one in a few thousand with random logits, is done again on pairs of
// floats (about 45 bits).  Not in 64-bit floats: this chip has so few units for
// those that one such row took 15 us.  Neighbouring picks that are too close
// are put in order among themselves, a lane each; only groups that are, and more
// than 32 close picks, take the whole row.  Where all scores are below the bound (a
// sigmoid of logits around -15 and a bias of zero) that is every row: 44 us for 2500
// tokens of 256 experts, 8.2 around 0.
#include <algorithm>
#include <climits>

#include "exl3_common.cuh"
#include "router.cuh"

namespace exl3 {
namespace rt {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 2;          // of a block (4096 tokens of 256 experts: 6.0 us, 6.5 with four or eight)

__device__ __forceinline__ float neg_inf() { return __int_as_float((int)0xff800000u); }

// A key that orders as the value does (-0 as 0); NaN below everything (-infinity
// has 0x007fffff).  0 is a place without an expert, or one that is gone.
constexpr unsigned kNanKey = 64;
__device__ __forceinline__ unsigned order_key(float v) {
  const unsigned b = __float_as_uint(v + 0.0f);
  const unsigned k = b ^ ((unsigned)((int)b >> 31) | 0x80000000u);
  return v != v ? kNanKey : k;
}
__device__ __forceinline__ float key_value(unsigned k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

template <bool F16>
__device__ __forceinline__ float load_logit(const Args &a, int64_t row, int e) {
  if (F16) return __half2float(static_cast<const __half *>(a.logits)[row * a.stride + e]);
  return static_cast<const float *>(a.logits)[row * a.stride + e];
}

__device__ __forceinline__ float sigmoid(float l) {
  const float t = expf(-fabsf(l)), r = 1.0f / (1.0f + t);
  return l >= 0.0f ? r : t * r;
}

// Sum over the warp (the same order of additions every time).
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
// Does the order of two computed values (v above w) hold for the exact ones?  They
// are off by tol together, and by `rel` of themselves.  Infinities are exact;
// what is barred (-infinity) is never asked about.
__device__ __forceinline__ bool uncertain(float v, float w, float tol, float rel) {
  return w > neg_inf() && !(v - w > tol + rel * fabsf(v));
}

// ------------------------------------------------------ pairs of floats
//
// A value as the unevaluated sum of two floats, the second below half a unit of
// the first (Dekker's and Knuth's error-free sums and products).

struct Pair {
  float h, l;
};

__device__ __forceinline__ Pair quick_sum(float a, float b) {      // |a| >= |b|
  const float s = a + b;
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  Pair s = two_sum(a.h, b.h);
  const Pair t = two_sum(a.l, b.l);
  s = quick_sum(s.h, s.l + t.h);
  return quick_sum(s.h, s.l + t.l);
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
  const float p = __fmul_rn(a.h, b.h);
  return quick_sum(p, fmaf(a.h, b.h, -p) + fmaf(a.h, b.l, a.l * b.h));
}
__device__ __forceinline__ Pair div(Pair a, Pair b) {
  const float q = a.h / b.h;
  const Pair p = mul({q, 0.0f}, b);
  const Pair r = add(a, {-p.h, -p.l});
  return quick_sum(q, (r.h + r.l) / b.h);
}

// 1 / k as a pair.
template <int K>
__device__ __forceinline__ Pair inverse() {
  constexpr double v = 1.0 / K;
  constexpr float h = (float)v;
  return {h, (float)(v - (double)h)};
}

// 1 + r (1 + r / 2 (1 + r / 3 (...))): Taylor's series from its K-th factor on.
template <int K>
__device__ __forceinline__ Pair series(Pair r, Pair tail) {
  return add({1.0f, 0.0f}, mul(mul(r, inverse<K>()), tail));
}

// exp(x) for x <= 0: x = n ln 2 + r with ln 2 in parts of which the first has
// nine bits (n times it is exact; Cody and Waite), then the series.  From the
// eighth factor on (below 2^-27 of the result) single floats do.  Zero from exp(-69) down.
__device__ __forceinline__ Pair exp_pair(Pair x) {
  if (!(x.h > -69.0f)) return {x.h == x.h ? 0.0f : x.h, 0.0f};
  const float n = rintf(x.h * 1.44269504f);
  constexpr double ln2 = 0.693147180559945309417;
  constexpr float c1 = 0.693359375f, c2 = (float)(ln2 - c1), c3 = (float)(ln2 - c1 - c2);
  const float p = __fmul_rn(n, c2);
  Pair r = add({__fsub_rn(x.h, n * c1), x.l}, {-p, -fmaf(n, c2, -p)});
  r = add(r, {-n * c3, 0.0f});
  float t = 1.0f;
#pragma unroll
  for (int k = 13; k >= 8; --k) t = fmaf(r.h / (float)k, t, 1.0f);
  Pair e = series<7>(r, {t, 0.0f});
  e = series<6>(r, e);
  e = series<5>(r, e);
  e = series<4>(r, e);
  e = series<3>(r, e);
  e = series<2>(r, e);
  e = series<1>(r, e);
  const float f = scalbnf(1.0f, (int)n);
  return {e.h * f, e.l * f};
}

// Order keys of a pair, high and low.
__device__ __forceinline__ unsigned long long pair_key(Pair v) {
  const unsigned hi = order_key(v.h);
  return (unsigned long long)hi << 32 | (hi == kNanKey || isinf(v.h) ? 0u : order_key(v.l));
}
__device__ __forceinline__ Pair key_pair(unsigned long long k) {
  const float h = key_value((unsigned)(k >> 32));
  return {h, (unsigned)k ? key_value((unsigned)k) : 0.0f};
}

// The softmax's largest logit and sum of a row.
template <bool F16>
__device__ __forceinline__ void row_sum(const Args &a, int64_t row, int lane, float &mx, Pair &sum) {
  mx = neg_inf();
  for (int e = lane; e < a.E; e += 32) mx = fmaxf(mx, load_logit<F16>(a, row, e));
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
  if (mx == neg_inf()) mx = 0.0f;
  sum = {0.0f, 0.0f};
#pragma unroll 2
  for (int e = lane; e < a.E; e += 32) {
    const float l = load_logit<F16>(a, row, e);
    sum = add(sum, l == neg_inf() ? Pair{0.0f, 0.0f} : exp_pair(two_sum(l, -mx)));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum = add(sum, {__shfl_xor_sync(kFull, sum.h, o), __shfl_xor_sync(kFull, sum.l, o)});
}

// The key of expert e's c, or (VALUE false) of its logit.
template <bool F16, bool VALUE>
__device__ __forceinline__ unsigned long long value_key(const Args &a, int64_t row, int e, float mx, Pair sum) {
  const bool soft = a.score == EXL3_SCORE_SOFTMAX;
  const float l = load_logit<F16>(a, row, e);
  if (!VALUE) return (unsigned long long)order_key(l) << 32;
  const Pair t = exp_pair(soft ? two_sum(l, -mx) : Pair{-fabsf(l), 0.0f});
  Pair v = div(soft || !(l >= 0.0f) ? t : Pair{1.0f, 0.0f}, soft ? sum : add({1.0f, 0.0f}, t));
  if (l == neg_inf()) v = {0.0f, 0.0f};
  if (a.bias) {
    const float b = a.bias[e];
    v = isfinite(b) ? add(v, {b, 0.0f}) : Pair{v.h + b, 0.0f};
  }
  return pair_key(v);
}

// A row with picks that are too close: lane j has the j-th of `count` experts,
// of which everything else is known to be below; they are put in order.
template <bool F16, bool VALUE>
__device__ __noinline__ int order_pairs(const Args &a, int64_t row, int lane, int id, int count, int *place) {
  float mx = 0.0f;
  Pair sum = {0.0f, 0.0f};
  if (VALUE && a.score == EXL3_SCORE_SOFTMAX) row_sum<F16>(a, row, lane, mx, sum);
  const unsigned long long key = lane < count ? value_key<F16, VALUE>(a, row, id, mx, sum) : 0;
  int before = 0;
  for (int o = 0; o < count; ++o) {
    const unsigned long long v = __shfl_sync(kFull, key, o);
    const int other = __shfl_sync(kFull, id, o);
    before += v > key || (v == key && other < id);
  }
  __syncwarp();
  if (lane < count) place[before] = id;
  __syncwarp();
  return lane < count ? place[lane] : -1;
}

// The whole selection on pairs, the row's keys in shared memory: groups that are
// too close, or too many equal picks.  Lane j gets the j-th chosen expert.  Rare,
// so the simplest form.
template <bool F16, bool VALUE>
__device__ __noinline__ int select_pairs(const Args &a, int64_t row, int lane, unsigned long long *c) {
  float mx = 0.0f;
  Pair sum = {0.0f, 0.0f};
  if (VALUE && a.score == EXL3_SCORE_SOFTMAX) row_sum<F16>(a, row, lane, mx, sum);
  __syncwarp();
#pragma unroll 2
  for (int e = lane; e < a.E; e += 32) c[e] = value_key<F16, VALUE>(a, row, e, mx, sum);
  __syncwarp();
  const int size = a.E / a.groups;
  unsigned keep = kFull;
  if (a.kept < a.groups) {
    unsigned long long g = 0;
    if (lane < a.groups) {
      unsigned long long first = 0, second = 0;
      for (int i = 0; i < size; ++i) {
        const unsigned long long v = c[lane * size + i];
        second = max(second, min(first, v));
        first = max(first, v);
      }
      g = first;
      if (a.group_score == EXL3_GROUP_TOP2 && size > 1) {
        const Pair p = key_pair(first), q = key_pair(second);
        g = first >> 32 == kNanKey || second >> 32 == kNanKey ? (unsigned long long)kNanKey << 32
            : isinf(p.h) || isinf(q.h)              ? pair_key({p.h + q.h, 0.0f})
                                                    : pair_key(add(p, q));
      }
    }
    // rank of a group: how many stand before it
    int before = 0;
    for (int o = 0; o < a.groups; ++o) {
      const unsigned long long v = __shfl_sync(kFull, g, o);
      before += v > g || (v == g && o < lane);
    }
    keep = __ballot_sync(kFull, lane < a.groups && before < a.kept);
  }
  // left out: key 0, as what is chosen later
  for (int e = lane; e < a.E; e += 32)
    if (a.kept < a.groups && !(keep >> (e / size) & 1u)) c[e] = 0;
  int mine = -1;
  for (int j = 0; j < a.topk; ++j) {
    unsigned long long best = 0;
    int id = INT_MAX;
    for (int e = lane; e < a.E; e += 32)
      if (c[e] > best) {
        best = c[e];
        id = e;
      }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const unsigned long long v = __shfl_xor_sync(kFull, best, o);
      const int other = __shfl_xor_sync(kFull, id, o);
      if (v > best || (v == best && other < id)) {
        best = v;
        id = other;
      }
    }
    if (best == 0) break;
    if ((id & 31) == lane) c[id] = 0;       // (that lane reads it again)
    if (j == lane) mine = id;
  }
  return mine;
}

// V: experts per lane.  VALUE: c is computed (a bias, or groups by the sum of
// two); else the logits are the keys.  GROUPS: some groups are left out.
template <int V, bool F16, bool VALUE, bool GROUPS>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(const Args a) {
  extern __shared__ __align__(16) unsigned char smem[];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = (int64_t)blockIdx.x * kWarps + warp;
  if (row >= a.T) return;
  const bool soft = a.score == EXL3_SCORE_SOFTMAX;

  float l[V];
#pragma unroll
  for (int i = 0; i < V; ++i) l[i] = lane + 32 * i < a.E ? load_logit<F16>(a, row, lane + 32 * i) : neg_inf();
  // the whole row's softmax, where it is asked for
  float mx = 0.0f, inv = 1.0f;
  if (soft && (VALUE || !a.renormalise)) {
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) top = max(top, lane + 32 * i < a.E ? order_key(l[i]) : 0u);
    top = __reduce_max_sync(kFull, top);
    mx = top > kNanKey ? key_value(top) : 0.0f;
    if (mx == neg_inf()) mx = 0.0f;              // a row that is masked throughout: scores of zero
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += lane + 32 * i < a.E ? expf(l[i] - mx) : 0.0f;
    sum = warp_sum(sum);
    inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  }
  unsigned key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    float c = l[i];
    if (VALUE) {
      // (the fast exponential: both forms stay well within the bound below; the
      // sigmoid's may be too large to divide by)
      c = soft ? __expf(l[i] - mx) * inv : l[i] < -80.0f ? 0.0f : __fdividef(1.0f, 1.0f + __expf(-l[i]));
      if (a.bias && e < a.E) c += __ldg(a.bias + e);
    }
    key[i] = e < a.E ? order_key(c) : 0u;
  }
  // Bound on the error of two computed c together, apart from their own rounding.
  // Sigmoid: the exponential's units times s (1 - s) 0.7, the division 2, the sum
  // half a unit, of 2^-23 each.  Softmax: its exponential's and its sum's (32 + 5
  // additions), below 2^-18 of the largest score.
  const float tol = soft ? 0x1p-17f * inv : 0x1p-20f;
  bool doubt = false, again = false;       // picks or groups too close to call

  if (GROUPS) {
    // group values: `per` lanes to a group, every lane its share of the experts
    unsigned *keys = reinterpret_cast<unsigned *>(smem) + (size_t)warp * a.smem_per_warp / 4;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane + 32 * i < a.E) keys[lane + 32 * i] = key[i];
    __syncwarp();
    const int size = a.group_size, per = 1 << a.group_shift, g = lane >> a.group_shift, sub = lane & (per - 1);
    unsigned first = 0, second = 0;
    if (g < a.groups) {
      const unsigned *own = keys + g * size;
      int e = sub + ((g & 7) << a.group_shift);            // (started at different places: other banks)
      if (e >= size) e = sub;
      for (int i = sub; i < size; i += per) {
        const unsigned k = own[e];
        second = max(second, min(first, k));
        first = max(first, k);
        e += per;
        if (e >= size) e = sub;
      }
    }
    for (int o = per / 2; o; o >>= 1) {
      const unsigned f = __shfl_xor_sync(kFull, first, o), s = __shfl_xor_sync(kFull, second, o);
      second = max(max(second, s), min(first, f));
      first = max(first, f);
    }
    unsigned value = first;
    if (VALUE && a.group_score == EXL3_GROUP_TOP2 && size > 1) {
      const float p = key_value(first), q = key_value(second);
      value = first > kNanKey && second > kNanKey ? order_key(p + q) : kNanKey;
    }
    // how many groups stand before each (its first lane speaks for it)
    const bool speaks = g < a.groups && sub == 0;
    int before = 0;
    for (int o = 0; o < a.groups; ++o) {
      const unsigned v = __shfl_sync(kFull, value, o << a.group_shift);
      before += v > value || (v == value && o < g);
    }
    const unsigned keep = __ballot_sync(kFull, speaks && before < a.kept);
    if (VALUE) {                                           // the last that stays and the first that does not
      const int in = __ffs(__ballot_sync(kFull, speaks && before == a.kept - 1)) - 1;
      const int out = __ffs(__ballot_sync(kFull, speaks && before == a.kept)) - 1;
      const unsigned v = __shfl_sync(kFull, value, in), w = __shfl_sync(kFull, value, out);
      again = w > kNanKey && uncertain(key_value(v), key_value(w), 2.0f * tol, 0x1p-21f);
    }
#pragma unroll
    for (int i = 0; i < V; ++i)                            // (the product's upper bits: e / size for e below 2^10)
      if (!(keep >> (((lane + 32 * i) * a.group_inverse >> 20) << a.group_shift & 31) & 1u)) key[i] = 0;
  }

  // Picks: a key's lowest bits give way to the place within the lane (the first place
  // the largest; equal keys in one place go to the lower lane: the order of their
  // ids).  The owner's next key is its largest below the one that it gave: the one
  // for which key - top is largest modulo 2^32.
  constexpr unsigned LOW = V - 1;
  unsigned best = 0, top = 0, given = 0;                   // `given`: lane j's, the j-th pick's key,
  int from = 0, picks = a.topk;                            // and its lane
#pragma unroll
  for (int i = 0; i < V; ++i) {
    key[i] = key[i] ? (key[i] & ~LOW) | (LOW - i) : 0u;
    best = max(best, key[i]);
  }
  const auto pick = [&](int j) {
    top = __reduce_max_sync(kFull, best);
    const int owner = __ffs(__ballot_sync(kFull, best == top)) - 1;
    if (j == lane) {
      given = top;
      from = owner;
    }
    if (lane == owner) {
      unsigned rest = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) rest = max(rest, key[i] - top);
      best = rest + top;                                   // (of keys that are gone: 0)
      if (best >= top) best = 0;                           // (nothing below, only what it gave before)
    }
  };
  for (int j = 0; j < a.topk; ++j) pick(j);                // (there are as many)

  if (VALUE || !F16) {                                     // (an fp16 logit has no bits where the place went)
    // Could the exact values of two neighbouring picks stand in another order?
    const auto close = [&](unsigned upper, unsigned lower) {
      if (!VALUE) return (upper | LOW) == (lower | LOW);
      return lower > (kNanKey | LOW) &&
             uncertain(key_value(upper | LOW), key_value(lower & ~LOW), tol, 0x1p-22f + 0x1p-22f * V);
    };
    const unsigned next = __shfl_down_sync(kFull, given, 1);
    doubt = __any_sync(kFull, lane + 1 < a.topk && close(given, next));
    if (!VALUE && doubt) {                                 // (equal logits are in order)
      const unsigned k = order_key(load_logit<F16>(a, row, lane < a.topk ? from + 32 * (int)(LOW - (given & LOW)) : 0));
      const unsigned n = __shfl_down_sync(kFull, k, 1);
      doubt = __any_sync(kFull, lane + 1 < a.topk && close(given, next) && k != n);
    }
    // on until a pick is certainly below the topk-th
    for (;;) {
      const unsigned below = __reduce_max_sync(kFull, best);
      if (below == 0 || !close(top, below)) break;
      if (!VALUE) {                                        // all equal: the lower ids come first as they are
        unsigned high = 0, low = 0xffffffffu;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if ((key[i] | LOW) == (top | LOW)) {
            high = max(high, order_key(l[i]));
            low = min(low, order_key(l[i]));
          }
        if (__reduce_max_sync(kFull, high) == __reduce_min_sync(kFull, low)) break;
      }
      doubt = true;
      if (picks == 32) {
        again = true;
        break;
      }
      pick(picks++);
    }
  }
  int mine = lane < picks ? from + 32 * (int)(LOW - (given & LOW)) : -1;
  if (VALUE || !F16) {
    unsigned char *mem = smem + (size_t)warp * a.smem_per_warp;
    if (again) mine = select_pairs<F16, VALUE>(a, row, lane, reinterpret_cast<unsigned long long *>(mem));
    else if (doubt) mine = order_pairs<F16, VALUE>(a, row, lane, mine, picks, reinterpret_cast<int *>(mem));
  }

  // weights of the chosen
  const bool have = lane < a.topk && mine >= 0;
  float z = have ? load_logit<F16>(a, row, mine) : neg_inf();
  if (have && a.bias && a.bias[mine] == neg_inf()) z = neg_inf();       // barred: weight 0
  float w;
  if (a.renormalise) {
    // relative to the largest of them, so that scores below fp32's range keep their ratios
    float m = z;
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    if (m == neg_inf()) m = 0.0f;
    if (soft) {
      w = expf(z - m);
    } else {
      m = fminf(m, 0.0f);
      w = z > 0.0f ? 1.0f / (1.0f + expf(-z)) : expf(z - m) / (1.0f + expf(z));
    }
    if (!have) w = 0.0f;
    const float sum = warp_sum(w);
    w = sum == 0.0f ? 0.0f : w / sum;
  } else {
    w = soft ? expf(z - mx) * inv : sigmoid(z);
  }
  if (lane < a.topk) {
    a.ids[row * a.topk + lane] = max(mine, 0);
    a.weights[row * a.topk + lane] = w * a.scale;
  }
}

}  // namespace rt
}  // namespace exl3

using namespace exl3;

namespace {

template <int V, bool F16>
cudaError_t launch(const rt::Args &a, bool value, bool groups, cudaStream_t s) {
  const dim3 grid((a.T + rt::kWarps - 1) / rt::kWarps), block(32 * rt::kWarps);
  const size_t smem = (size_t)a.smem_per_warp * rt::kWarps;
  if (value) return groups ? launch_pdl(rt::route_kernel<V, F16, true, true>, grid, block, smem, s, a)
                           : launch_pdl(rt::route_kernel<V, F16, true, false>, grid, block, smem, s, a);
  return groups ? launch_pdl(rt::route_kernel<V, F16, false, true>, grid, block, smem, s, a)
                : launch_pdl(rt::route_kernel<V, F16, false, false>, grid, block, smem, s, a);
}

template <bool F16>
cudaError_t launch_v(const rt::Args &a, bool value, bool groups, cudaStream_t s) {
  if (a.E <= 32) return launch<1, F16>(a, value, groups, s);
  if (a.E <= 64) return launch<2, F16>(a, value, groups, s);
  if (a.E <= 128) return launch<4, F16>(a, value, groups, s);
  if (a.E <= 256) return launch<8, F16>(a, value, groups, s);
  if (a.E <= 512) return launch<16, F16>(a, value, groups, s);
  return launch<32, F16>(a, value, groups, s);
}

}  // namespace

cudaError_t exl3_launch_route(const rt::Args &in, bool f16, cudaStream_t s) {
  rt::Args a = in;
  const bool groups = a.kept < a.groups;
  const bool value = a.bias || (groups && a.group_score == EXL3_GROUP_TOP2);
  a.group_shift = 5;
  while ((a.groups << a.group_shift) > 32) --a.group_shift;
  a.group_size = a.E / a.groups;
  a.group_inverse = ((1 << 20) + a.group_size - 1) / a.group_size;
  // 64-bit keys where a doubtful row is done again, 32-bit keys for groups
  a.smem_per_warp = value || !f16 ? std::max(128, (a.E * 8 + 15) / 16 * 16) : groups ? (a.E * 4 + 15) / 16 * 16 : 0;
  return f16 ? launch_v<true>(a, value, groups, s) : launch_v<false>(a, value, groups, s);
}
