// route.cu -- routing to experts: from a token's logits to the ids and weights
// that the grouped experts take.
//
//   s_e = softmax_e(l) or 1 / (1 + exp(-l_e));  c_e = s_e + bias_e
//   groups of consecutive experts are ranked by their largest c or by the sum
//   of their two largest, the best `kept` stay; the topk largest c of those are
//   chosen (equal values: the lower id); weights are the chosen s, divided by
//   their sum if asked, times `scale`.
//
// A warp takes a token; lane l holds experts l, l + 32, ... as keys that order
// as their values do (the float's bits, made monotone).  A pick is two warp
// reductions (redux: the largest key, then the lowest id that has it) and one
// pass over the owner's keys.  Softmax and the sigmoid are monotone, so without
// a bias and without sums of two the keys are the logits themselves: exact, and
// no exponential before the topk chosen ones.
//
// Otherwise values are computed in 32 bits, and every comparison that decides
// something (neighbouring picks, the last group kept and the first left out) is
// tested against a bound on their error.  A row with one that is closer than
// that is done again in 64 bits, so that ids are those of exact arithmetic; with
// random logits that is one row in a few hundred.
#include <algorithm>
#include <climits>

#include "exl3_common.cuh"
#include "router.cuh"

namespace exl3 {
namespace rt {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4;

__device__ __forceinline__ float neg_inf() { return __int_as_float((int)0xff800000u); }

// A key that orders as the value does (-0 as 0); NaN below everything.  Keys
// start at 1: 0 is a place without an expert, or one that is gone.
__device__ __forceinline__ unsigned order_key(float v) {
  const unsigned b = __float_as_uint(v + 0.0f);
  const unsigned k = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return v != v ? 1u : k;
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

__device__ __forceinline__ double sigmoid(double l) {
  const double t = exp(-fabs(l)), r = 1.0 / (1.0 + t);
  return l >= 0.0 ? r : t * r;
}

// Sum and maximum over the warp (the same order of additions every time).
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// Does the order of two computed values (v above w) hold for the exact ones?
// Infinities are exact; what is barred (-infinity) is never asked about.
__device__ __forceinline__ bool uncertain(float v, float w, float tol) {
  return w > neg_inf() && !(v - w > tol + 0x1p-22f * fabsf(v));
}

// The whole selection in 64 bits, from the row's values in shared memory.
// Lane j gets the j-th chosen expert.  Rare, so the simplest form.
template <bool F16>
__device__ __noinline__ int select_exact(const Args &a, int64_t row, int lane, double *c) {
  double mx = -INFINITY, sum = 0.0;
  if (a.score == EXL3_SCORE_SOFTMAX) {
    for (int e = lane; e < a.E; e += 32) mx = fmax(mx, (double)load_logit<F16>(a, row, e));
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmax(mx, __shfl_xor_sync(kFull, mx, o));
    if (mx == -INFINITY) mx = 0.0;
    for (int e = lane; e < a.E; e += 32) sum += exp((double)load_logit<F16>(a, row, e) - mx);
    sum = warp_sum(sum);
  }
  __syncwarp();
  for (int e = lane; e < a.E; e += 32) {
    const double l = load_logit<F16>(a, row, e);
    double v = a.score == EXL3_SCORE_SOFTMAX ? (sum == 0.0 ? 0.0 : exp(l - mx) / sum) : sigmoid(l);
    if (a.bias) v += (double)a.bias[e];
    // NaN ranks last, after what is barred (every finite value is above -1e300)
    c[e] = v != v ? -INFINITY : v == -INFINITY ? -1e300 : v;
  }
  __syncwarp();
  const int size = a.E / a.groups;
  unsigned keep = kFull;
  if (a.kept < a.groups) {
    double g = -INFINITY;
    if (lane < a.groups) {
      double first = -INFINITY, second = -INFINITY;
      for (int i = 0; i < size; ++i) {
        const double v = c[lane * size + i];
        second = fmax(second, fmin(first, v));
        first = fmax(first, v);
      }
      g = a.group_score == EXL3_GROUP_TOP2 && size > 1 ? first + second : first;
    }
    // rank of a group: how many stand before it
    int before = 0;
    for (int o = 0; o < a.groups; ++o) {
      const double v = __shfl_sync(kFull, g, o);
      before += v > g || (v == g && o < lane);
    }
    keep = __ballot_sync(kFull, lane < a.groups && before < a.kept);
  }
  unsigned taken = 0;      // bit i: expert lane + 32 i is chosen or left out
  for (int i = 0; lane + 32 * i < a.E; ++i)
    if (a.kept < a.groups && !(keep >> ((lane + 32 * i) / size) & 1u)) taken |= 1u << i;
  int mine = -1;
  for (int j = 0; j < a.topk; ++j) {
    double best = 0.0;
    int id = INT_MAX;
    for (int i = 0; lane + 32 * i < a.E; ++i) {
      const double v = c[lane + 32 * i];
      if (!(taken >> i & 1u) && (id == INT_MAX || v > best)) {
        best = v;
        id = lane + 32 * i;
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const double v = __shfl_xor_sync(kFull, best, o);
      const int other = __shfl_xor_sync(kFull, id, o);
      if (other != INT_MAX && (id == INT_MAX || v > best || (v == best && other < id))) {
        best = v;
        id = other;
      }
    }
    if (id == INT_MAX) break;
    if ((id & 31) == lane) taken |= 1u << (id >> 5);
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
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    l[i] = e < a.E ? load_logit<F16>(a, row, e) : neg_inf();
  }
  // the whole row's softmax, where it is asked for
  float mx = 0.0f, inv = 1.0f;
  if (soft && (VALUE || !a.renormalise)) {
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) top = max(top, lane + 32 * i < a.E ? order_key(l[i]) : 0u);
    top = __reduce_max_sync(kFull, top);
    mx = top > 1u ? key_value(top) : 0.0f;
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
      c = soft ? expf(l[i] - mx) * inv : sigmoid(l[i]);
      if (a.bias && e < a.E) c += a.bias[e];
    }
    key[i] = e < a.E ? order_key(c) : 0u;
  }
  // Bound on the error of a computed c, apart from its last rounding: the
  // sigmoid is off by 3 roundings (2^-22), the softmax by its exponential's
  // and its sum's (32 + 5 additions: below 2^-18 of the largest score).
  const float tol = soft ? 0x1p-18f * inv : 0x1p-21f;
  bool doubt = false;

  if (GROUPS) {
    // group values: `per` lanes to a group, every lane its share of the experts
    unsigned *keys = reinterpret_cast<unsigned *>(smem) + (size_t)warp * a.smem_per_warp / 4;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane + 32 * i < a.E) keys[lane + 32 * i] = key[i];
    __syncwarp();
    const int size = a.E / a.groups, per = a.group_lanes, g = lane / per, sub = lane % per;
    unsigned first = 0, second = 0;
    if (g < a.groups) {
      const int n = (size - sub + per - 1) / per;          // this lane's experts: sub, sub + per, ...
      for (int i = 0, at = n ? g % n : 0; i < n; ++i) {    // (started at different places: other banks)
        const unsigned k = keys[g * size + sub + per * at];
        second = max(second, min(first, k));
        first = max(first, k);
        at = at + 1 == n ? 0 : at + 1;
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
      value = first > 1u && second > 1u ? order_key(p + q) : 1u;
    }
    if (g >= a.groups || sub) value = 0;
    // the rank of each group among all of them
    unsigned left = value, keep = 0;
    float last = 0.0f;
    for (int j = 0; j <= a.kept; ++j) {                    // (kept < groups: one more than stays)
      const unsigned top = __reduce_max_sync(kFull, left);
      const int who = __ffs(__ballot_sync(kFull, left == top)) - 1;
      const float v = key_value(top);
      if (j == a.kept) {
        if (VALUE) doubt = top > 1u && uncertain(last, v, 2.0f * tol);
      } else {
        keep |= 1u << (who / per);
        if (lane == who) left = 0;
        last = v;
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane + 32 * i < a.E && !(keep >> ((lane + 32 * i) / size) & 1u)) key[i] = 0;
  }

  int mine = -1;
  {
    unsigned best = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) best = max(best, key[i]);
    const int picks = VALUE ? a.topk + 1 : a.topk;         // one more, to see how far off it is
    float last = 0.0f;
    for (int j = 0; j < picks; ++j) {
      const unsigned top = __reduce_max_sync(kFull, best);
      if (top == 0) break;                                 // (nothing behind the last pick)
      int id = INT_MAX;
#pragma unroll
      for (int i = V - 1; i >= 0; --i)
        if (key[i] == top) id = lane + 32 * i;
      id = __reduce_min_sync(kFull, id);
      if (VALUE) {
        const float v = key_value(top);
        doubt |= j > 0 && top > 1u && uncertain(last, v, tol);
        last = v;
      }
      if (j == lane && j < a.topk) mine = id;
      if ((id & 31) == lane) {
        best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (i == (id >> 5)) key[i] = 0;
          best = max(best, key[i]);
        }
      }
    }
  }
  if (VALUE && doubt)
    mine = select_exact<F16>(a, row, lane, reinterpret_cast<double *>(smem + (size_t)warp * a.smem_per_warp));

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
  a.group_lanes = 32;
  while (a.group_lanes * a.groups > 32) a.group_lanes /= 2;
  // the row's values in 64 bits where a doubtful row is done again; 32-bit keys for groups
  a.smem_per_warp = value ? (a.E * 8 + 15) / 16 * 16 : groups ? (a.E * 4 + 15) / 16 * 16 : 0;
  return f16 ? launch_v<true>(a, value, groups, s) : launch_v<false>(a, value, groups, s);
}
