// head_transform.cu -- norms of query and key heads with the rotary position
// rotation in one pass, and the same with an append to a paged cache.
//
//   n = x * rsqrt(mean(x^2) + eps) * w                       (per head)
//   (a, b) -> magnitude * (a cos t - b sin t, b cos t + a sin t)
//
// Both calls are bound by memory: each input is read once and each output
// written once, 2 to 4 bytes either way against about seven operations an
// element.  Nothing is shared between warps: no block-wide barrier, and 20
// warps per SM with up to four loads in flight each cover the memory's latency
// (9,310 tokens at 40/8 heads of 128, 267 MB: 54.4 us, 4.9 TB/s; what the
// warps wait for is still mostly loads).  All warps take equal runs of the
// tokens' passes, cutting tokens where they have to: whole tokens left most
// warps without one in the last round (59.1 us).  A
// lane holds eight neighbouring elements (16 bytes of fp16) of a head, so D / 8
// lanes hold a head, the mean is a few shuffles, and the lane keeps its place
// in the head while the warp walks over the token's heads: the norm weights
// and the cosines and sines of its elements stay in registers.  The warp works
// out the token's R / 2 angles once, 32 at a time.
//
// Angles.  A position times a frequency has to be known to a fraction of a
// turn however far the position is.  The frequency in turns (f / 2 pi) is held
// as a 64-bit fixed-point fraction, from f's 24-bit significand times 2^64 / 2
// pi in integers (an FP64 product would be exact enough too, but GB300 has few
// FP64 units); its product with the int32 position, modulo 2^64, is the angle
// modulo a turn with an error below |position| * 2^-62 turns for f <= 1, and
// its upper 32 bits go to sincospif.  No large argument is left to reduce.
#include "exl3_common.cuh"
#include "head_transform.cuh"

namespace exl3 {
namespace ht {

constexpr int kWarps = 4, kThreads = 32 * kWarps, kCtas = 5;   // per CTA, per SM
// Passes whose data is under way beside the one at hand, and passes per turn
// of the loop: fp32 rows are twice as long and three ahead spill (1,777 tokens
// at 24/8 heads of 64: 4.3 us with one, 6.8 with three), fp16 rows gain from
// three (9,310 tokens appended: 54.4 us; two ahead 57.1, one 57.7).  Six CTAs
// per SM (80 registers) take 56.8 us, four 58.1.
template <bool F32>
constexpr int kAhead = F32 ? 1 : 3;
template <bool F32>
constexpr int kUnroll = F32 ? 1 : 4;

// The frequency in turns, modulo one, times 2^64: |f| = m 2^-s.
__device__ __forceinline__ unsigned long long turn_step(float freq) {
  constexpr unsigned long long kInv2Pi = 0x28be60db9391054aull;   // floor(2^64 / 2 pi)
  const unsigned bits = __float_as_uint(freq), ex = (bits >> 23) & 255;
  const unsigned long long m = ex ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
  const int s = 150 - (ex ? (int)ex : 1);
  const unsigned long long lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
  unsigned long long r;
  if (s <= 0) r = -s < 64 ? lo << -s : 0;
  else if (s < 64) r = (lo >> s) | (hi << (64 - s));
  else r = s < 128 ? hi >> (s - 64) : 0;
  return bits >> 31 ? 0 - r : r;
}

// An angle in half turns, within [-1, 1].
__device__ __forceinline__ float half_turns(int pos, unsigned long long step) {
  const unsigned long long ang = step * (unsigned long long)(long long)pos;
  return (float)(int)(unsigned)(ang >> 32) * 4.656612873077393e-10f;   // * 2^-31
}

struct Row8 {
  float v[8];
};

// Eight elements as they lie in memory.
template <bool F32>
struct Raw8 {
  uint4 u[F32 ? 2 : 1];
};

template <bool F32>
__device__ __forceinline__ Raw8<F32> load_raw(const void *base, int64_t i) {
  Raw8<F32> r;
  const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const char *>(base) + i * (F32 ? 4 : 2));
  r.u[0] = p[0];
  if constexpr (F32) r.u[1] = p[1];
  return r;
}

template <bool F32>
__device__ __forceinline__ Row8 unpack(const Raw8<F32> &w) {
  Row8 r;
  if constexpr (F32) {
    const float4 x = *reinterpret_cast<const float4 *>(&w.u[0]), y = *reinterpret_cast<const float4 *>(&w.u[1]);
    r.v[0] = x.x; r.v[1] = x.y; r.v[2] = x.z; r.v[3] = x.w;
    r.v[4] = y.x; r.v[5] = y.y; r.v[6] = y.z; r.v[7] = y.w;
  } else {
    const __half2 *h = reinterpret_cast<const __half2 *>(&w.u[0]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(h[j]);
      r.v[2 * j] = f.x;
      r.v[2 * j + 1] = f.y;
    }
  }
  return r;
}

__device__ __forceinline__ void store8(void *base, int64_t i, const Row8 &r, bool f32) {
  if (f32) {
    float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + i);
    p[0] = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
    p[1] = make_float4(r.v[4], r.v[5], r.v[6], r.v[7]);
  } else {
    __half2 h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = __floats2half2_rn(r.v[2 * j], r.v[2 * j + 1]);
    *reinterpret_cast<uint4 *>(static_cast<__half *>(base) + i) = *reinterpret_cast<uint4 *>(h);
  }
}

// Sequence of row t: the number of starts q_start[1 .. B] that are <= t
// (B: the row belongs to none).  32 starts are looked at in each step.
__device__ __forceinline__ int find_seq(const int *q_start, int B, int t, int lane) {
  if (__ldg(q_start) > t) return B;
  int lo = 0, hi = B;                      // the count lies in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + (lane + 1) * step;  // is q_start[i] <= t ?
    const bool le = i <= hi && __ldg(q_start + i) <= t;
    const int n = __popc(__ballot_sync(0xffffffffu, le));
    lo += n * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

// The passes over a token's heads, 32 / LPH heads each: queries, keys, values.
struct Passes {
  int q, k, all;
};

__host__ __device__ inline Passes count_passes(int Hq, int Hkv, int per_pass, bool append) {
  Passes p;
  p.q = (Hq + per_pass - 1) / per_pass;
  const int kv = (Hkv + per_pass - 1) / per_pass;
  p.k = p.q + kv;
  p.all = p.k + (append ? kv : 0);
  return p;
}

// How a lane's eight elements meet their partners: all eight in another lane
// (half layout, R / 2 a multiple of 8, or no rotation), in the same lane
// (pairs, R a multiple of 8), or one by one.
enum { kByLane, kInLane, kAny };

// The passes of all tokens are a line of which every warp takes `run`: whole
// tokens, but for its first and last one.
template <int D, bool F32IN, bool APPEND, int MODE>
__global__ void __launch_bounds__(kThreads, kCtas) head_transform_kernel(const Args a, int run) {
  constexpr int LPH = D / 8;               // lanes per head
  constexpr int HPP = 32 / LPH;            // heads per pass
  __shared__ __align__(16) float2 table[kWarps][D / 2];
  __shared__ float stage_mem[kWarps][MODE == kAny ? 32 : 1][9];   // partners that are looked up one by one

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = lane % LPH, e0 = 8 * c;    // this lane's eight elements of its heads
  const Passes ps = count_passes(a.Hq, a.Hkv, HPP, APPEND);
  const int R = a.rotary_dim, half = R / 2;
  float2 *cs = table[warp];
  float(*stage)[9] = stage_mem[warp];
  pdl_trigger();
  pdl_wait();

  const bool pairs = MODE == kInLane || (MODE == kAny && a.layout == EXL3_ROPE_PAIRS);
  const bool rotated = e0 < R, second = e0 >= half;
  const int away = second ? -half : half;            // (by lane) the partner elements
  const int partner = rotated ? lane + away / 8 : lane;
  unsigned long long step[D / 64];                   // of frequencies lane, lane + 32, ...
#pragma unroll
  for (int k = 0; k < D / 64; ++k) step[k] = lane + 32 * k < half ? turn_step(a.inv_freq[lane + 32 * k]) : 0;
  // this lane's place in a token's rows, in bytes
  constexpr int kIn = HPP * D * (F32IN ? 4 : 2);     // a pass
  const char *q_in = static_cast<const char *>(a.q) + lane * 8 * (F32IN ? 4 : 2);
  const char *k_in = static_cast<const char *>(a.k) + lane * 8 * (F32IN ? 4 : 2);
  const char *v_in = static_cast<const char *>(a.v) + lane * 8 * (F32IN ? 4 : 2);
  const int64_t q_row = a.q_stride * (F32IN ? 4 : 2), k_row = a.k_stride * (F32IN ? 4 : 2),
                v_row = a.v_stride * (F32IN ? 4 : 2);
  // passes of a kind that have a head for this lane: all, or all but the last
  const int live_q = ps.q - ((ps.q - 1) * HPP + lane / LPH < a.Hq ? 0 : 1);
  const int live_kv = ps.k - ps.q - ((ps.k - ps.q - 1) * HPP + lane / LPH < a.Hkv ? 0 : 1);

  const auto look_up = [&](int b, int index) -> int {          // -1: no such page
    const int i = index / a.page_size;
    return index >= 0 && i < a.max_pages ? a.table[(int64_t)b * a.max_pages + i] : -1;
  };
  const int64_t first = ((int64_t)blockIdx.x * kWarps + warp) * run;
  int left = (int)max(min((int64_t)run, (int64_t)a.T * ps.all - first), (int64_t)0);   // passes still to do
  int t = (int)(first / ps.all), p0 = (int)(first - (int64_t)t * ps.all);
  // the sequence of the token before, its end, what makes rows cache indexes,
  // and the next token's page, looked up during the passes of the one before
  int b = a.B, seq_end = 0, shift = 0, next_page = -1;
  for (; left > 0; ++t, p0 = 0) {
    const int p1 = min(ps.all, p0 + left);
    left -= p1 - p0;
    // the first heads of every kind are under way while the angles are worked out
    const int qa = p0, qb = min(p1, ps.q), ka = max(p0 - ps.q, 0), kb = min(p1, ps.k) - ps.q;
    const int va = max(p0 - ps.k, 0), vb = p1 - ps.k;
    const char *q_src = q_in + t * q_row + (int64_t)qa * kIn, *k_src = k_in + t * k_row + (int64_t)ka * kIn,
               *v_src = v_in + t * v_row + (int64_t)va * kIn;
    const auto load_if = [&](bool ok, const char *p) -> Raw8<F32IN> {
      if (ok) return load_raw<F32IN>(p, 0);
      return Raw8<F32IN>{};
    };
    const Raw8<F32IN> q0 = load_if(qa < min(qb, live_q), q_src), k0 = load_if(ka < min(kb, live_kv), k_src),
                      v0 = load_if(APPEND && va < min(vb, live_kv), v_src);

    int index = 0, page = -1, off = 0;               // cache index (negative: padding) and place
    if (APPEND) {
      if (t >= seq_end) {
        b = find_seq(a.q_start, a.B, t, lane);
        seq_end = t;                                 // (of no sequence: look again for the next token)
        if (b < a.B) {
          seq_end = a.q_start[b + 1];
          shift = a.kv_len[b] - seq_end;
          next_page = look_up(b, t + shift);
        }
      }
      index = -1;
      if (b < a.B) {
        index = t + shift;
        page = next_page;
        off = index % a.page_size;
        if ((unsigned)page >= (unsigned)a.num_pages) {
          if (lane == 0) set_device_error(a.err, kErrBounds);
          page = -1;
        }
        if (left > 0 && t + 1 < seq_end) next_page = look_up(b, index + 1);
      }
    }
    const int pos = a.positions ? a.positions[t] : index;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < D / 64; ++k) {
      const int f = lane + 32 * k;
      if (f < half) {
        float si, co;
        sincospif(half_turns(pos, step[k]), &si, &co);
        cs[f] = make_float2(co * a.magnitude, si * a.magnitude);
      }
    }
    __syncwarp();
    // out = r (own * own_w + partner * partner_w): the norm weight of each
    // element times its cosine or sine, for one kind of head at a time
    float own_w[8], partner_w[8];
    const auto set_weights = [&](const void *norm) {
      Row8 w, wp;
#pragma unroll
      for (int j = 0; j < 8; ++j) w.v[j] = wp.v[j] = 1.0f;
      if (norm) w = unpack<false>(load_raw<false>(norm, e0));
      if constexpr (MODE != kAny) {
        if (rotated) {
          if (MODE == kByLane && norm) wp = unpack<false>(load_raw<false>(norm, e0 + away));
          const float4 *tab = reinterpret_cast<const float4 *>(cs + (MODE == kInLane ? e0 / 2 : second ? e0 - half : e0));
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            if (MODE == kInLane && (j & 3)) continue;
            const float4 t = tab[MODE == kInLane ? j / 4 : j / 2];
            if constexpr (MODE == kByLane) {
              const float sg = second ? 1.0f : -1.0f;
              own_w[j] = w.v[j] * t.x;
              own_w[j + 1] = w.v[j + 1] * t.z;
              partner_w[j] = sg * t.y * wp.v[j];
              partner_w[j + 1] = sg * t.w * wp.v[j + 1];
            } else {
              own_w[j] = w.v[j] * t.x;
              own_w[j + 1] = w.v[j + 1] * t.x;
              own_w[j + 2] = w.v[j + 2] * t.z;
              own_w[j + 3] = w.v[j + 3] * t.z;
              partner_w[j] = -t.y * w.v[j + 1];
              partner_w[j + 1] = t.y * w.v[j];
              partner_w[j + 2] = -t.w * w.v[j + 3];
              partner_w[j + 3] = t.w * w.v[j + 2];
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) own_w[j] = w.v[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = e0 + j, m = pairs ? e ^ 1 : e >= half ? e - half : e + half;
          const float2 t = e < R ? cs[pairs ? e / 2 : e >= half ? e - half : e] : make_float2(1.0f, 0.0f);
          const float v = norm && e < R ? __half2float(static_cast<const __half *>(norm)[m]) : 1.0f;
          own_w[j] = w.v[j] * t.x;
          partner_w[j] = ((pairs ? j & 1 : e >= half) ? t.y : -t.y) * v;
        }
      }
    };
    // Passes pa .. pb - 1 of one kind, kAhead loads ahead of the arithmetic.
    const auto walk = [&](int pa, int pb, int live, const char *src, Raw8<F32IN> raw, char *dst, int64_t step,
                          bool f32out, bool norm, bool zero, bool write) {
      const int end = min(pb, live);
      constexpr int AHEAD = kAhead<F32IN>, UNROLL = kUnroll<F32IN>;
      Raw8<F32IN> ahead[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) ahead[k] = load_if(pa + 1 + k < end, src + (k + 1) * kIn);
      src += (AHEAD + 1) * kIn;
#pragma unroll UNROLL
      for (int p = pa; p < pb; ++p, src += kIn, dst += step) {
        Row8 o = unpack<F32IN>(raw);
        raw = ahead[0];
#pragma unroll
        for (int k = 0; k + 1 < AHEAD; ++k) ahead[k] = ahead[k + 1];
        ahead[AHEAD - 1] = load_if(p + 1 + AHEAD < end, src);
        float r = 1.0f;
        if (norm) {
          float ss = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) ss = fmaf(o.v[j], o.v[j], ss);
#pragma unroll
          for (int m = 1; m < LPH; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
          r = rsqrtf(ss * (1.0f / D) + a.eps);
        }
        if constexpr (MODE == kInLane) {
          if (rotated) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = o.v[j ^ 1];
#pragma unroll
            for (int j = 0; j < 8; ++j) o.v[j] = fmaf(x[j], partner_w[j], o.v[j] * own_w[j]) * r;
          }
        } else if constexpr (MODE == kByLane) {
          float x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = __shfl_sync(0xffffffffu, o.v[j], partner);
          if (rotated) {
#pragma unroll
            for (int j = 0; j < 8; ++j) o.v[j] = fmaf(x[j], partner_w[j], o.v[j] * own_w[j]) * r;
          }
        } else {
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) stage[lane][j] = o.v[j];
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int e = e0 + j, m = e >= R ? e : pairs ? e ^ 1 : e < half ? e + half : e - half;
            const float y = o.v[j] * own_w[j], x = stage[lane - c + m / 8][m % 8];
            o.v[j] = (e < R ? fmaf(x, partner_w[j], y) : y) * r;
          }
        }
        if (MODE != kAny && !rotated) {
#pragma unroll
          for (int j = 0; j < 8; ++j) o.v[j] *= own_w[j] * r;
        }
        if (APPEND && zero) o = Row8{};
        if (p < live && write) store8(dst, 0, o, f32out);
      }
    };
    const bool f32out = !APPEND && a.f32out;
    const int osz = f32out ? 4 : 2;
    const bool place = !APPEND || page >= 0;
    const int64_t cache_at = APPEND ? (int64_t)page * a.stride_page + (int64_t)off * a.stride_token + e0 : 0;
    const int64_t cache_step = HPP * a.stride_head * 2;
    if (qa < qb) {
      set_weights(a.q_norm);
      walk(qa, qb, live_q, q_src, q0,
           static_cast<char *>(a.q_out) + ((int64_t)t * a.Hq * D + (int64_t)qa * (HPP * D) + lane * 8) * osz,
           HPP * D * osz, f32out, a.q_norm != nullptr, index < 0, true);
    }
    if (ka < kb) {
      set_weights(a.k_norm);
      char *dst = APPEND ? static_cast<char *>(a.k_cache) + (cache_at + (ka * HPP + lane / LPH) * a.stride_head) * 2
                         : static_cast<char *>(a.k_out) +
                               ((int64_t)t * a.Hkv * D + (int64_t)ka * (HPP * D) + lane * 8) * osz;
      walk(ka, kb, live_kv, k_src, k0, dst, APPEND ? cache_step : HPP * D * osz, f32out, a.k_norm != nullptr, false,
           place);
    }
    if (APPEND && va < vb) {                           // values go as they are
      char *dst = static_cast<char *>(a.v_cache) + (cache_at + (va * HPP + lane / LPH) * a.stride_head) * 2;
      Raw8<F32IN> raw = v0;
      for (int p = va; p < vb; ++p, dst += cache_step) {
        v_src += kIn;
        const Raw8<F32IN> next = load_if(p + 1 < min(vb, live_kv), v_src);
        if (p < live_kv && place) {
          if constexpr (F32IN) store8(dst, 0, unpack<F32IN>(raw), false);
          else *reinterpret_cast<uint4 *>(dst) = raw.u[0];
        }
        raw = next;
      }
    }
  }
}

template <int D, bool F32IN, bool APPEND>
cudaError_t launch(const Args &a, cudaStream_t s) {
  const int passes = count_passes(a.Hq, a.Hkv, 32 / (D / 8), APPEND).all;
  const int64_t total = (int64_t)a.T * passes, warps = (int64_t)exl3_sm_count() * kCtas * kWarps;
  const int run = (int)((total + warps - 1) / warps);
  const int64_t grid = (total + (int64_t)run * kWarps - 1) / ((int64_t)run * kWarps);
  const dim3 g((unsigned)grid), b(kThreads);
  const bool pairs = a.layout == EXL3_ROPE_PAIRS;
  if (pairs ? a.rotary_dim == 0 : a.rotary_dim % 16 == 0)
    return launch_pdl(head_transform_kernel<D, F32IN, APPEND, kByLane>, g, b, 0, s, a, run);
  if (pairs && a.rotary_dim % 8 == 0)
    return launch_pdl(head_transform_kernel<D, F32IN, APPEND, kInLane>, g, b, 0, s, a, run);
  return launch_pdl(head_transform_kernel<D, F32IN, APPEND, kAny>, g, b, 0, s, a, run);
}

template <bool F32IN, bool APPEND>
cudaError_t by_dim(const Args &a, int D, cudaStream_t s) {
  switch (D) {
    case 64: return launch<64, F32IN, APPEND>(a, s);
    case 128: return launch<128, F32IN, APPEND>(a, s);
    default: return launch<256, F32IN, APPEND>(a, s);
  }
}

}  // namespace ht
}  // namespace exl3

cudaError_t exl3_launch_head_transform(const exl3::ht::Args &a, int D, bool f32in, bool append, cudaStream_t s) {
  using namespace exl3::ht;
  if (append) return f32in ? by_dim<true, true>(a, D, s) : by_dim<false, true>(a, D, s);
  return f32in ? by_dim<true, false>(a, D, s) : by_dim<false, false>(a, D, s);
}
