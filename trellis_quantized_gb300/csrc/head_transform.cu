// head_transform.cu -- norms of query and key heads with the rotary position
// rotation in one pass, and the same with an append to a paged cache.
//
//   n = x * rsqrt(mean(x^2) + eps) * w                       (per head)
//   (a, b) -> magnitude * (a cos t - b sin t, b cos t + a sin t)
//
// Both calls are bound by memory: each input is read once and each output
// written once, 2 to 4 bytes either way against about seven operations an
// element.  A CTA takes one token; a thread holds eight neighbouring elements
// (16 bytes of fp16) of a head, so D / 8 lanes hold a head, the mean is a few
// shuffles, and the thread keeps its place in the head while the CTA walks
// over the token's heads: the norm weights and the eight cosines and sines of
// its elements stay in registers.  They come from a table that the CTA fills
// once per token.
//
// Angles.  A position times a frequency has to be known to a fraction of a
// turn however far the position is.  The frequency in turns (f / 2 pi, one
// double-precision product) is held as a 64-bit fixed-point fraction; its
// product with the int32 position, modulo 2^64, is the angle modulo a turn
// with an error below |position| * 2^-55 turns, and its upper 32 bits go to
// sincospif.  No reduction of a large argument is left to do.
#include "exl3_common.cuh"
#include "head_transform.cuh"

namespace exl3 {
namespace ht {

constexpr int kThreads = 256;

// The upper 32 bits of position * f as a fraction of a turn, in half turns.
__device__ __forceinline__ float half_turns(int pos, float freq) {
  constexpr double kInv2Pi = 0.15915494309189533577;
  double t = (double)freq * kInv2Pi;
  t -= floor(t);
  const unsigned long long step = (unsigned long long)(t * 18446744073709551616.0);   // * 2^64, t < 1
  const unsigned long long ang = step * (unsigned long long)(long long)pos;
  return (float)(int)(unsigned)(ang >> 32) * 4.656612873077393e-10f;                  // * 2^-31: [-1, 1]
}

struct Row8 {
  float v[8];
};

template <bool F32>
__device__ __forceinline__ Row8 load8(const void *base, int64_t i) {
  Row8 r;
  if (F32) {
    const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + i);
    const float4 x = p[0], y = p[1];
    r.v[0] = x.x; r.v[1] = x.y; r.v[2] = x.z; r.v[3] = x.w;
    r.v[4] = y.x; r.v[5] = y.y; r.v[6] = y.z; r.v[7] = y.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const __half *>(base) + i);
    const __half2 *h = reinterpret_cast<const __half2 *>(&u);
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

template <int D, bool F32IN, bool APPEND>
__global__ void __launch_bounds__(kThreads) head_transform_kernel(const Args a) {
  constexpr int LPH = D / 8;               // lanes per head
  constexpr int HPP = kThreads / LPH;      // heads per pass of the CTA
  __shared__ float2 cs[D / 2];
  __shared__ float stage[kThreads][9];     // half layout with an odd number of eights: partners through here
  __shared__ int place[3];                 // position, page (-1: not appended), offset in the page

  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  const int c = tid % LPH, e0 = 8 * c;     // this thread's eight elements of its heads
  const int h0 = blockIdx.y * HPP + tid / LPH, hstep = gridDim.y * HPP;
  const int nheads = a.Hq + a.Hkv + (APPEND ? a.Hkv : 0);
  const int R = a.rotary_dim, half = R / 2;
  pdl_trigger();
  pdl_wait();

  const auto load_head = [&](int h) -> Row8 {
    if (h < a.Hq) return load8<F32IN>(a.q, (int64_t)t * a.q_stride + (int64_t)h * D + e0);
    if (h < a.Hq + a.Hkv) return load8<F32IN>(a.k, (int64_t)t * a.k_stride + (int64_t)(h - a.Hq) * D + e0);
    return load8<F32IN>(a.v, (int64_t)t * a.v_stride + (int64_t)(h - a.Hq - a.Hkv) * D + e0);
  };
  // the first head's data is under way while the angles are worked out
  Row8 x;
  if (h0 < nheads) x = load_head(h0);

  if (APPEND && tid < 32) {
    const int b = find_seq(a.q_start, a.B, t, lane);
    if (lane == 0) {
      int pos = -1, page = -1, off = 0;
      if (b < a.B) {
        pos = a.kv_len[b] - (a.q_start[b + 1] - t);
        const int i = pos < 0 ? a.max_pages : pos / a.page_size;
        if (i < a.max_pages) {
          page = a.table[(int64_t)b * a.max_pages + i];
          off = pos - i * a.page_size;
        }
        if ((unsigned)page >= (unsigned)a.num_pages) {
          set_device_error(a.err, kErrBounds);
          page = -1;
        }
      }
      place[0] = pos;
      place[1] = page;
      place[2] = off;
    }
  }
  if (APPEND) __syncthreads();
  const int index = APPEND ? place[0] : 0;           // cache index; negative: padding
  if (tid < half) {
    const int pos = a.positions ? a.positions[t] : index;
    float s, co;
    sincospif(half_turns(pos, a.inv_freq[tid]), &s, &co);
    cs[tid] = make_float2(co * a.magnitude, s * a.magnitude);
  }
  __syncthreads();

  // where this thread's elements stand in the rotation
  const bool pairs = a.layout == EXL3_ROPE_PAIRS;
  const bool by_lane = !pairs && half % 8 == 0;      // half layout, partners eight by eight
  const bool by_smem = !pairs && R > 0 && half % 8 != 0;
  const bool second = e0 >= half;                    // (by_lane) upper element of its pairs
  const bool rotated = e0 < R;
  const int partner = (lane - c % 32) + (c + (second ? -half : half) / 8) % 32;   // (by_lane) lane of the other eight
  float co[8], si[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    int i;
    if (pairs) i = (e0 + j) / 2;
    else i = (e0 + j) % (half > 0 ? half : 1);
    const bool in = e0 + j < R;
    const float2 w = in ? cs[i] : make_float2(1.0f, 0.0f);
    co[j] = w.x;
    // out = own * co + partner * si
    const bool upper = pairs ? (j & 1) : (e0 + j >= half);
    si[j] = upper ? w.y : -w.y;
  }
  Row8 wq, wk;
  if (a.q_norm) wq = load8<false>(a.q_norm, e0);
  if (a.k_norm) wk = load8<false>(a.k_norm, e0);

  for (int hb = blockIdx.y * HPP; hb < nheads; hb += hstep) {
    const int h = hb + tid / LPH;
    const bool live = h < nheads;
    const bool isq = h < a.Hq, isk = !isq && h < a.Hq + a.Hkv;
    Row8 nx;
    if (h + hstep < nheads) nx = load_head(h + hstep);
    if (!live) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x.v[j] = 0.0f;
    }
    const bool norm = isq ? a.q_norm != nullptr : (isk && a.k_norm != nullptr);
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(x.v[j], x.v[j], ss);
#pragma unroll
    for (int m = 1; m < LPH; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    Row8 o = x;
    if (norm) {
      const float r = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
      for (int j = 0; j < 8; ++j) o.v[j] = x.v[j] * r * (isq ? wq.v[j] : wk.v[j]);
    }
    Row8 p;                                          // the partner of each element
    if (pairs) {
#pragma unroll
      for (int j = 0; j < 8; ++j) p.v[j] = o.v[j ^ 1];
    } else if (by_lane) {
#pragma unroll
      for (int j = 0; j < 8; ++j) p.v[j] = __shfl_sync(0xffffffffu, o.v[j], rotated ? partner : lane);
    } else if (by_smem) {
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j) stage[tid][j] = o.v[j];
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = e0 + j;
        const int q = e < half ? e + half : (e < R ? e - half : e);
        p.v[j] = stage[tid - c + q / 8][q % 8];
      }
    } else {
      p = o;
    }
    if (isq || isk) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (e0 + j < R) o.v[j] = fmaf(o.v[j], co[j], p.v[j] * si[j]);
    }
    if (live) {
      if (isq) {
        if (APPEND && index < 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j) o.v[j] = 0.0f;
        }
        store8(a.q_out, ((int64_t)t * a.Hq + h) * D + e0, o, !APPEND && a.f32out);
      } else if (!APPEND) {
        store8(a.k_out, ((int64_t)t * a.Hkv + (h - a.Hq)) * D + e0, o, a.f32out);
      } else if (place[1] >= 0) {
        const int hk = isk ? h - a.Hq : h - a.Hq - a.Hkv;
        const int64_t at = (int64_t)place[1] * a.stride_page + (int64_t)place[2] * a.stride_token +
                           (int64_t)hk * a.stride_head + e0;
        store8(isk ? a.k_cache : a.v_cache, at, o, false);
      }
    }
    x = nx;
  }
}

template <int D, bool F32IN, bool APPEND>
cudaError_t launch(const Args &a, cudaStream_t s) {
  constexpr int HPP = kThreads / (D / 8);
  const int heads = a.Hq + a.Hkv + (APPEND ? a.Hkv : 0);
  const int passes = ceil_div(heads, HPP);
  // few tokens: a CTA for every pass over the heads
  const int gy = a.T >= 4 * exl3_sm_count() ? 1 : passes;
  return launch_pdl(head_transform_kernel<D, F32IN, APPEND>, dim3(a.T, gy), dim3(kThreads), 0, s, a);
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
