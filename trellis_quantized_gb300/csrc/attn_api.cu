// attn_api.cu -- the C entry points of the attention operators: argument
// checks, tensor maps, workspace layout and the choice of the kernel.
#include <cmath>
#include <numeric>

#include "api_util.cuh"
#include "attn_common.cuh"
#include "exl3_common.cuh"
#include "head_transform.cuh"

// ---- kernels (other translation units)
int exl3_attn_step_rows();
int exl3_attn_step_keys();
int exl3_attn_step_grid(int D);
cudaError_t exl3_launch_attn_step(const CUtensorMap &mk, const CUtensorMap &mv, const exl3::attn::Args &a, int D,
                                  cudaStream_t s);
int exl3_attn_tc_rows(int D);
int exl3_attn_tc_keys();
int exl3_attn_tc_grid();
cudaError_t exl3_launch_attn_tc(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                                const exl3::attn::Args &a, int D, cudaStream_t s);
cudaError_t exl3_launch_attn_join(const exl3::attn::Args &a, int D, int ctas, int tile_rows, cudaStream_t s);

namespace {

constexpr double kPi = 3.14159265358979323846;

int check_int_ptr(const void *p, const char *name) {
  if (!p) return exl3_fail(EXL3_ERR_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) & 3u) return exl3_fail(EXL3_ERR_ARG, "%s is not 4-byte aligned", name);
  return EXL3_OK;
}

int check_heads(int T, int heads_q, int heads_kv, int head_dim) {
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return exl3_fail(EXL3_ERR_SHAPE, "head_dim = %d is not 64, 128 or 256", head_dim);
  if (T < 0 || heads_q < 1 || heads_q > 65536 || heads_kv < 0 || heads_kv > 65536)
    return exl3_fail(EXL3_ERR_SHAPE, "T = %d, heads_q = %d, heads_kv = %d out of range", T, heads_q, heads_kv);
  return EXL3_OK;
}

// Rows of `heads` dense heads, `stride` elements apart.
int check_rows(const void *p, const char *name, int64_t stride, int heads, int head_dim, int dtype) {
  EXL3_TRY(check_ptr(p, name));
  const int64_t per16 = dtype == EXL3_OUT_F32 ? 4 : 8;
  if (stride < (int64_t)heads * head_dim || stride % per16 || stride > ((int64_t)1 << 40))
    return exl3_fail(EXL3_ERR_SHAPE, "%s: stride %lld must be a multiple of 16 bytes and hold %d heads of %d", name,
                     (long long)stride, heads, head_dim);
  return EXL3_OK;
}

int check_dtype(int dtype, const char *name) {
  if (dtype != EXL3_OUT_F16 && dtype != EXL3_OUT_F32) return exl3_fail(EXL3_ERR_ARG, "%s %d invalid", name, dtype);
  return EXL3_OK;
}

int check_transform(const exl3_head_transform *t, int head_dim) {
  if (!t) return exl3_fail(EXL3_ERR_ARG, "transform is NULL");
  EXL3_TRY(check_ptr(t->q_norm, "q_norm", false));
  EXL3_TRY(check_ptr(t->k_norm, "k_norm", false));
  if (t->rotary_dim < 0 || t->rotary_dim > head_dim || t->rotary_dim % 2)
    return exl3_fail(EXL3_ERR_SHAPE, "rotary_dim = %d must be even and within 0..%d", t->rotary_dim, head_dim);
  if (t->rotary_dim > 0) EXL3_TRY(check_int_ptr(t->inv_freq, "inv_freq"));
  if (t->layout != EXL3_ROPE_HALF && t->layout != EXL3_ROPE_PAIRS)
    return exl3_fail(EXL3_ERR_ARG, "layout %d invalid", t->layout);
  if (!(t->eps >= 0.0f) || !std::isfinite(t->eps) || !std::isfinite(t->magnitude))
    return exl3_fail(EXL3_ERR_ARG, "eps must be >= 0, eps and magnitude finite");
  return EXL3_OK;
}

int check_batch(const exl3_paged_batch *b, const exl3_kv_cache *c) {
  if (!b) return exl3_fail(EXL3_ERR_ARG, "batch is NULL");
  if (!c) return exl3_fail(EXL3_ERR_ARG, "cache is NULL");
  EXL3_TRY(check_int_ptr(b->q_start, "q_start"));
  EXL3_TRY(check_int_ptr(b->kv_len, "kv_len"));
  EXL3_TRY(check_int_ptr(b->page_table, "page_table"));
  EXL3_TRY(check_ptr(c->k, "cache.k"));
  EXL3_TRY(check_ptr(c->v, "cache.v"));
  if (b->batch < 1 || b->batch > (1 << 20) || b->max_pages < 1)
    return exl3_fail(EXL3_ERR_SHAPE, "batch = %d (1..2^20) or max_pages = %d out of range", b->batch, b->max_pages);
  if (c->num_pages < 1 || c->page_size < 16 || c->page_size % 16)
    return exl3_fail(EXL3_ERR_SHAPE, "num_pages = %d must be positive and page_size = %d a multiple of 16",
                     c->num_pages, c->page_size);
  if ((int64_t)b->max_pages * c->page_size > ((int64_t)1 << 30))
    return exl3_fail(EXL3_ERR_SHAPE, "max_pages * page_size = %lld above 2^30",
                     (long long)b->max_pages * c->page_size);
  if (c->heads_kv < 1) return exl3_fail(EXL3_ERR_SHAPE, "cache.heads_kv = %d < 1", c->heads_kv);
  const int64_t lim = (int64_t)1 << 39;   // a tensor map's strides end at 2^40 bytes
  for (int64_t st : {c->stride_page, c->stride_token, c->stride_head})
    if (st <= 0 || st % 8 || st >= lim)
      return exl3_fail(EXL3_ERR_SHAPE, "cache stride %lld must be a positive multiple of 8 elements below 2^39",
                       (long long)st);
  if (c->stride_token < c->head_dim || c->stride_head < c->head_dim)
    return exl3_fail(EXL3_ERR_SHAPE, "cache strides overlap: token %lld, head %lld, head_dim %d",
                     (long long)c->stride_token, (long long)c->stride_head, c->head_dim);
  return EXL3_OK;
}

// Tensor map of a cache: 64-element columns by `box` tokens of one head and
// page, 128-byte swizzle; the smaller of the token and head strides first.
int cache_map(CUtensorMap *m, const exl3_kv_cache *c, const void *base, int box, bool head_first) {
  auto fn = exl3_tmap_encode_fn();
  if (!fn) return exl3_fail(EXL3_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const cuuint64_t tok = (cuuint64_t)c->stride_token * 2, head = (cuuint64_t)c->stride_head * 2;
  cuuint64_t dims[4] = {(cuuint64_t)c->head_dim, (cuuint64_t)c->page_size, (cuuint64_t)c->heads_kv,
                        (cuuint64_t)c->num_pages};
  cuuint64_t strides[3] = {tok, head, (cuuint64_t)c->stride_page * 2};
  cuuint32_t bx[4] = {64, (cuuint32_t)box, 1, 1};
  if (head_first) {
    std::swap(dims[1], dims[2]);
    std::swap(strides[0], strides[1]);
    std::swap(bx[1], bx[2]);
  }
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void *>(base), dims, strides, bx, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return exl3_fail(EXL3_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return EXL3_OK;
}

// Few rows per sequence and key head take the step kernel (16 rows a unit),
// more the tensor-core kernel (128 rows a tile): 64 sequences of 4 tokens (20
// rows) behind 4,000 at 40/8 heads of 128 take 188 us there and 331 us in units
// of 16, 3 tokens (15 rows) 181 us.  The host knows the average only: one chunk
// among many steps runs in units of 16 as well (63 steps and 141 tokens behind
// 30,000: 592 us, as two calls 118 and 89).
bool few_rows(int T, int G, int batch) {
  return G <= exl3_attn_step_rows() && (int64_t)T * G <= (int64_t)exl3_attn_step_rows() * batch;
}

// Tensor map of the queries: G heads of `tokens` tokens, 64 columns, 128-byte
// swizzle.
int query_map(CUtensorMap *m, const void *q, int64_t stride, int T, int heads, int D, int G, int tokens) {
  auto fn = exl3_tmap_encode_fn();
  if (!fn) return exl3_fail(EXL3_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)T};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)tokens};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(q), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return exl3_fail(EXL3_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return EXL3_OK;
}

// ---- exl3_paged_attention workspace layout: a record per CTA of the unit
// that it leaves unfinished, and two partial results per CTA
struct AttnWs {
  size_t cuts = 0, part_o = 0, part_ml = 0, total = 0;
  int grid = 0, rows = 0;
};

AttnWs attn_ws(int T, int G, int D, int batch) {
  AttnWs w;
  const bool few = few_rows(T, G, batch);
  w.grid = few ? exl3_attn_step_grid(D) : exl3_attn_tc_grid();
  w.rows = few ? exl3_attn_step_rows() : exl3_attn_tc_rows(D);
  const size_t rows = (size_t)w.grid * 2 * w.rows;
  size_t off = kDataOff;
  w.cuts = off;
  off = align_up(off + sizeof(exl3::attn::Cut) * w.grid);
  w.part_o = off;
  off = align_up(off + sizeof(float) * rows * D);
  w.part_ml = off;
  off = align_up(off + sizeof(float2) * rows);
  w.total = off;
  return w;
}

bool attn_shape_ok(int T, int heads_q, int heads_kv, int D, int batch) {
  return (D == 64 || D == 128 || D == 256) && T >= 0 && heads_kv >= 1 && heads_q >= heads_kv && heads_q <= 65536 &&
         heads_q % heads_kv == 0 && heads_q / heads_kv <= 128 && batch >= 1 && batch <= (1 << 20) && (int64_t)T * heads_q <= INT32_MAX;
}

}  // namespace

extern "C" {

int exl3_rope_frequencies(int rotary_dim, double base, int scaling, double factor, int original_len, double low,
                          double high, float *inv_freq, float *magnitude) {
  exl3_clear_error();
  const int R = rotary_dim;
  if (!inv_freq || !magnitude) return exl3_fail(EXL3_ERR_ARG, "inv_freq or magnitude is NULL");
  if (scaling < EXL3_ROPE_NONE || scaling > EXL3_ROPE_YARN)
    return exl3_fail(EXL3_ERR_ARG, "unknown rope scaling %d", scaling);
  if (R < 2 || R % 2 || (scaling == EXL3_ROPE_NTK && R < 4))
    return exl3_fail(EXL3_ERR_SHAPE, "rotary_dim = %d must be even and >= 2 (NTK: 4)", R);
  if (!(base > 1.0) || !std::isfinite(base)) return exl3_fail(EXL3_ERR_ARG, "base must be > 1 and finite");
  if (scaling != EXL3_ROPE_NONE && (!(factor > 0.0) || !std::isfinite(factor)))
    return exl3_fail(EXL3_ERR_ARG, "factor must be > 0 and finite");
  const bool parts = scaling == EXL3_ROPE_BANDS || scaling == EXL3_ROPE_YARN;
  if (parts && (original_len < 1 || !(low > 0.0) || !(high > low) || !std::isfinite(high)))
    return exl3_fail(EXL3_ERR_ARG, "original_len = %d must be >= 1 and 0 < low < high", original_len);
  if (scaling == EXL3_ROPE_NTK) base *= std::pow(factor, (double)R / (R - 2));
  double first = 0, last = 0;
  if (scaling == EXL3_ROPE_YARN) {
    const auto place = [&](double n) { return R * std::log(original_len / (2 * kPi * n)) / (2 * std::log(base)); };
    first = std::fmax(0.0, std::floor(place(high)));
    last = std::fmin(R - 1.0, std::ceil(place(low)));
  }
  for (int i = 0; i < R / 2; ++i) {
    double f = std::pow(base, -2.0 * i / R);
    double keep = 1.0;
    if (scaling == EXL3_ROPE_LINEAR) keep = 0.0;
    if (scaling == EXL3_ROPE_BANDS) keep = (original_len * f / (2 * kPi) - low) / (high - low);
    if (scaling == EXL3_ROPE_YARN) keep = 1.0 - std::fmin(std::fmax((i - first) / std::fmax(last - first, 0.001), 0.0), 1.0);
    keep = std::fmin(std::fmax(keep, 0.0), 1.0);
    if (scaling == EXL3_ROPE_LINEAR || parts) f = keep * f + (1.0 - keep) * f / factor;
    inv_freq[i] = (float)f;
  }
  *magnitude = scaling == EXL3_ROPE_YARN && factor > 1.0 ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  return EXL3_OK;
}

int exl3_qk_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride, int in_dtype, int T,
                      int heads_q, int heads_kv, int head_dim, const exl3_head_transform *transform,
                      const int32_t *positions, void *q_out, void *k_out, int out_dtype, exl3_stream_t stream) {
  exl3_clear_error();
  EXL3_TRY(check_dtype(in_dtype, "in_dtype"));
  EXL3_TRY(check_dtype(out_dtype, "out_dtype"));
  EXL3_TRY(check_heads(T, heads_q, heads_kv, head_dim));
  EXL3_TRY(check_transform(transform, head_dim));
  EXL3_TRY(check_rows(q, "q", q_stride, heads_q, head_dim, in_dtype));
  EXL3_TRY(check_ptr(q_out, "q_out"));
  if (heads_kv > 0) {
    EXL3_TRY(check_rows(k, "k", k_stride, heads_kv, head_dim, in_dtype));
    EXL3_TRY(check_ptr(k_out, "k_out"));
  }
  if (transform->rotary_dim > 0) EXL3_TRY(check_int_ptr(positions, "positions"));
  if (T == 0) return EXL3_OK;
  exl3::ht::Args a = {};
  a.q = q;
  a.k = k;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.T = T;
  a.Hq = heads_q;
  a.Hkv = heads_kv;
  a.q_norm = transform->q_norm;
  a.k_norm = transform->k_norm;
  a.eps = transform->eps;
  a.magnitude = transform->magnitude;
  a.inv_freq = transform->inv_freq;
  a.rotary_dim = transform->rotary_dim;
  a.layout = transform->layout;
  a.positions = positions;
  a.q_out = q_out;
  a.k_out = k_out;
  a.f32out = out_dtype == EXL3_OUT_F32;
  return exl3_cuda_check(exl3_launch_head_transform(a, head_dim, in_dtype == EXL3_OUT_F32, false, stream),
                         "head transform launch");
}

size_t exl3_qkv_append_workspace_size(void) { return kCtrlBytes; }

int exl3_qkv_append(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                    int64_t v_stride, int in_dtype, int T, int heads_q, const exl3_head_transform *transform,
                    const int32_t *positions, const exl3_paged_batch *batch, const exl3_kv_cache *cache,
                    uint16_t *q_out, void *workspace, size_t ws_bytes, exl3_stream_t stream) {
  exl3_clear_error();
  EXL3_TRY(check_dtype(in_dtype, "in_dtype"));
  EXL3_TRY(check_batch(batch, cache));
  EXL3_TRY(check_heads(T, heads_q, cache->heads_kv, cache->head_dim));
  EXL3_TRY(check_transform(transform, cache->head_dim));
  EXL3_TRY(check_rows(q, "q", q_stride, heads_q, cache->head_dim, in_dtype));
  EXL3_TRY(check_rows(k, "k", k_stride, cache->heads_kv, cache->head_dim, in_dtype));
  EXL3_TRY(check_rows(v, "v", v_stride, cache->heads_kv, cache->head_dim, in_dtype));
  EXL3_TRY(check_ptr(q_out, "q_out"));
  if (positions) EXL3_TRY(check_int_ptr(positions, "positions"));
  EXL3_TRY(check_workspace(workspace, ws_bytes, kCtrlBytes));
  if (T == 0) return EXL3_OK;
  exl3::ht::Args a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.T = T;
  a.Hq = heads_q;
  a.Hkv = cache->heads_kv;
  a.q_norm = transform->q_norm;
  a.k_norm = transform->k_norm;
  a.eps = transform->eps;
  a.magnitude = transform->magnitude;
  a.inv_freq = transform->inv_freq;
  a.rotary_dim = transform->rotary_dim;
  a.layout = transform->layout;
  a.positions = positions;
  a.q_out = q_out;
  a.q_start = batch->q_start;
  a.kv_len = batch->kv_len;
  a.table = batch->page_table;
  a.B = batch->batch;
  a.max_pages = batch->max_pages;
  a.page_size = cache->page_size;
  a.num_pages = cache->num_pages;
  a.k_cache = cache->k;
  a.v_cache = cache->v;
  a.stride_page = cache->stride_page;
  a.stride_token = cache->stride_token;
  a.stride_head = cache->stride_head;
  a.err = at<int>(workspace, 0);
  return exl3_cuda_check(exl3_launch_head_transform(a, cache->head_dim, in_dtype == EXL3_OUT_F32, true, stream),
                         "append launch");
}

size_t exl3_paged_attention_workspace_size(int T, int heads_q, int heads_kv, int head_dim, int batch) {
  if (!attn_shape_ok(T, heads_q, heads_kv, head_dim, batch)) return 0;
  return attn_ws(T, heads_q / heads_kv, head_dim, batch).total;
}

int exl3_paged_attention(const uint16_t *q, int64_t q_stride, int T, int heads_q, const exl3_paged_batch *batch,
                         const exl3_kv_cache *cache, float scale, int causal, int window, void *y, int out_dtype,
                         float *lse, void *workspace, size_t ws_bytes, exl3_stream_t stream) {
  exl3_clear_error();
  EXL3_TRY(check_dtype(out_dtype, "out_dtype"));
  EXL3_TRY(check_batch(batch, cache));
  EXL3_TRY(check_heads(T, heads_q, cache->heads_kv, cache->head_dim));
  if (!attn_shape_ok(T, heads_q, cache->heads_kv, cache->head_dim, batch->batch))
    return exl3_fail(EXL3_ERR_SHAPE,
                     "heads_q = %d must be a multiple of heads_kv = %d, at most 128 times it, and T * heads_q below 2^31",
                     heads_q, cache->heads_kv);
  EXL3_TRY(check_rows(q, "q", q_stride, heads_q, cache->head_dim, EXL3_OUT_F16));
  EXL3_TRY(check_ptr(y, "y"));
  if (lse) EXL3_TRY(check_int_ptr(lse, "lse"));
  if (!(scale > 0.0f) || !std::isfinite(scale)) return exl3_fail(EXL3_ERR_ARG, "scale must be > 0 and finite");
  if (causal != 0 && causal != 1) return exl3_fail(EXL3_ERR_ARG, "causal %d invalid", causal);
  if (window < 0) return exl3_fail(EXL3_ERR_ARG, "window = %d < 0", window);
  const int D = cache->head_dim, G = heads_q / cache->heads_kv;
  const bool few = few_rows(T, G, batch->batch);
  const AttnWs L = attn_ws(T, G, D, batch->batch);
  EXL3_TRY(check_workspace(workspace, ws_bytes, L.total));
  if (T == 0) return EXL3_OK;
  exl3::attn::Args a = {};
  a.q = reinterpret_cast<const __half *>(q);
  a.q_stride = q_stride;
  a.T = T;
  a.Hq = heads_q;
  a.Hkv = cache->heads_kv;
  a.G = G;
  a.g_inv = G > 1 ? (unsigned)((((uint64_t)1 << 32) + G - 1) / G) : 0u;
  a.tile_tok = (few ? exl3_attn_step_rows() : 128) / G;
  a.unit_tok = few ? a.tile_tok : a.tile_tok * (exl3_attn_tc_rows(D) / 128);
  a.q_start = batch->q_start;
  a.kv_len = batch->kv_len;
  a.table = batch->page_table;
  a.B = batch->batch;
  a.max_pages = batch->max_pages;
  a.page_size = cache->page_size;
  a.num_pages = cache->num_pages;
  const int box = std::gcd(cache->page_size, few ? exl3_attn_step_keys() : exl3_attn_tc_keys());
  while ((1 << a.box_log2) < box) ++a.box_log2;        // (a power of two: a block is)
  a.head_first = cache->stride_head < cache->stride_token;
  a.scale_log2 = scale * 1.44269504088896340736f;
  a.causal = causal;
  // a window that reaches past the page table hides nothing
  a.window = window > batch->max_pages * cache->page_size ? 0 : window;
  a.y = y;
  a.f32out = out_dtype == EXL3_OUT_F32;
  a.y_aligned32 = (reinterpret_cast<uintptr_t>(y) & 31u) == 0;
  a.lse = lse;
  a.part_o = at<float>(workspace, L.part_o);
  a.part_ml = at<float2>(workspace, L.part_ml);
  a.cuts = at<exl3::attn::Cut>(workspace, L.cuts);
  a.err = at<int>(workspace, 0);
  CUtensorMap mk, mv;
  EXL3_TRY(cache_map(&mk, cache, cache->k, box, a.head_first));
  EXL3_TRY(cache_map(&mv, cache, cache->v, box, a.head_first));
  if (few) {
    EXL3_TRY(exl3_cuda_check(exl3_launch_attn_step(mk, mv, a, D, stream), "attention launch"));
  } else {
    CUtensorMap mq;
    EXL3_TRY(query_map(&mq, q, q_stride, T, heads_q, D, G, a.tile_tok));
    EXL3_TRY(exl3_cuda_check(exl3_launch_attn_tc(mq, mk, mv, a, D, stream), "attention launch"));
  }
  return exl3_cuda_check(exl3_launch_attn_join(a, D, L.grid, L.rows, stream), "attention join launch");
}

}  // extern "C"
