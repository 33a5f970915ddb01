// adapter_api.cu -- the C entry points of the low-rank adapters: argument
// checks and the choice of the kernel.
#include "adapter.cuh"
#include "api_util.cuh"

// ---- kernels (other translation units)
cudaError_t exl3_launch_adapter_plan(const exl3::ad::PlanArgs &p, cudaStream_t s);
cudaError_t exl3_launch_adapter_step(const exl3::ad::Args &a, bool f32, cudaStream_t s);
int exl3_launch_adapter_tc(const exl3::ad::Args &a, bool f32, cudaStream_t s);

namespace {

// Tiles of 128 rows from here on, of 16 before: the small tiles read A and B once for
// every 16 rows and their time grows with rank and columns, the large ones start two
// kernels and pass over y at the copy rate.  One prompt, us on small and large tiles:
//   k 5120, n 5120:  rank 16: 2048 rows 16 and 19, 4096 38 and 30;
//                    rank 64: 512 rows 18 and 16, 1536 29 and 19;
//   k 5120, n 17408: rank 16: 768 rows 20 and 18, 1536 43 and 28;
//                    rank 64: 64 rows 15 and 13, 192 23 and 17; rank 128: 64 rows 28 and 15;
//   k 17408, n 5120: rank 16: 1536 rows 24 and 25, 4096 56 and 49; rank 128: 256 rows 30 and 25.
// Rows of many short sequences gather, which costs the large tiles up to twice as much
// (768 rows of rank 16, n 17408: 22 and 36).  Over 1200 such calls the time is 1.03 of
// the better side's; in all of them n is 0.29 k or more.  With fewer columns beside a
// wide input the small tiles, which read all of A for every 16 rows, are kept for too
// long (k 17408, n 128, rank 128: to T = 6472); that was not measured.
// (The small tiles' grid stays within 2^15 tiles: T < 2^18 here.)
bool large_tiles(int T, int R, int n) { return T >= 48 && (int64_t)T * (R + 16) * (R + 16) * n >= (int64_t)1 << 34; }

bool plan_shape_ok(int T, int batch, int count) {
  return T >= 0 && T <= (1 << 22) && batch >= 1 && batch <= (1 << 20) && count >= 1 && count <= exl3::ad::kMaxCount;
}

bool rank_ok(int R) { return R >= 8 && R <= exl3::ad::kMaxRank && R % 8 == 0; }

int check_words(const void *p, const char *name, bool required = true) {
  if (!p) return required ? exl3_fail(EXL3_ERR_ARG, "%s is NULL", name) : EXL3_OK;
  if (reinterpret_cast<uintptr_t>(p) & 3u) return exl3_fail(EXL3_ERR_ARG, "%s is not 4-byte aligned", name);
  return EXL3_OK;
}

// ---- exl3_adapter_add workspace layout: h of all rows in two fp16 parts and
// each row's factor, for calls on large tiles (behind the counters, which
// the linears that share a workspace have to find at zero)
struct AddWs {
  size_t h = kDataOff, back = 0, total = kCtrlBytes;
};

AddWs add_ws(int T, int R) {
  AddWs w;
  w.back = align_up(w.h + (size_t)T * R * 4);
  w.total = align_up(w.back + (size_t)T * 4);
  return w;
}

int check_stride(const char *name, int64_t stride, int width, int per16) {
  if (stride < width || stride % per16 || stride >= ((int64_t)1 << 38))
    return exl3_fail(EXL3_ERR_SHAPE, "%s: stride %lld must be a multiple of 16 bytes, at least %d and below 2^38", name,
                     (long long)stride, width);
  return EXL3_OK;
}

int check_call(const uint16_t *x, int64_t x_stride, const void *y, int64_t y_stride, void *out, int64_t out_stride,
               int dtype, const exl3_adapters *ad, const void *plan, int T, int batch) {
  if (!ad) return exl3_fail(EXL3_ERR_ARG, "adapters is NULL");
  if (dtype != EXL3_OUT_F16 && dtype != EXL3_OUT_F32) return exl3_fail(EXL3_ERR_ARG, "dtype %d invalid", dtype);
  if (!plan_shape_ok(T, batch, ad->count))
    return exl3_fail(EXL3_ERR_SHAPE, "T = %d (0..2^22), batch = %d (1..2^20) or count = %d (1..%d) out of range", T,
                     batch, ad->count, exl3::ad::kMaxCount);
  if (!rank_ok(ad->max_rank))
    return exl3_fail(EXL3_ERR_SHAPE, "max_rank = %d must be a multiple of 8 in 8..%d", ad->max_rank, exl3::ad::kMaxRank);
  if (ad->k < 128 || ad->k % 128 || ad->n < 128 || ad->n % 128 || ad->k > (1 << 20) || ad->n > (1 << 20))
    return exl3_fail(EXL3_ERR_SHAPE, "k = %d and n = %d must be multiples of 128 up to 2^20", ad->k, ad->n);
  EXL3_TRY(check_ptr(ad->a, "adapters.a"));
  EXL3_TRY(check_ptr(ad->b, "adapters.b"));
  EXL3_TRY(check_words(ad->scale, "adapters.scale"));
  EXL3_TRY(check_words(ad->rank, "adapters.rank", false));
  EXL3_TRY(check_ptr(x, "x"));
  EXL3_TRY(check_ptr(y, "y"));
  EXL3_TRY(check_ptr(out, "out"));
  const int per16 = dtype == EXL3_OUT_F32 ? 4 : 8;
  EXL3_TRY(check_stride("x", x_stride, ad->k, 8));
  EXL3_TRY(check_stride("y", y_stride, ad->n, per16));
  EXL3_TRY(check_stride("out", out_stride, ad->n, per16));
  if (out == y && out_stride != y_stride)
    return exl3_fail(EXL3_ERR_SHAPE, "out is y, but their strides differ: %lld and %lld", (long long)out_stride,
                     (long long)y_stride);
  if (!plan) return exl3_fail(EXL3_ERR_ARG, "plan is NULL");
  if (reinterpret_cast<uintptr_t>(plan) & (kAlign - 1))
    return exl3_fail(EXL3_ERR_ARG, "plan is not %zu-byte aligned", kAlign);
  return EXL3_OK;
}

// A checked call; `scratch`: add_ws's parts from h on.
int launch(const uint16_t *x, int64_t x_stride, const void *y, int64_t y_stride, void *out, int64_t out_stride,
           int dtype, const exl3_adapters *ad, const void *plan, int T, int batch, void *workspace, void *scratch,
           exl3_stream_t stream) {
  if (T == 0) return EXL3_OK;
  const exl3::ad::PlanLayout L = exl3::ad::plan_layout(T, batch, ad->count);
  exl3::ad::Args a = {};
  a.x = reinterpret_cast<const __half *>(x);
  a.y = y;
  a.out = out;
  a.x_stride = x_stride;
  a.y_stride = y_stride;
  a.out_stride = out_stride;
  a.a = reinterpret_cast<const __half *>(ad->a);
  a.b = reinterpret_cast<const __half *>(ad->b);
  a.scale = ad->scale;
  a.rank = ad->rank;
  a.N = ad->count;
  a.R = ad->max_rank;
  a.k = ad->k;
  a.n = ad->n;
  a.T = T;
  a.B = batch;
  const auto in_plan = [&](size_t off) { return static_cast<const char *>(plan) + off; };
  a.ctrl = reinterpret_cast<const int *>(in_plan(0));
  a.perm = reinterpret_cast<const int *>(in_plan(L.perm));
  a.err = at<int>(workspace, 0);
  if (large_tiles(T, ad->max_rank, ad->n)) {
    a.tiles = reinterpret_cast<const int4 *>(in_plan(L.tc_tiles));
    a.max_tiles = L.max_tc_tiles;
    a.h = at<__half>(scratch, 0);
    a.back = at<float>(scratch, add_ws(T, ad->max_rank).back - kDataOff);
    return exl3_launch_adapter_tc(a, dtype == EXL3_OUT_F32, stream);
  }
  a.tiles = reinterpret_cast<const int4 *>(in_plan(L.step_tiles));
  a.max_tiles = L.max_step_tiles;
  return exl3_cuda_check(exl3_launch_adapter_step(a, dtype == EXL3_OUT_F32, stream), "adapter launch");
}

}  // namespace

extern "C" {

size_t exl3_adapter_plan_size(int T, int batch, int count) {
  return plan_shape_ok(T, batch, count) ? exl3::ad::plan_layout(T, batch, count).total : 0;
}

int exl3_adapter_plan(const int32_t *q_start, const int32_t *adapter, int T, int batch, int count, void *plan,
                      size_t plan_bytes, exl3_stream_t stream) {
  exl3_clear_error();
  if (!plan_shape_ok(T, batch, count))
    return exl3_fail(EXL3_ERR_SHAPE, "T = %d (0..2^22), batch = %d (1..2^20) or count = %d (1..%d) out of range", T,
                     batch, count, exl3::ad::kMaxCount);
  EXL3_TRY(check_words(q_start, "q_start"));
  EXL3_TRY(check_words(adapter, "adapter"));
  const exl3::ad::PlanLayout L = exl3::ad::plan_layout(T, batch, count);
  EXL3_TRY(check_workspace(plan, plan_bytes, L.total));
  exl3::ad::PlanArgs p = {};
  p.q_start = q_start;
  p.adapter = adapter;
  p.T = T;
  p.B = batch;
  p.N = count;
  p.ctrl = at<int>(plan, 0);
  p.base = at<int>(plan, L.base);
  p.perm = at<int>(plan, L.perm);
  p.step_tiles = at<int4>(plan, L.step_tiles);
  p.tc_tiles = at<int4>(plan, L.tc_tiles);
  p.max_step_tiles = L.max_step_tiles;
  p.max_tc_tiles = L.max_tc_tiles;
  return exl3_cuda_check(exl3_launch_adapter_plan(p, stream), "adapter plan launch");
}

size_t exl3_adapter_add_workspace_size(int T, int max_rank) {
  if (T < 0 || T > (1 << 22) || !rank_ok(max_rank)) return 0;
  return add_ws(T, max_rank).total;
}

size_t exl3_adapter_scratch_size(int T, int max_rank, int n) {
  if (T < 0 || T > (1 << 22) || !rank_ok(max_rank) || n < 128 || n > (1 << 20)) return 0;
  return large_tiles(T, max_rank, n) ? add_ws(T, max_rank).total - kDataOff : 0;
}

int exl3_adapter_add(const uint16_t *x, int64_t x_stride, const void *y, int64_t y_stride, void *out,
                     int64_t out_stride, int dtype, const exl3_adapters *ad, const void *plan, int T, int batch,
                     void *workspace, size_t ws_bytes, exl3_stream_t stream) {
  exl3_clear_error();
  EXL3_TRY(check_call(x, x_stride, y, y_stride, out, out_stride, dtype, ad, plan, T, batch));
  EXL3_TRY(check_workspace(workspace, ws_bytes, add_ws(T, ad->max_rank).total));
  return launch(x, x_stride, y, y_stride, out, out_stride, dtype, ad, plan, T, batch, workspace,
                at<char>(workspace, kDataOff), stream);
}

int exl3_adapter_add_scratch(const uint16_t *x, int64_t x_stride, const void *y, int64_t y_stride, void *out,
                             int64_t out_stride, int dtype, const exl3_adapters *ad, const void *plan, int T,
                             int batch, void *workspace, size_t ws_bytes, void *scratch, size_t scratch_bytes,
                             exl3_stream_t stream) {
  exl3_clear_error();
  EXL3_TRY(check_call(x, x_stride, y, y_stride, out, out_stride, dtype, ad, plan, T, batch));
  EXL3_TRY(check_workspace(workspace, ws_bytes, kCtrlBytes));
  const size_t need = exl3_adapter_scratch_size(T, ad->max_rank, ad->n);
  if (need && !scratch) return exl3_fail(EXL3_ERR_WORKSPACE, "scratch is NULL (%zu bytes needed)", need);
  if (need && reinterpret_cast<uintptr_t>(scratch) & (kAlign - 1))
    return exl3_fail(EXL3_ERR_WORKSPACE, "scratch must be %zu-byte aligned", kAlign);
  if (scratch_bytes < need)
    return exl3_fail(EXL3_ERR_WORKSPACE, "scratch has %zu bytes, %zu needed", scratch_bytes, need);
  return launch(x, x_stride, y, y_stride, out, out_stride, dtype, ad, plan, T, batch, workspace, scratch, stream);
}

}  // extern "C"
