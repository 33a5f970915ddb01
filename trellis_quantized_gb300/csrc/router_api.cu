// router_api.cu -- the C entry points of the router's product and of routing:
// argument checks.
#include <cmath>

#include "api_util.cuh"
#include "router.cuh"

// ---- kernels (other translation units)
int exl3_launch_router_logits(const exl3::rt::LogitArgs &a, bool packed, cudaStream_t s);
cudaError_t exl3_launch_router_pack(const float *w, int E, int k, __half *out, float *scale, cudaStream_t s);
cudaError_t exl3_launch_route(const exl3::rt::Args &a, bool f16, cudaStream_t s);

namespace {

constexpr int kMaxExperts = 1024, kMaxRows = 1 << 22;

int check_natural(const void *p, const char *name, size_t align, bool required = true) {
  if (!p) return required ? exl3_fail(EXL3_ERR_ARG, "%s is NULL", name) : EXL3_OK;
  if (reinterpret_cast<uintptr_t>(p) & (align - 1))
    return exl3_fail(EXL3_ERR_ARG, "%s is not %zu-byte aligned", name, align);
  return EXL3_OK;
}

int check_router_shape(int E, int k) {
  if (E < 1 || E > kMaxExperts || k < 8 || k % 8 || k > (1 << 20))
    return exl3_fail(EXL3_ERR_SHAPE, "E = %d must be 1..%d and k = %d a multiple of 8 up to 2^20", E, kMaxExperts, k);
  return EXL3_OK;
}

}  // namespace

extern "C" {

int exl3_router_pack(const float *w, int E, int k, uint16_t *packed, float *scale, exl3_stream_t stream) {
  exl3_clear_error();
  EXL3_TRY(check_ptr(w, "w"));
  EXL3_TRY(check_ptr(packed, "packed"));
  EXL3_TRY(check_natural(scale, "scale", 4));
  EXL3_TRY(check_router_shape(E, k));
  return exl3_cuda_check(exl3_launch_router_pack(w, E, k, reinterpret_cast<__half *>(packed), scale, stream),
                         "router pack launch");
}

size_t exl3_router_logits_workspace_size(void) { return kCtrlBytes; }

int exl3_router_logits(const uint16_t *x, int64_t x_stride, int T, const exl3_router *router, float *logits,
                       void *workspace, size_t ws_bytes, exl3_stream_t stream) {
  exl3_clear_error();
  if (!router) return exl3_fail(EXL3_ERR_ARG, "router is NULL");
  EXL3_TRY(check_router_shape(router->E, router->k));
  EXL3_TRY(check_ptr(router->w, "router.w"));
  EXL3_TRY(check_natural(router->w_scale, "router.w_scale", 4, false));
  EXL3_TRY(check_natural(router->bias, "router.bias", 4, false));
  EXL3_TRY(check_ptr(x, "x"));
  EXL3_TRY(check_ptr(logits, "logits"));
  if (T < 0 || T > kMaxRows) return exl3_fail(EXL3_ERR_SHAPE, "T = %d out of range (0..2^22)", T);
  if (x_stride < router->k || x_stride % 8 || x_stride >= ((int64_t)1 << 39))
    return exl3_fail(EXL3_ERR_SHAPE, "x: stride %lld must be a multiple of 8 elements, at least k = %d and below 2^39",
                     (long long)x_stride, router->k);
  EXL3_TRY(check_workspace(workspace, ws_bytes, kCtrlBytes));
  if (T == 0) return EXL3_OK;
  exl3::rt::LogitArgs a = {};
  a.x = reinterpret_cast<const __half *>(x);
  a.x_stride = x_stride;
  a.w = reinterpret_cast<const __half *>(router->w);
  a.w_scale = router->w_scale;
  a.bias = router->bias;
  a.logits = logits;
  a.T = T;
  a.E = router->E;
  a.k = router->k;
  a.err = at<int>(workspace, 0);
  return exl3_launch_router_logits(a, router->w_scale != nullptr, stream);
}

int exl3_route(const void *logits, int64_t stride, int in_dtype, int T, int E, const exl3_route_rule *rule,
               int32_t *ids, float *weights, exl3_stream_t stream) {
  exl3_clear_error();
  if (!rule) return exl3_fail(EXL3_ERR_ARG, "rule is NULL");
  if (in_dtype != EXL3_OUT_F16 && in_dtype != EXL3_OUT_F32)
    return exl3_fail(EXL3_ERR_ARG, "in_dtype %d invalid", in_dtype);
  if (rule->score != EXL3_SCORE_SOFTMAX && rule->score != EXL3_SCORE_SIGMOID)
    return exl3_fail(EXL3_ERR_ARG, "score %d invalid", rule->score);
  if (rule->group_score != EXL3_GROUP_MAX && rule->group_score != EXL3_GROUP_TOP2)
    return exl3_fail(EXL3_ERR_ARG, "group_score %d invalid", rule->group_score);
  if (rule->renormalise != 0 && rule->renormalise != 1)
    return exl3_fail(EXL3_ERR_ARG, "renormalise %d invalid", rule->renormalise);
  if (!std::isfinite(rule->scale)) return exl3_fail(EXL3_ERR_ARG, "scale must be finite");
  if (T < 0 || T > kMaxRows || E < 1 || E > kMaxExperts)
    return exl3_fail(EXL3_ERR_SHAPE, "T = %d (0..2^22) or E = %d (1..%d) out of range", T, E, kMaxExperts);
  if (rule->groups < 1 || rule->groups > 32 || E % rule->groups || rule->groups_kept < 1 ||
      rule->groups_kept > rule->groups)
    return exl3_fail(EXL3_ERR_SHAPE, "groups = %d must be 1..32 and divide E = %d, groups_kept = %d be 1..groups",
                     rule->groups, E, rule->groups_kept);
  if (rule->topk < 1 || rule->topk > 32 || rule->topk > rule->groups_kept * (E / rule->groups))
    return exl3_fail(EXL3_ERR_SHAPE, "topk = %d must be 1..32 and at most the %d experts of the groups kept",
                     rule->topk, rule->groups_kept * (E / rule->groups));
  if (stride < E || stride >= ((int64_t)1 << 39))
    return exl3_fail(EXL3_ERR_SHAPE, "logits: stride %lld must be at least E = %d and below 2^39", (long long)stride, E);
  EXL3_TRY(check_natural(logits, "logits", in_dtype == EXL3_OUT_F32 ? 4 : 2));
  EXL3_TRY(check_natural(rule->bias, "rule.bias", 4, false));
  EXL3_TRY(check_natural(ids, "ids", 4));
  EXL3_TRY(check_natural(weights, "weights", 4));
  if (T == 0) return EXL3_OK;
  exl3::rt::Args a = {};
  a.logits = logits;
  a.stride = stride;
  a.T = T;
  a.E = E;
  a.topk = rule->topk;
  a.bias = rule->bias;
  a.score = rule->score;
  a.groups = rule->groups;
  a.kept = rule->groups_kept;
  a.group_score = rule->group_score;
  a.renormalise = rule->renormalise;
  a.scale = rule->scale;
  a.ids = ids;
  a.weights = weights;
  return exl3_cuda_check(exl3_launch_route(a, in_dtype == EXL3_OUT_F16, stream), "route launch");
}

}  // extern "C"
