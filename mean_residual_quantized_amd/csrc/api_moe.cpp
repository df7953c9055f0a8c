// C ABI of the routing, token exchange and gradient clipping calls: argument
// validation and launches.  Every check runs before the first HIP call.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <new>

#include "api_common.hpp"
#include "launch.hpp"

using namespace averis;

static_assert(AVERIS_MAX_EXPERTS == kMaxExperts && AVERIS_MAX_TOPK == kMaxTopk &&
                  AVERIS_MAX_GRADS == kMaxGrads && AVERIS_MAX_GROUPS == kMaxGroups &&
                  AVERIS_SCORE_SOFTMAX == kScoreSoftmax && AVERIS_SCORE_SIGMOID == kScoreSigmoid,
              "limits and names");

namespace {

// tokens x topk slots, numbered in 32 bits
averis_status_t check_slots(int64_t tokens, int topk) {
  if (tokens < 0 || tokens > INT32_MAX) return AVERIS_E_SHAPE;
  if (topk < 1 || topk > kMaxTopk) return AVERIS_E_ARG;
  if (tokens * topk > INT32_MAX) return AVERIS_E_SHAPE;
  return AVERIS_OK;
}

averis_status_t check_router(int64_t tokens, int experts, int64_t ld, int topk) {
  if (experts < 1 || experts > kMaxExperts) return AVERIS_E_ARG;
  const averis_status_t s = check_slots(tokens, topk);
  if (s != AVERIS_OK) return s;
  if (topk > experts) return AVERIS_E_ARG;
  return ld < experts ? AVERIS_E_SHAPE : AVERIS_OK;
}

// a rows x cols matrix of the exchange
averis_status_t check_matrix(const void* p, averis_dtype_t dtype, int64_t rows, int64_t cols,
                             int64_t ld) {
  if (ld < cols) return AVERIS_E_SHAPE;
  if (rows > 0 && !p) return AVERIS_E_NULL;
  return aligned(p, elem_size(dtype)) ? AVERIS_OK : AVERIS_E_ALIGN;
}

}  // namespace

extern "C" {

averis_status_t averis_moe_route(const void* logits, averis_dtype_t dtype, int64_t tokens,
                                 int experts, int64_t ld, int topk, int renorm,
                                 int32_t* expert_ids, float* weights, hipStream_t stream) {
  if (!dtype_ok(dtype)) return AVERIS_E_DTYPE;
  averis_status_t s = check_router(tokens, experts, ld, topk);
  if (s != AVERIS_OK) return s;
  if (renorm != 0 && renorm != 1) return AVERIS_E_ARG;
  if (tokens > 0 && (!logits || !expert_ids || !weights)) return AVERIS_E_NULL;
  if (!aligned(logits, elem_size(dtype)) || !aligned(expert_ids, 4) || !aligned(weights, 4))
    return AVERIS_E_ALIGN;
  return hip_status(launch_moe_route(logits, dtype == AVERIS_BF16, tokens, experts, ld, topk,
                                     renorm != 0, expert_ids, weights, stream));
}

averis_status_t averis_moe_route_grad(const void* logits, averis_dtype_t dtype, int64_t tokens,
                                      int experts, int64_t ld, int topk, int renorm,
                                      const int32_t* expert_ids, const float* dweights,
                                      void* dlogits, int64_t ldd, hipStream_t stream) {
  if (!dtype_ok(dtype)) return AVERIS_E_DTYPE;
  averis_status_t s = check_router(tokens, experts, ld, topk);
  if (s != AVERIS_OK) return s;
  if (renorm != 0 && renorm != 1) return AVERIS_E_ARG;
  if (ldd < experts) return AVERIS_E_SHAPE;
  if (tokens > 0 && (!logits || !expert_ids || !dweights || !dlogits)) return AVERIS_E_NULL;
  const size_t es = elem_size(dtype);
  if (!aligned(logits, es) || !aligned(dlogits, es) || !aligned(expert_ids, 4) ||
      !aligned(dweights, 4))
    return AVERIS_E_ALIGN;
  return hip_status(launch_moe_route_grad(logits, dtype == AVERIS_BF16, tokens, experts, ld, topk,
                                          renorm != 0, expert_ids, dweights, dlogits, ldd,
                                          stream));
}

averis_status_t averis_moe_route_groups(const void* logits, averis_dtype_t dtype, int64_t tokens,
                                        int experts, int64_t ld, int topk, const float* bias,
                                        averis_score_t score, int groups, int topk_groups,
                                        int group_top, int renorm, float scale,
                                        int32_t* expert_ids, float* weights, hipStream_t stream) {
  if (!dtype_ok(dtype)) return AVERIS_E_DTYPE;
  const averis_status_t s = check_router(tokens, experts, ld, topk);
  if (s != AVERIS_OK) return s;
  if (score != AVERIS_SCORE_SOFTMAX && score != AVERIS_SCORE_SIGMOID) return AVERIS_E_ARG;
  if (groups < 1 || groups > kMaxGroups || experts % groups != 0) return AVERIS_E_ARG;
  if (topk_groups < 1 || topk_groups > groups) return AVERIS_E_ARG;
  const int size = experts / groups;
  if (topk > topk_groups * size || group_top < 1 || group_top > 2) return AVERIS_E_ARG;
  if (renorm != 0 && renorm != 1) return AVERIS_E_ARG;
  if (tokens > 0 && (!logits || !expert_ids || !weights)) return AVERIS_E_NULL;
  if (!aligned(logits, elem_size(dtype)) || !aligned(bias, 4) || !aligned(expert_ids, 4) ||
      !aligned(weights, 4))
    return AVERIS_E_ALIGN;
  const RouteGroups a{tokens, ld, experts, topk, bias, score, groups, topk_groups, group_top,
                      renorm != 0, scale, expert_ids, weights, size, 0, 0};
  return hip_status(launch_route_groups(logits, dtype == AVERIS_BF16, a, stream));
}

averis_status_t averis_moe_route_groups_grad(const void* logits, averis_dtype_t dtype,
                                             int64_t tokens, int experts, int64_t ld, int topk,
                                             averis_score_t score, int renorm, float scale,
                                             const int32_t* expert_ids, const float* dweights,
                                             void* dlogits, int64_t ldd, hipStream_t stream) {
  if (!dtype_ok(dtype)) return AVERIS_E_DTYPE;
  const averis_status_t s = check_router(tokens, experts, ld, topk);
  if (s != AVERIS_OK) return s;
  if (score != AVERIS_SCORE_SOFTMAX && score != AVERIS_SCORE_SIGMOID) return AVERIS_E_ARG;
  if (renorm != 0 && renorm != 1) return AVERIS_E_ARG;
  if (ldd < experts) return AVERIS_E_SHAPE;
  if (tokens > 0 && (!logits || !expert_ids || !dweights || !dlogits)) return AVERIS_E_NULL;
  const size_t es = elem_size(dtype);
  if (!aligned(logits, es) || !aligned(dlogits, es) || !aligned(expert_ids, 4) ||
      !aligned(dweights, 4))
    return AVERIS_E_ALIGN;
  const RouteGroupsGrad a{tokens, ld, ldd, experts, topk, score, renorm != 0, scale, expert_ids,
                          dweights};
  return hip_status(launch_route_groups_grad(logits, dtype == AVERIS_BF16, a, dlogits, stream));
}

averis_status_t averis_moe_sort(const int32_t* expert_ids, int64_t tokens, int topk, int experts,
                                int64_t* seg_offsets, int32_t* pos, int32_t* src, void* ws,
                                size_t ws_bytes, hipStream_t stream) {
  if (experts < 1 || experts > kMaxExperts) return AVERIS_E_ARG;
  const averis_status_t s = check_slots(tokens, topk);
  if (s != AVERIS_OK) return s;
  if (!seg_offsets || (tokens > 0 && (!expert_ids || !pos))) return AVERIS_E_NULL;
  if (!aligned(seg_offsets, 8) || !aligned(expert_ids, 4) || !aligned(pos, 4) || !aligned(src, 4))
    return AVERIS_E_ALIGN;
  const size_t need = moe_sort_ws_bytes(tokens * topk, experts);
  if (need && (!ws || ws_bytes < need)) return AVERIS_E_WORKSPACE;
  if (ws && !aligned(ws, 256)) return AVERIS_E_ALIGN;
  return hip_status(launch_moe_sort(expert_ids, tokens * topk, experts, seg_offsets, pos, src, ws,
                                    stream));
}

averis_status_t averis_moe_dispatch(const void* x, averis_dtype_t dtype, int64_t tokens,
                                    int64_t cols, int64_t ldx, const int32_t* pos, int topk,
                                    void* rows, int64_t ldr, hipStream_t stream) {
  if (!dtype_ok(dtype)) return AVERIS_E_DTYPE;
  averis_status_t s = check_slots(tokens, topk);
  if (s != AVERIS_OK) return s;
  if (cols <= 0) return AVERIS_E_SHAPE;
  if ((s = check_matrix(x, dtype, tokens, cols, ldx)) != AVERIS_OK) return s;
  if ((s = check_matrix(rows, dtype, tokens, cols, ldr)) != AVERIS_OK) return s;
  if (tokens > 0 && !pos) return AVERIS_E_NULL;
  if (!aligned(pos, 4)) return AVERIS_E_ALIGN;
  return hip_status(launch_moe_dispatch(x, dtype == AVERIS_BF16, tokens, cols, ldx, pos, topk,
                                        rows, ldr, stream));
}

averis_status_t averis_moe_combine(const void* rows, averis_dtype_t dtype, int64_t tokens,
                                   int64_t cols, int64_t ldr, const int32_t* pos,
                                   const float* weights, int topk, void* y, int64_t ldy,
                                   hipStream_t stream) {
  if (!dtype_ok(dtype)) return AVERIS_E_DTYPE;
  averis_status_t s = check_slots(tokens, topk);
  if (s != AVERIS_OK) return s;
  if (cols <= 0) return AVERIS_E_SHAPE;
  if ((s = check_matrix(rows, dtype, tokens, cols, ldr)) != AVERIS_OK) return s;
  if ((s = check_matrix(y, dtype, tokens, cols, ldy)) != AVERIS_OK) return s;
  if (tokens > 0 && !pos) return AVERIS_E_NULL;
  if (!aligned(pos, 4) || !aligned(weights, 4)) return AVERIS_E_ALIGN;
  return hip_status(launch_moe_combine(rows, dtype == AVERIS_BF16, tokens, cols, ldr, pos, weights,
                                       topk, y, ldy, stream));
}

averis_status_t averis_moe_combine_grad(const void* dy, averis_dtype_t dtype, int64_t tokens,
                                        int64_t cols, int64_t ldy, const void* rows, int64_t ldr,
                                        const int32_t* pos, const float* weights, int topk,
                                        void* drows, int64_t lddr, float* dweights,
                                        hipStream_t stream) {
  if (!dtype_ok(dtype)) return AVERIS_E_DTYPE;
  averis_status_t s = check_slots(tokens, topk);
  if (s != AVERIS_OK) return s;
  if (cols <= 0) return AVERIS_E_SHAPE;
  if ((s = check_matrix(dy, dtype, tokens, cols, ldy)) != AVERIS_OK) return s;
  if ((s = check_matrix(rows, dtype, tokens, cols, ldr)) != AVERIS_OK) return s;
  if ((s = check_matrix(drows, dtype, tokens, cols, lddr)) != AVERIS_OK) return s;
  if (tokens > 0 && (!pos || !weights || !dweights)) return AVERIS_E_NULL;
  if (!aligned(pos, 4) || !aligned(weights, 4) || !aligned(dweights, 4)) return AVERIS_E_ALIGN;
  return hip_status(launch_moe_combine_grad(dy, dtype == AVERIS_BF16, tokens, cols, ldy, rows, ldr,
                                            pos, weights, topk, drows, lddr, dweights, stream));
}

static averis_status_t clip_common(int n, const averis_grad_t* g, bool scale, double max_norm,
                                   double eps, float* norm, void* ws, size_t ws_bytes,
                                   hipStream_t stream) {
  if (n < 0 || n > kMaxGrads) return AVERIS_E_ARG;
  if (!norm || (n > 0 && !g)) return AVERIS_E_NULL;
  if (!aligned(norm, 4)) return AVERIS_E_ALIGN;
  if (scale && !(max_norm >= 0.0 && eps >= 0.0)) return AVERIS_E_ARG;
  for (int i = 0; i < n; ++i) {
    if (!dtype_ok(g[i].dtype)) return AVERIS_E_DTYPE;
    if (g[i].numel < 0 || g[i].numel > ((int64_t)1 << 40)) return AVERIS_E_SHAPE;
    if (g[i].numel > 0 && (!g[i].grad || (scale && !g[i].out))) return AVERIS_E_NULL;
    const size_t es = elem_size(g[i].dtype);
    if (!aligned(g[i].grad, es) || (scale && !aligned(g[i].out, es))) return AVERIS_E_ALIGN;
  }
  if (!ws || ws_bytes < grad_norm_ws_bytes(n)) return AVERIS_E_WORKSPACE;
  if (!aligned(ws, 256)) return AVERIS_E_ALIGN;
  // the checked list in the launches' own form: short ones on the stack
  constexpr int kShort = 512;
  GradTensor few[kShort];
  GradTensor* w = n <= kShort ? few : new (std::nothrow) GradTensor[n];
  if (!w) return hip_status(hipErrorOutOfMemory);
  for (int i = 0; i < n; ++i)
    w[i] = GradTensor{g[i].grad, g[i].out, g[i].numel, g[i].dtype == AVERIS_BF16};
  const averis_status_t s =
      hip_status(launch_grad_clip(n, w, scale, max_norm, eps, norm, ws, stream));
  if (w != few) delete[] w;
  return s;
}

averis_status_t averis_grad_norm(int n, const averis_grad_t* grads, float* norm, void* ws,
                                 size_t ws_bytes, hipStream_t stream) {
  return clip_common(n, grads, false, 0.0, 0.0, norm, ws, ws_bytes, stream);
}

averis_status_t averis_grad_clip(int n, const averis_grad_t* grads, double max_norm, double eps,
                                 float* norm, void* ws, size_t ws_bytes, hipStream_t stream) {
  return clip_common(n, grads, true, max_norm, eps, norm, ws, ws_bytes, stream);
}

}  // extern "C"
