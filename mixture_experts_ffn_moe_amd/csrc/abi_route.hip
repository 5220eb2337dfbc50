// abi_route.hip -- host side of the C ABI's general router (moe_route_topk) and
// of its gradient: argument checks before anything is enqueued, then the launch.
#include <cmath>

#include "abi_checks.h"

namespace {

int check_route(int32_t elem, int64_t T, int32_t E, int32_t top_k, int32_t scoring, float scale) {
  if (elem < MOE_ELEM_BF16 || elem > MOE_ELEM_F32)
    return abi_fail(MOE_ERR_UNSUPPORTED, "logits must be bf16, fp16 or fp32 (element type %d)", elem);
  if (scoring != MOE_SCORE_SOFTMAX && scoring != MOE_SCORE_SIGMOID)
    return abi_fail(MOE_ERR_UNSUPPORTED, "unknown scoring %d", scoring);
  if (T < 0) return abi_fail(MOE_ERR_SHAPE, "T must be >= 0 (got %lld)", (long long)T);
  if (E < 1) return abi_fail(MOE_ERR_SHAPE, "E must be >= 1 (got %d)", E);
  if (top_k < 1) return abi_fail(MOE_ERR_SHAPE, "top_k must be >= 1 (got %d)", top_k);
  if (T > (int64_t(1) << 26) - 4)  // a workgroup of 256 threads has four tokens
    return abi_fail(MOE_ERR_UNSUPPORTED, "T must be at most 2^26 - 4");
  if (E > kRouteMaxExperts)
    return abi_fail(MOE_ERR_UNSUPPORTED, "E must be at most %d (got %d)", kRouteMaxExperts, E);
  if (top_k > kRouteMaxTopK || top_k > E)
    return abi_fail(MOE_ERR_UNSUPPORTED, "top_k must be at most %d and at most E (got %d)", kRouteMaxTopK, top_k);
  if (!std::isfinite(scale)) return abi_fail(MOE_ERR_SHAPE, "scale must be finite");
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_route_topk(int32_t elem, const void* logits, const float* bias, int64_t T, int32_t E,
                   int32_t top_k, int32_t scoring, int32_t n_group, int32_t topk_group,
                   int32_t group_top, int32_t renormalize, float scale, int32_t* topk_ids,
                   float* topk_weights, void* stream) {
  int rc = check_route(elem, T, E, top_k, scoring, scale);
  if (rc) return rc;
  if (n_group < 1 || E % n_group)
    return abi_fail(MOE_ERR_SHAPE, "n_group must divide E (got %d of %d)", n_group, E);
  if (n_group > kRouteMaxGroups)
    return abi_fail(MOE_ERR_UNSUPPORTED, "n_group must be at most %d (got %d)", kRouteMaxGroups, n_group);
  if (topk_group < 1 || topk_group > n_group)
    return abi_fail(MOE_ERR_SHAPE, "topk_group must be in [1, n_group] (got %d)", topk_group);
  if (group_top != 1 && group_top != 2)
    return abi_fail(MOE_ERR_UNSUPPORTED, "group_top must be 1 or 2 (got %d)", group_top);
  if (top_k > topk_group * (E / n_group))
    return abi_fail(MOE_ERR_SHAPE, "top_k is more than the experts of topk_group groups");
  if ((rc = check_ptrs({{logits, T > 0}, {bias, false}, {topk_ids, T > 0}, {topk_weights, T > 0}})))
    return rc;
  RouteArgs a{logits, bias, T, E, top_k, elem, scoring, n_group, topk_group, group_top, renormalize != 0,
              scale};
  return launched(launch_route_topk(a, topk_ids, topk_weights, static_cast<hipStream_t>(stream)));
}

int moe_route_topk_backward(int32_t elem, const void* logits, const int32_t* topk_ids,
                            const float* d_weights, int64_t T, int32_t E, int32_t top_k,
                            int32_t scoring, int32_t renormalize, float scale, void* d_logits,
                            void* stream) {
  int rc = check_route(elem, T, E, top_k, scoring, scale);
  if (rc) return rc;
  if ((rc = check_ptrs({{logits, T > 0}, {topk_ids, T > 0}, {d_weights, T > 0}, {d_logits, T > 0}})))
    return rc;
  RouteArgs a{logits, nullptr, T, E, top_k, elem, scoring, 1, 1, 1, renormalize != 0, scale};
  return launched(launch_route_topk_backward(a, topk_ids, d_weights, d_logits,
                                             static_cast<hipStream_t>(stream)));
}

}  // extern "C"
