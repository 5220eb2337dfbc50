// abi_w4.hip -- host side of the C ABI's products with 4-bit weights
// (moe_w4_matvec, fused_moe_w4): argument checks before anything is enqueued,
// workspace layout, launches.
#include "abi_checks.h"

namespace {

int check_sizes(int32_t format, int32_t elem, int64_t T, int64_t K, int64_t N, int32_t E,
                int32_t top_k, int64_t group) {
  if (format != MOE_W4_INT && format != MOE_W4_MX)
    return abi_fail(MOE_ERR_UNSUPPORTED, "unknown 4-bit format %d", format);
  if (elem != MOE_ELEM_BF16 && elem != MOE_ELEM_F16)
    return abi_fail(MOE_ERR_UNSUPPORTED, "4-bit products take bf16 or fp16 activations");
  if (T < 0) return abi_fail(MOE_ERR_SHAPE, "T must be >= 0 (got %lld)", (long long)T);
  if (K < 1 || N < 1) return abi_fail(MOE_ERR_SHAPE, "K and N must be >= 1");
  if (E < 1) return abi_fail(MOE_ERR_SHAPE, "E must be >= 1 (got %d)", E);
  if (top_k < 1) return abi_fail(MOE_ERR_SHAPE, "top_k must be >= 1 (got %d)", top_k);
  if (group < 0) return abi_fail(MOE_ERR_SHAPE, "group must be >= 0 (got %lld)", (long long)group);
  if (K >= (int64_t(1) << 31) || N >= (int64_t(1) << 31) || N * K >= (int64_t(1) << 32))
    return abi_fail(MOE_ERR_UNSUPPORTED, "an expert's 4-bit weights must stay below 2 GiB");
  if (T > kW4MaxRoutes || T * top_k > kW4MaxRoutes)
    return abi_fail(MOE_ERR_UNSUPPORTED, "4-bit products take T * top_k <= %d routes", kW4MaxRoutes);
  return MOE_OK;
}

// Scale groups along a contraction of length L.
int check_group(int32_t format, int64_t L, int64_t group) {
  if (format == MOE_W4_MX && group != 32)
    return abi_fail(MOE_ERR_UNSUPPORTED, "the microscaling format has groups of 32");
  if (group != 0 && group != 32 && group != 64 && group != 128)
    return abi_fail(MOE_ERR_UNSUPPORTED, "group must be 32, 64, 128 or 0 (got %lld)", (long long)group);
  const int64_t unit = group ? group : 128;
  if (L % unit)
    return abi_fail(MOE_ERR_UNSUPPORTED, "the contraction (%lld) must be a multiple of %lld",
                    (long long)L, (long long)unit);
  return MOE_OK;
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// The intermediate: three bf16 parts of R rows.
size_t parts_bytes(size_t R, size_t I) { return R * I * 6; }

}  // namespace

extern "C" {

int moe_w4_matvec(int32_t format, int32_t elem, const void* x, int32_t x_per_route, const void* w,
                  const void* w_scale, const uint8_t* w_zero, const int32_t* topk_ids, void* out,
                  int64_t T, int64_t K, int64_t N, int32_t E, int32_t top_k, int32_t group,
                  int32_t swiglu, void* stream) {
  int rc = check_sizes(format, elem, T, K, N, E, top_k, group);
  if (rc) return rc;
  if ((rc = check_group(format, K, group))) return rc;
  if (swiglu && N % 2) return abi_fail(MOE_ERR_SHAPE, "N (gate and up rows) must be even");
  if (T > 0 && !topk_ids && (E != 1 || top_k != 1))
    return abi_fail(MOE_ERR_NULL, "without topk_ids there must be one expert and one route");
  if (format == MOE_W4_MX && w_zero)
    return abi_fail(MOE_ERR_UNSUPPORTED, "the microscaling format has no zero points");
  if ((rc = check_ptrs({{x, T > 0}, {w, true}, {w_scale, true}, {w_zero, false}, {topk_ids, false},
                        {out, T > 0}})))
    return rc;
  W4Args a{x, static_cast<const uint8_t*>(w), w_scale, w_zero, topk_ids, out,
           (int)K, (int)N, E, (int)(T * top_k), top_k, group ? group : (int)K,
           elem, elem, elem, x_per_route != 0, swiglu != 0, 0};
  return launched(launch_w4(format, a, static_cast<hipStream_t>(stream)));
}

int moe_w4_workspace_size(int64_t T, int64_t K, int64_t N, int32_t top_k, size_t* bytes) {
  if (!bytes) return abi_fail(MOE_ERR_NULL, "bytes is NULL");
  int rc = check_sizes(MOE_W4_INT, MOE_ELEM_BF16, T, K, N, 1, top_k, 0);
  if (rc) return rc;
  if (N % 2) return abi_fail(MOE_ERR_SHAPE, "N (gate and up rows) must be even");
  const size_t R = (size_t)T * top_k;
  *bytes = up256(parts_bytes(R, N / 2)) + up256(R * K * 4);
  return abi_ok();
}

int fused_moe_w4(int32_t format, int32_t elem, const void* x, const void* w1, const void* w1_scale,
                 const uint8_t* w1_zero, const void* w2, const void* w2_scale,
                 const uint8_t* w2_zero, const int32_t* topk_ids, const float* topk_weights,
                 void* out, int64_t T, int64_t K, int64_t N, int32_t E, int32_t top_k,
                 int32_t group, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_sizes(format, elem, T, K, N, E, top_k, group);
  if (rc) return rc;
  if (N % 2) return abi_fail(MOE_ERR_SHAPE, "N (gate and up rows) must be even");
  if ((rc = check_group(format, K, group)) || (rc = check_group(format, N / 2, group))) return rc;
  if (format == MOE_W4_MX && (w1_zero || w2_zero))
    return abi_fail(MOE_ERR_UNSUPPORTED, "the microscaling format has no zero points");
  if ((rc = check_ptrs({{x, T > 0}, {w1, true}, {w1_scale, true}, {w1_zero, false}, {w2, true},
                        {w2_scale, true}, {w2_zero, false}, {topk_ids, T > 0},
                        {topk_weights, T > 0}, {out, T > 0}})))
    return rc;
  size_t need = 0;
  if ((rc = moe_w4_workspace_size(T, K, N, top_k, &need))) return rc;
  if (T == 0) return abi_ok();
  if (!workspace || workspace_bytes < need)
    return abi_fail(MOE_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes",
                    workspace ? workspace_bytes : (size_t)0, need);
  if (!aligned(workspace)) return abi_fail(MOE_ERR_ALIGN, "the workspace must be 16-byte aligned");
  const int R = (int)(T * top_k), I = (int)(N / 2);
  void* h = workspace;  // (R, 3, I) bf16 parts
  float* y = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + up256(parts_bytes(R, I)));
  hipStream_t s = static_cast<hipStream_t>(stream);
  W4Args up{x, static_cast<const uint8_t*>(w1), w1_scale, w1_zero, topk_ids, h,
            (int)K, (int)N, E, R, top_k, group ? group : (int)K,
            elem, ELEM_PARTS, elem, 0, 1, 0};
  W4Args down{h, static_cast<const uint8_t*>(w2), w2_scale, w2_zero, topk_ids, out,
              I, (int)K, E, R, top_k, group ? group : I,
              ELEM_PARTS, elem, elem, 1, 0, 0};
  hipError_t e = launch_w4(format, up, s);
  if (e == hipSuccess) e = launch_w4_down(format, down, topk_weights, y, (int)T, s);
  return launched(e);
}

}  // extern "C"
