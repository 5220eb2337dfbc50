// abi_rows.hip -- host side of the C ABI's operators on the rows of a plan
// (moe_route_rows, moe_permute, moe_unpermute and their gradients) and of the
// router's gradient: argument checks before anything is enqueued, then the
// launch.
#include "abi_checks.h"

namespace {

// workgroups of 256 threads in one launch: the grid's thread count is 32-bit
constexpr int64_t kMaxGroups = (int64_t(1) << 24) - 1;

int check_rows(int32_t elem, int64_t T, int64_t K, int32_t top_k, int32_t n_shared,
               int64_t rows_cap, bool sums) {
  if (elem < MOE_ELEM_BF16 || elem > MOE_ELEM_U8)
    return abi_fail(MOE_ERR_UNSUPPORTED, "unknown element type %d", elem);
  if (sums && elem == MOE_ELEM_U8)
    return abi_fail(MOE_ERR_UNSUPPORTED, "rows of bytes can be moved, not summed");
  if (T < 0) return abi_fail(MOE_ERR_SHAPE, "T must be >= 0 (got %lld)", (long long)T);
  if (K < 1) return abi_fail(MOE_ERR_SHAPE, "K must be >= 1 (got %lld)", (long long)K);
  if (top_k < 1) return abi_fail(MOE_ERR_SHAPE, "top_k must be >= 1 (got %d)", top_k);
  if (n_shared < 0) return abi_fail(MOE_ERR_SHAPE, "n_shared must be >= 0 (got %d)", n_shared);
  const int64_t per = (int64_t)top_k + n_shared;
  if (T >= (int64_t(1) << 31) || T * per >= (int64_t(1) << 31))
    return abi_fail(MOE_ERR_SHAPE, "T*(top_k + n_shared) must be < 2^31");
  if (rows_cap < 0 || rows_cap >= (int64_t(1) << 31))
    return abi_fail(MOE_ERR_SHAPE, "rows_cap must be in [0, 2^31) (got %lld)", (long long)rows_cap);
  if (K >= (int64_t(1) << 31)) return abi_fail(MOE_ERR_UNSUPPORTED, "K must be < 2^31");
  // the launch's workgroups: about one per 4,096 bytes of a token (or per
  // route), and one per four plan rows
  const int64_t cols = K / 1024 + 2;
  if (T * (cols > per ? cols : per) + rows_cap / 4 + 1 > kMaxGroups)
    return abi_fail(MOE_ERR_UNSUPPORTED, "T * K is too large for one launch");
  return MOE_OK;
}

int check_ntp(const int32_t* ntp) {
  if (!ntp) return abi_fail(MOE_ERR_NULL, "num_tokens_post_padded is NULL");
  if (!aligned(ntp, 4))
    return abi_fail(MOE_ERR_ALIGN, "num_tokens_post_padded must be 4-byte aligned");
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_route_rows(const int32_t* topk_ids, int64_t T, int32_t top_k, int32_t E, int32_t n_shared,
                   const int32_t* sorted_token_ids, const int32_t* num_tokens_post_padded,
                   int64_t rows_cap, int32_t* row_of_route, void* stream) {
  int rc = check_rows(MOE_ELEM_F32, T, 1, top_k, n_shared, rows_cap, false);
  if (rc) return rc;
  if (E < 1) return abi_fail(MOE_ERR_SHAPE, "E must be >= 1 (got %d)", E);
  if ((rc = check_ntp(num_tokens_post_padded))) return rc;
  if ((rc = check_ptrs({{topk_ids, T > 0}, {sorted_token_ids, rows_cap > 0}, {row_of_route, T > 0}})))
    return rc;
  if (T == 0) return abi_ok();
  RowsArgs a{sorted_token_ids, num_tokens_post_padded, nullptr, nullptr, T, 1, rows_cap, top_k,
             n_shared};
  return launched(launch_route_rows(topk_ids, a, E, row_of_route, static_cast<hipStream_t>(stream)));
}

int moe_permute(int32_t elem, const void* x, const int32_t* row_of_route,
                const int32_t* sorted_token_ids, const int32_t* num_tokens_post_padded, void* rows,
                int64_t T, int64_t K, int32_t top_k, int32_t n_shared, int64_t rows_cap,
                void* stream) {
  int rc = check_rows(elem, T, K, top_k, n_shared, rows_cap, false);
  if (rc) return rc;
  if ((rc = check_ntp(num_tokens_post_padded))) return rc;
  if ((rc = check_ptrs({{x, T > 0}, {row_of_route, T > 0}, {sorted_token_ids, rows_cap > 0},
                        {rows, rows_cap > 0}})))
    return rc;
  RowsArgs a{sorted_token_ids, num_tokens_post_padded, row_of_route, nullptr, T, K, rows_cap, top_k,
             n_shared};
  return launched(launch_permute(elem, a, x, rows, static_cast<hipStream_t>(stream)));
}

int moe_permute_backward(int32_t elem, const void* d_rows, const int32_t* row_of_route, void* d_x,
                         int64_t T, int64_t K, int32_t top_k, int32_t n_shared, int64_t rows_cap,
                         void* stream) {
  return moe_unpermute(elem, d_rows, row_of_route, nullptr, d_x, T, K, top_k, n_shared, rows_cap,
                       stream);
}

int moe_unpermute(int32_t elem, const void* rows, const int32_t* row_of_route,
                  const float* topk_weights, void* out, int64_t T, int64_t K, int32_t top_k,
                  int32_t n_shared, int64_t rows_cap, void* stream) {
  int rc = check_rows(elem, T, K, top_k, n_shared, rows_cap, true);
  if (rc) return rc;
  if ((rc = check_ptrs({{rows, T > 0 && rows_cap > 0}, {row_of_route, false}, {topk_weights, false},
                        {out, T > 0}})))
    return rc;
  RowsArgs a{nullptr, nullptr, row_of_route, topk_weights, T, K, rows_cap, top_k, n_shared};
  return launched(launch_unpermute(elem, a, rows, out, static_cast<hipStream_t>(stream)));
}

int moe_unpermute_backward(int32_t elem, const void* d_out, const void* rows,
                           const int32_t* row_of_route, const int32_t* sorted_token_ids,
                           const int32_t* num_tokens_post_padded, const float* topk_weights,
                           void* d_rows, float* d_weights, int64_t T, int64_t K, int32_t top_k,
                           int32_t n_shared, int64_t rows_cap, void* stream) {
  int rc = check_rows(elem, T, K, top_k, n_shared, rows_cap, true);
  if (rc) return rc;
  if ((rc = check_ntp(num_tokens_post_padded))) return rc;
  if ((rc = check_ptrs({{d_out, T > 0}, {rows, d_weights && rows_cap > 0}, {row_of_route, T > 0},
                        {sorted_token_ids, rows_cap > 0}, {topk_weights, false},
                        {d_rows, rows_cap > 0}, {d_weights, false}})))
    return rc;
  RowsArgs a{sorted_token_ids, num_tokens_post_padded, row_of_route, topk_weights, T, K, rows_cap,
             top_k, n_shared};
  return launched(launch_unpermute_backward(elem, a, d_out, rows, d_rows, d_weights,
                                            static_cast<hipStream_t>(stream)));
}

int moe_route_backward(const int32_t* topk_ids, const float* topk_weights, const float* d_weights,
                       float* d_logits, int64_t T, int32_t E, int32_t top_k, void* stream) {
  if (T < 0) return abi_fail(MOE_ERR_SHAPE, "T must be >= 0 (got %lld)", (long long)T);
  if (E < 1) return abi_fail(MOE_ERR_SHAPE, "E must be >= 1 (got %d)", E);
  if (top_k < 1) return abi_fail(MOE_ERR_SHAPE, "top_k must be >= 1 (got %d)", top_k);
  if ((T + 3) / 4 > kMaxGroups)  // a workgroup has four tokens
    return abi_fail(MOE_ERR_UNSUPPORTED, "moe_route_backward needs T <= 2^26 - 4");
  if (E > 1024) return abi_fail(MOE_ERR_UNSUPPORTED, "moe_route_backward supports E <= 1024 (got %d)", E);
  if (top_k > 16)
    return abi_fail(MOE_ERR_UNSUPPORTED, "moe_route_backward needs top_k <= 16 (got %d)", top_k);
  int rc = check_ptrs({{topk_ids, T > 0}, {topk_weights, T > 0}, {d_weights, T > 0}, {d_logits, T > 0}});
  if (rc) return rc;
  return launched(launch_route_backward(topk_ids, topk_weights, d_weights, d_logits, T, E, top_k,
                                        static_cast<hipStream_t>(stream)));
}

}  // extern "C"
