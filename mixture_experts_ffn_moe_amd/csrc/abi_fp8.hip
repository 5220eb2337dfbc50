// abi_fp8.hip -- host side of the C ABI's 8-bit quantizers (moe_fp8_quant,
// moe_fp8_quant_weights) and linear layers (moe_fp8_linear, moe_fp8_linear_dw):
// argument checks before anything is enqueued, then the launch.
#include "abi_checks.h"

namespace {

constexpr int64_t kMaxSize = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxY = 65535;              // workgroups along a grid's second and third axis
constexpr int64_t kMaxContraction = int64_t(1) << 22;  // 256 rows of bytes: offsets of 32 bits
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;  // of one launch

int check_size(const char* name, int64_t n, int64_t least, int64_t multiple = 1) {
  if (n < least || n % multiple)
    return abi_fail(MOE_ERR_SHAPE, "%s must be at least %lld and a multiple of %lld (got %lld)", name,
                    (long long)least, (long long)multiple, (long long)n);
  if (n > kMaxSize) return abi_fail(MOE_ERR_UNSUPPORTED, "%s must be below 2^31", name);
  return MOE_OK;
}

int check_types(int32_t elem, int32_t last, int32_t scale_type) {
  if (elem < MOE_ELEM_BF16 || elem > last)
    return abi_fail(MOE_ERR_UNSUPPORTED, "unsupported element type %d", elem);
  if (scale_type != MOE_SCALE_F32 && scale_type != MOE_SCALE_E8M0)
    return abi_fail(MOE_ERR_UNSUPPORTED, "unknown scale type %d", scale_type);
  return MOE_OK;
}

int check_ntp(const int32_t* ntp, bool needed) {
  if (needed && !ntp) return abi_fail(MOE_ERR_NULL, "num_tokens_post_padded is NULL");
  if (ntp && !aligned(ntp, 4))
    return abi_fail(MOE_ERR_ALIGN, "num_tokens_post_padded must be 4-byte aligned");
  return MOE_OK;
}

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to; }

}  // namespace

extern "C" {

int moe_fp8_quant(int32_t elem, int32_t scale_type, const void* x, int64_t M, int64_t K,
                  const int32_t* num_tokens_post_padded, void* q, void* q_scale, void* qt,
                  void* qt_scale, void* stream) {
  int rc = check_types(elem, MOE_ELEM_F32, scale_type);
  if (rc) return rc;
  if ((rc = check_size("M", M, 0))) return rc;
  if ((rc = check_size("K", K, 16, 16))) return rc;
  if (qt ? up(M, 128) > kMaxY || up(M, 128) * up(K, 128) * 256 > kMaxThreads : M * up(K, 128) > kMaxThreads / 16)
    return abi_fail(MOE_ERR_UNSUPPORTED, "M * K is too large for one launch");
  if (!q && !qt && M > 0) return abi_fail(MOE_ERR_NULL, "neither q nor qt is given");
  if ((rc = check_ntp(num_tokens_post_padded, false))) return rc;
  if ((rc = check_ptrs({{x, M > 0}, {q, false}, {q_scale, q && M > 0}, {qt, false}, {qt_scale, qt && M > 0}})))
    return rc;
  QuantArgs a{x, num_tokens_post_padded, static_cast<uint8_t*>(q), q_scale, static_cast<uint8_t*>(qt),
              qt_scale, M, K, elem, scale_type};
  return launched(launch_quant(a, static_cast<hipStream_t>(stream)));
}

int moe_fp8_quant_weights(int32_t elem, int32_t scale_type, const void* w, int64_t E, int64_t N,
                          int64_t K, void* q, void* q_scale, void* qt, void* qt_scale,
                          void* stream) {
  int rc = check_types(elem, MOE_ELEM_F32, scale_type);
  if (rc) return rc;
  if ((rc = check_size("E", E, 0))) return rc;
  if ((rc = check_size("N", N, qt ? 16 : 1, qt ? 16 : 1))) return rc;
  if ((rc = check_size("K", K, 16, 16))) return rc;
  if (E > kMaxY || up(N, 128) > kMaxY || up(K, 128) > (int64_t(1) << 24) / 2 ||
      E * up(N, 128) > kMaxThreads / 256 / up(K, 128))
    return abi_fail(MOE_ERR_UNSUPPORTED, "the weights are too large for one launch");
  if ((rc = check_ptrs({{w, E > 0}, {q, E > 0}, {q_scale, E > 0}, {qt, false}, {qt_scale, qt && E > 0}})))
    return rc;
  return launched(launch_quant_weights(w, E, N, K, elem, scale_type, static_cast<uint8_t*>(q), q_scale,
                                       static_cast<uint8_t*>(qt), qt_scale,
                                       static_cast<hipStream_t>(stream)));
}

int moe_fp8_linear(int32_t elem, int32_t scale_type, const void* x, const void* x_scale,
                   const void* w, const void* w_scale, const int32_t* expert_ids,
                   const int32_t* num_tokens_post_padded, void* out, int64_t M, int64_t K, int64_t N,
                   int32_t E, int32_t block_m, void* stream) {
  int rc = check_types(elem, MOE_ELEM_F16, scale_type);
  if (rc) return rc;
  if ((rc = check_size("M", M, 0))) return rc;
  if ((rc = check_size("K", K, 16, 16))) return rc;
  if ((rc = check_size("N", N, 1))) return rc;
  if (K > kMaxContraction) return abi_fail(MOE_ERR_UNSUPPORTED, "K must be at most 2^22");
  if (E < 1) return abi_fail(MOE_ERR_SHAPE, "E must be >= 1 (got %d)", E);
  if (!expert_ids && E != 1)
    return abi_fail(MOE_ERR_SHAPE, "without expert_ids there is one expert (got E = %d)", E);
  if (expert_ids && block_m != 16 && block_m != 32 && block_m != 64 && block_m != 128 && block_m != 256)
    return abi_fail(MOE_ERR_UNSUPPORTED, "block_m must be 16, 32, 64, 128 or 256 (got %d)", block_m);
  const bool few = (expert_ids ? block_m : M) <= 32;  // a workgroup for each 16 rows of weights
  const bool blocks64 = expert_ids && block_m == 64;   // one for each block and 128 of them
  if (few ? up(M, 16) * 512 > kMaxThreads / up(N, 16)
          : up(M, 64) > (blocks64 ? kMaxThreads / 512 : kMaxSize) / up(N, 64))
    return abi_fail(MOE_ERR_UNSUPPORTED, "M * N is too large for one launch");
  if ((rc = check_ntp(num_tokens_post_padded, expert_ids != nullptr))) return rc;
  if ((rc = check_ptrs({{x, M > 0}, {x_scale, M > 0}, {w, M > 0}, {w_scale, M > 0}, {expert_ids, false},
                        {out, M > 0}})))
    return rc;
  Fp8Args a{static_cast<const uint8_t*>(x), x_scale, static_cast<const uint8_t*>(w), w_scale, expert_ids,
            num_tokens_post_padded, out, M, N, K, E, expert_ids ? block_m : 0,
            expert_ids ? (int)up(M, block_m) : 0, elem, scale_type, 0};
  return launched(launch_fp8_linear(a, static_cast<hipStream_t>(stream)));
}

int moe_fp8_linear_dw(int32_t elem, int32_t scale_type, const void* dyt, const void* dyt_scale,
                      const void* xt, const void* xt_scale, const int32_t* expert_ids,
                      const int32_t* num_tokens_post_padded, void* dw, int64_t M, int64_t N, int64_t K,
                      int32_t E, int32_t block_m, int64_t n_blocks, void* stream) {
  int rc = check_types(elem, MOE_ELEM_F16, scale_type);
  if (rc) return rc;
  if ((rc = check_size("M", M, 0, 128))) return rc;
  if ((rc = check_size("N", N, 1))) return rc;
  if ((rc = check_size("K", K, 1))) return rc;
  if (M > kMaxContraction) return abi_fail(MOE_ERR_UNSUPPORTED, "M must be at most 2^22");
  if (E < 1) return abi_fail(MOE_ERR_SHAPE, "E must be >= 1 (got %d)", E);
  if (!expert_ids && E != 1)
    return abi_fail(MOE_ERR_SHAPE, "without expert_ids there is one expert (got E = %d)", E);
  if (expert_ids && block_m != 128 && block_m != 256)
    return abi_fail(MOE_ERR_UNSUPPORTED,
                    "block_m must be 128 or 256, so that a scale's rows are one expert's (got %d)", block_m);
  if (expert_ids && E > kFp8MaxPlanExperts)
    return abi_fail(MOE_ERR_UNSUPPORTED, "a plan's gradient supports E <= %d (got %d)", kFp8MaxPlanExperts, E);
  if (expert_ids && (rc = check_size("n_blocks", n_blocks, 0))) return rc;
  if (up(N, 64) > kMaxSize / up(K, 64) / E)
    return abi_fail(MOE_ERR_UNSUPPORTED, "E * N * K is too large for one launch");
  if ((rc = check_ntp(num_tokens_post_padded, expert_ids != nullptr))) return rc;
  if ((rc = check_ptrs({{dyt, M > 0}, {dyt_scale, M > 0}, {xt, M > 0}, {xt_scale, M > 0},
                        {expert_ids, false}, {dw, true}})))
    return rc;
  // rows of the product: dy's columns; its columns: x's; summed over the rows
  Fp8Args a{static_cast<const uint8_t*>(dyt), dyt_scale, static_cast<const uint8_t*>(xt), xt_scale,
            expert_ids, num_tokens_post_padded, dw, N, K, M, E, expert_ids ? block_m : 0,
            expert_ids ? (int)n_blocks : 0, elem, scale_type, 1};
  return launched(launch_fp8_linear(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
