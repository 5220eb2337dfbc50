// ops.h -- internal launchers of the operators around the plan (rows.hip), of
// the 4-bit products (w4.hip), the general router (route.hip), the 8-bit
// quantizers (quant.hip) and the 8-bit linear layers (fp8_linear.hip), and the
// error reporting they share with abi.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

// Records the message of a failing call and returns `code` / clears the
// message and returns MOE_OK (the calling thread's, as moe_last_error reads it).
int abi_fail(int code, const char* fmt, ...);
int abi_ok();

// Element types, in the order of moe_elem.
enum : int { ELEM_BF16 = 0, ELEM_F16 = 1, ELEM_F32 = 2, ELEM_U8 = 3 };
constexpr int elem_bytes(int elem) { return elem == ELEM_F32 ? 4 : elem == ELEM_U8 ? 1 : 2; }

// Routes of a plan: T tokens with top_k routed and n_shared shared routes
// each; route ids t * top_k + j, then T * top_k + t * n_shared + s.
struct RowsArgs {
  const int32_t* sorted;  // plan: route id of each row, -1 for padding
  const int32_t* ntp;     // rows in use (device scalar)
  const int32_t* row;     // row of each route, -1 where it has none (null: row r is route r)
  const float* w;         // (T, top_k) weights, or null for ones
  int64_t T, K, cap;      // tokens, columns, rows of the buffers
  int top_k, n_shared;
};

hipError_t launch_route_rows(const int32_t* ids, const RowsArgs& a, int E, int32_t* row,
                             hipStream_t stream);
hipError_t launch_permute(int elem, const RowsArgs& a, const void* x, void* rows,
                          hipStream_t stream);
hipError_t launch_unpermute(int elem, const RowsArgs& a, const void* rows, void* out,
                            hipStream_t stream);
hipError_t launch_unpermute_backward(int elem, const RowsArgs& a, const void* d_out,
                                     const void* rows, void* d_rows, float* d_w,
                                     hipStream_t stream);
hipError_t launch_route_backward(const int32_t* ids, const float* w, const float* dw,
                                 float* d_logits, int64_t T, int E, int top_k,
                                 hipStream_t stream);

// 4-bit weights: formats in the order of moe_w4_format.
enum : int { W4_INT = 0, W4_MX = 1 };

// Rows of K values, each as three bf16 parts p0 + p1 + 2 p2: (3, K) in the order
// the second product takes them.
constexpr int ELEM_PARTS = 4;

// One set of products y[r] = W[e(r)] x[r or its token] with 4-bit weights.
struct W4Args {
  const void* x;       // (T, K), or (R, K) with x_per_route; xelem
  const uint8_t* w;    // (E, N, K / 2)
  const void* scale;   // (E, N, K / group): scale_elem, or e8m0
  const uint8_t* zero; // (E, N, K / group), or null for 8
  const int32_t* ids;  // (R) expert of each route; null: one expert, every route
  void* out;           // (R, N), or (R, N / 2) with swiglu; oelem
  int K, N, E, R, top_k, group;
  int xelem, oelem, scale_elem;
  int x_per_route, swiglu;
  uint32_t inv_top_k;  // ceil(2^32 / top_k): r / top_k = umulhi(r, inv) for r < 4096 (top_k > 1)
};

constexpr int kW4MaxRoutes = 4096;  // routes of one call (a workgroup lists its expert's)
hipError_t launch_w4(int format, const W4Args& a, hipStream_t stream);
// The second product of the FFN and the weighted sum: a.x the intermediate (R,
// 3, K) in parts, a.out (T, N), out[t] = sum over t's routes with an expert in [0, E) of
// weights[r] W x[r].  y: R * N floats of workspace.  Up to kW4TokenMax tokens can
// take the kernel of a route per wave, which leaves y alone.
constexpr int kW4TokenMax = 4;
hipError_t launch_w4_down(int format, const W4Args& a, const float* weights, float* y, int T,
                          hipStream_t stream);

// The general router.  Scores in the order of moe_scoring.
enum : int { SCORE_SOFTMAX = 0, SCORE_SIGMOID = 1 };
constexpr int kRouteMaxExperts = 1024, kRouteMaxTopK = 16, kRouteMaxGroups = 64;

struct RouteArgs {
  const void* logits;  // (T, E) elem
  const float* bias;   // (E), or null
  int64_t T;
  int E, top_k, elem, scoring;
  int n_group, topk_group, group_top;
  int renormalize;
  float scale;
};

hipError_t launch_route_topk(const RouteArgs& a, int32_t* ids, float* weights, hipStream_t stream);
hipError_t launch_route_topk_backward(const RouteArgs& a, const int32_t* ids, const float* d_weights,
                                      void* d_logits, hipStream_t stream);

// Scales of 8-bit values, in the order of moe_scale_type.
enum : int { SCALE_F32 = 0, SCALE_E8M0 = 1 };
constexpr int scale_bytes(int type) { return type == SCALE_F32 ? 4 : 1; }

// e4m3 values of x (M, K) with a scale per 128 of a row (q) and, transposed, per
// 128 of a column (qt); either may be null.
struct QuantArgs {
  const void* x;
  const int32_t* ntp;  // rows in use (device scalar), or null for all
  uint8_t* q;          // (M, K)
  void* qs;            // (M, ceil(K / 128))
  uint8_t* qt;         // (K, Mp), Mp = M rounded up to 128
  void* qts;           // (K, Mp / 128)
  int64_t M, K;
  int elem, scale_type;
};
hipError_t launch_quant(const QuantArgs& a, hipStream_t stream);
// The same for weights (E, N, K) with a scale per 128 x 128 block: q (E, N, K), qs
// (E, NB, KB), and transposed (qt not null) qt (E, K, N), qts (E, KB, NB).
hipError_t launch_quant_weights(const void* w, int64_t E, int64_t N, int64_t K, int elem,
                                int scale_type, uint8_t* q, void* qs, uint8_t* qt, void* qts,
                                hipStream_t stream);

// out[m, n] = sum_k X[m, k] W[n, k] on e4m3 values with scales per 128 of k.
//   layer (dw = 0): X are rows, W the weights of one expert (a scale per 128 x
//     128 block); with a plan, block b of block_m rows takes expert experts[b].
//   gradient (dw = 1): X is dy transposed, W is x transposed (scales per row of
//     both), k the rows; with a plan, expert e sums over the rows of its blocks.
struct Fp8Args {
  const uint8_t* x;  // (M, K)
  const void* xs;    // (M, ceil(K / 128))
  const uint8_t* w;  // (E, N, K); dw: (N, K)
  const void* ws;    // (E, ceil(N / 128), ceil(K / 128)); dw: (N, K / 128)
  const int32_t* experts;  // expert of each block, or null (one layer)
  const int32_t* ntp;      // rows in use (device scalar)
  void* out;               // (M, N); dw: (E, M, N)
  int64_t M, N, K;
  int E, block_m, n_blocks;
  int oelem, scale_type, dw;
};
constexpr int kFp8MaxPlanExperts = 1024;  // of a gradient over a plan
hipError_t launch_fp8_linear(const Fp8Args& a, hipStream_t stream);
