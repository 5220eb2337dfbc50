// ops.h -- internal launchers of the operators around the plan (rows.hip) and
// of the 4-bit products (w4.hip), and the error reporting they share with
// abi.hip.
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
