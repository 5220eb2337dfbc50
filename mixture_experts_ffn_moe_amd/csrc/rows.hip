// rows.hip -- tokens moved into the rows of a plan and back, with weights, and
// the gradients of both and of the router's weights.
//
// With p = row[r] the plan's row of route r (token t(r), weight w[r]; -1 where
// the route has no row):
//   permute             rows[p] = x[t(r)], padding rows 0
//   unpermute           out[t] = sum over t's routes of w[r] rows[row[r]]
//   permute backward    unpermute of the rows' gradient with weights 1
//   unpermute backward  d_rows[p] = w[r] d_out[t(r)], padding rows 0;
//                       d_w[r] = <rows[p], d_out[t(r)]>, 0 without a row
// All of them move rows of K elements and compute next to nothing, so bytes
// bound them.  Each walks the tokens, not the rows: a token's vector is then
// read (or its sum kept) once for all its routes, and no two workgroups write
// the same place, so no atomics and the same bits on every run.  Walking the
// rows instead would read x top_k times.  Sums are fp32 in route order with
// one rounding at the end.
#include <type_traits>

#include "device.h"
#include "ops.h"

namespace {

constexpr int kThreads = 256;
constexpr int kPadRows = 4;  // plan rows a workgroup looks over for padding

// 16 bytes of a row.  Rows whose pitch is a multiple of 16 bytes take the
// aligned type; others the same loads at the element's alignment, which the
// hardware allows.
typedef uint32_t vec_a __attribute__((ext_vector_type(4)));
template <int A>
struct VecOf;
template <>
struct VecOf<16> {
  typedef vec_a type;
};
template <>
struct VecOf<4> {
  typedef vec_a type __attribute__((aligned(4)));
};
template <>
struct VecOf<2> {
  typedef vec_a type __attribute__((aligned(2)));
};
template <>
struct VecOf<1> {
  typedef vec_a type __attribute__((aligned(1)));
};

// STREAM: past the caches, for rows that would only push each other out of them.
template <int A, bool STREAM = false>
__device__ __forceinline__ vec_a load_vec(const uint8_t* p) {
  auto q = reinterpret_cast<const typename VecOf<A>::type*>(p);
  if constexpr (STREAM) return __builtin_nontemporal_load(q);
  return *q;
}

template <int A, bool STREAM = false>
__device__ __forceinline__ void store_vec(uint8_t* p, vec_a v) {
  auto q = reinterpret_cast<typename VecOf<A>::type*>(p);
  if constexpr (STREAM) __builtin_nontemporal_store(v, q);
  else *q = v;
}

template <int ELEM>
__device__ __forceinline__ float load_elem(const uint8_t* p) {
  if constexpr (ELEM == ELEM_F32) return *reinterpret_cast<const float*>(p);
  else if constexpr (ELEM == ELEM_F16) return (float)*reinterpret_cast<const _Float16*>(p);
  else return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16);
}

template <int ELEM>
__device__ __forceinline__ void store_elem(uint8_t* p, float v) {
  if constexpr (ELEM == ELEM_F32) *reinterpret_cast<float*>(p) = v;
  else if constexpr (ELEM == ELEM_F16) *reinterpret_cast<_Float16*>(p) = (_Float16)v;
  else *reinterpret_cast<uint16_t*>(p) = f32_to_bf16(v);
}

// elements of a 16-byte vector
template <int ELEM>
constexpr int per_vec() { return 16 / elem_bytes(ELEM); }

template <int ELEM>
__device__ __forceinline__ void unpack(vec_a v, float (&f)[per_vec<ELEM>()]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (ELEM == ELEM_F32) {
      f[q] = __uint_as_float(v[q]);
    } else if constexpr (ELEM == ELEM_F16) {
      f[2 * q] = (float)__builtin_bit_cast(_Float16, (uint16_t)(v[q] & 0xFFFFu));
      f[2 * q + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(v[q] >> 16));
    } else {
      f[2 * q] = __uint_as_float(v[q] << 16);
      f[2 * q + 1] = __uint_as_float(v[q] & 0xFFFF0000u);
    }
  }
}

template <int ELEM>
__device__ __forceinline__ vec_a pack(const float (&f)[per_vec<ELEM>()]) {
  vec_a v;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (ELEM == ELEM_F32) {
      v[q] = __float_as_uint(f[q]);
    } else if constexpr (ELEM == ELEM_F16) {
      v[q] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f[2 * q]) |
             ((uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f[2 * q + 1]) << 16);
    } else {
      v[q] = (uint32_t)f32_to_bf16(f[2 * q]) | ((uint32_t)f32_to_bf16(f[2 * q + 1]) << 16);
    }
  }
  return v;
}

// The id of token t's j-th route, its row (or -1) and its weight.
__device__ __forceinline__ int64_t route_of(const RowsArgs& a, int64_t t, int j) {
  return j < a.top_k ? t * a.top_k + j : a.T * a.top_k + t * a.n_shared + (j - a.top_k);
}

__device__ __forceinline__ int64_t row_of(const RowsArgs& a, int64_t r) {
  const int64_t p = a.row ? (int64_t)a.row[r] : r;
  return p >= 0 && p < a.cap ? p : -1;
}

__device__ __forceinline__ float weight_of(const RowsArgs& a, int64_t r, int j) {
  return a.w && j < a.top_k ? a.w[r] : 1.f;
}

// Zeroes the plan's padding rows among kPadRows rows from p0.
template <int A, bool STREAM>
__device__ __forceinline__ void zero_padding(const RowsArgs& a, int64_t p0, uint8_t* rows,
                                             int64_t pitch) {
  const int64_t used = min((int64_t)*a.ntp, a.cap);
  for (int u = 0; u < kPadRows; ++u) {
    const int64_t p = p0 + u;
    if (p >= used) return;
    if (a.sorted[p] >= 0) continue;
    uint8_t* d = rows + p * pitch;
    const int64_t n16 = pitch / 16;
    for (int64_t c = threadIdx.x; c < n16; c += kThreads)
      store_vec<A, STREAM>(d + 16 * c, vec_a{0, 0, 0, 0});
    for (int64_t b = 16 * n16 + threadIdx.x; b < pitch; b += kThreads) d[b] = 0;
  }
}

__global__ void __launch_bounds__(kThreads)
k_route_rows(const int32_t* __restrict__ ids, RowsArgs a, int E, int32_t* __restrict__ row) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t R = a.T * a.top_k, RT = R + a.T * a.n_shared;
  // a plan places exactly the routes whose expert is in [0, E), and every
  // shared one, so the two writes below never meet
  if (i < R && (unsigned)ids[i] >= (unsigned)E) row[i] = -1;
  if (i < a.cap && i < (int64_t)*a.ntp) {
    const int id = a.sorted[i];
    if (id >= 0 && id < RT) row[id] = (int32_t)i;
  }
}

// Workgroups [0, T * CB): the token blockIdx / CB, kThreads vectors of its
// columns; then one for each kPadRows rows of the plan.
// A token's row is n16 whole vectors and the elements behind them: thread c of
// the row has vector c, or element c - n16 of the rest.
template <int ES, int A, bool STREAM>
__global__ void __launch_bounds__(kThreads)
k_permute(RowsArgs a, const uint8_t* __restrict__ x, uint8_t* __restrict__ rows, int64_t pitch,
          int CB) {
  const int64_t b = blockIdx.x;
  if (b >= a.T * CB) {
    zero_padding<A, STREAM>(a, (b - a.T * CB) * kPadRows, rows, pitch);
    return;
  }
  const int64_t t = b / CB;
  const int64_t n16 = pitch / 16, c = (b % CB) * kThreads + threadIdx.x;
  const int nr = a.top_k + a.n_shared;
  if (c < n16) {
    const vec_a v = load_vec<A>(x + t * pitch + 16 * c);
    for (int j = 0; j < nr; ++j) {
      const int64_t p = row_of(a, route_of(a, t, j));
      if (p >= 0) store_vec<A, STREAM>(rows + p * pitch + 16 * c, v);
    }
  } else if (A < 16 && c - n16 < pitch % 16 / ES) {
    typedef typename std::conditional<ES == 4, uint32_t, typename std::conditional<ES == 2, uint16_t,
                                                                          uint8_t>::type>::type unit;
    const int64_t at = 16 * n16 + (c - n16) * ES;
    const unit v = *reinterpret_cast<const unit*>(x + t * pitch + at);
    for (int j = 0; j < nr; ++j) {
      const int64_t p = row_of(a, route_of(a, t, j));
      if (p >= 0) *reinterpret_cast<unit*>(rows + p * pitch + at) = v;
    }
  }
}

template <int ELEM, int A, bool STREAM>
__global__ void __launch_bounds__(kThreads)
k_unpermute(RowsArgs a, const uint8_t* __restrict__ rows, uint8_t* __restrict__ out, int CB) {
  constexpr int V = per_vec<ELEM>(), ES = elem_bytes(ELEM), kBatch = 8;
  const int64_t b = blockIdx.x, t = b / CB, pitch = a.K * ES;
  const int64_t n16 = pitch / 16, c = (b % CB) * kThreads + threadIdx.x;
  const int nr = a.top_k + a.n_shared;
  if (c < n16) {
    float s[V];
#pragma unroll
    for (int e = 0; e < V; ++e) s[e] = 0.f;
    // kBatch routes' rows are requested before any is added
    for (int j0 = 0; j0 < nr; j0 += kBatch) {
      vec_a y[kBatch];
      float w[kBatch];
      bool placed[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        placed[u] = false;
        if (j0 + u < nr) {
          const int64_t r = route_of(a, t, j0 + u), p = row_of(a, r);
          if (p >= 0) {
            placed[u] = true;
            w[u] = weight_of(a, r, j0 + u);
            y[u] = load_vec<A, STREAM>(rows + p * pitch + 16 * c);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (!placed[u]) continue;
        float f[V];
        unpack<ELEM>(y[u], f);
#pragma unroll
        for (int e = 0; e < V; ++e) s[e] += w[u] * f[e];
      }
    }
    store_vec<A>(out + t * pitch + 16 * c, pack<ELEM>(s));
  } else if (A < 16 && c - n16 < a.K % V) {  // an element behind the whole vectors
    const int64_t at = (n16 * V + (c - n16)) * ES;
    float s = 0.f;
    for (int j0 = 0; j0 < nr; j0 += kBatch) {
      float y[kBatch], w[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        y[u] = w[u] = 0.f;
        if (j0 + u < nr) {
          const int64_t r = route_of(a, t, j0 + u), p = row_of(a, r);
          if (p >= 0) {
            w[u] = weight_of(a, r, j0 + u);
            y[u] = load_elem<ELEM>(rows + p * pitch + at);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) s += w[u] * y[u];
    }
    store_elem<ELEM>(out + t * pitch + at, s);
  }
}

// Workgroups [0, T * JG): token blockIdx / JG, its JB routes from
// (blockIdx % JG) * JB; then one for each kPadRows rows of the plan.
// With DW the dot products too.
template <int ELEM, int A, int JB, bool DW, bool STREAM>
__global__ void __launch_bounds__(kThreads)
k_unpermute_backward(RowsArgs a, const uint8_t* __restrict__ d_out,
                     const uint8_t* __restrict__ rows, uint8_t* __restrict__ d_rows,
                     float* __restrict__ d_w, int JG) {
  constexpr int V = per_vec<ELEM>(), ES = elem_bytes(ELEM), kW = kThreads / 64;
  const int64_t pitch = a.K * ES, n16 = pitch / 16, b = blockIdx.x;
  if (b >= a.T * JG) {
    zero_padding<A, STREAM>(a, (b - a.T * JG) * kPadRows, d_rows, pitch);
    return;
  }
  const int64_t t = b / JG;
  const int j0 = (int)(b % JG) * JB, nr = a.top_k + a.n_shared;
  int64_t p[JB];
  float w[JB], dot[JB];
#pragma unroll
  for (int u = 0; u < JB; ++u) {
    p[u] = -1;
    dot[u] = 0.f;
    if (j0 + u < nr) {
      const int64_t r = route_of(a, t, j0 + u);
      p[u] = row_of(a, r);
      w[u] = weight_of(a, r, j0 + u);
    }
  }
  for (int64_t c = threadIdx.x; c < n16; c += kThreads) {
    const vec_a g = load_vec<A>(d_out + t * pitch + 16 * c);
    vec_a y[JB];
    if constexpr (DW) {
#pragma unroll
      for (int u = 0; u < JB; ++u)
        if (p[u] >= 0) y[u] = load_vec<A, STREAM>(rows + p[u] * pitch + 16 * c);
    }
    float f[V];
    unpack<ELEM>(g, f);
#pragma unroll
    for (int u = 0; u < JB; ++u) {
      if (p[u] < 0) continue;
      float d[V];
#pragma unroll
      for (int e = 0; e < V; ++e) d[e] = w[u] * f[e];
      store_vec<A, STREAM>(d_rows + p[u] * pitch + 16 * c, pack<ELEM>(d));
      if constexpr (DW) {
        float h[V];
        unpack<ELEM>(y[u], h);
#pragma unroll
        for (int e = 0; e < V; ++e) dot[u] += h[e] * f[e];
      }
    }
  }
  for (int64_t e = n16 * V + threadIdx.x; e < a.K; e += kThreads) {
    const float f = load_elem<ELEM>(d_out + t * pitch + e * ES);
#pragma unroll
    for (int u = 0; u < JB; ++u) {
      if (p[u] < 0) continue;
      store_elem<ELEM>(d_rows + p[u] * pitch + e * ES, w[u] * f);
      if constexpr (DW) dot[u] += load_elem<ELEM>(rows + p[u] * pitch + e * ES) * f;
    }
  }
  if constexpr (DW) {
    __shared__ float part[kW][JB];
#pragma unroll
    for (int u = 0; u < JB; ++u) {
      if (j0 + u >= a.top_k) break;  // shared routes have no weight of their own
      const float s = wave_sum(dot[u]);
      if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6][u] = s;
    }
    __syncthreads();
    const int u = threadIdx.x;
    if (u < JB && j0 + u < a.top_k) {
      float s = 0.f;
      for (int v = 0; v < kW; ++v) s += part[v][u];
      d_w[t * a.top_k + j0 + u] = s;
    }
  }
}

// d_logits[t, e] = sum over j with ids[t, j] = e of w_j (dw_j - <w, dw>): the
// gradient of a softmax over the selected logits, which is what the
// normalized routing weights are.  4 T E bytes of output bound it.  One wave a
// token; lane j < top_k holds route j and adds the terms of the routes with its
// id in their order, so that an id that occurs twice needs no atomics.  The row
// is put together in LDS: comparing every output with every route's id instead
// made the vector units the bound (8,192 tokens, 288 experts, top-8: 8.0 us).
constexpr int kMaxTopK = 16;
constexpr int kMaxExperts = 1024;

template <int A>
__global__ void __launch_bounds__(kThreads)
k_route_backward(const int32_t* __restrict__ ids, const float* __restrict__ w,
                 const float* __restrict__ dw, float* __restrict__ d_logits, int64_t T, int E,
                 int top_k) {
  __shared__ __align__(16) float lds[kThreads / 64][kMaxExperts];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int64_t t = (int64_t)blockIdx.x * (kThreads / 64) + wave;
  if (t >= T) return;
  int id = -1;
  float wj = 0.f, gj = 0.f;
  if (lane < top_k) {
    id = ids[t * top_k + lane];
    wj = w[t * top_k + lane];
    gj = dw[t * top_k + lane];
  }
  float* line = lds[wave];  // the wave's own: its LDS operations stay in order
  for (int e = lane * 4; e < E; e += 256)
    *reinterpret_cast<float4*>(line + e) = make_float4(0.f, 0.f, 0.f, 0.f);
  const float mean = wave_sum(wj * gj);
  const float d = wj * (gj - mean);
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j) {
    if (j >= top_k) break;
    const int ij = __builtin_amdgcn_readlane(id, j);
    const float dj = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(d), j));
    if (id == ij) s += dj;
  }
  wave_lds_fence();
  if (lane < top_k && (unsigned)id < (unsigned)E) line[id] = s;
  wave_lds_fence();
  float* row = d_logits + t * E;
  constexpr int V = A / 4;
  for (int e = lane * V; e < E; e += 64 * V) {
    if constexpr (V == 4)
      *reinterpret_cast<float4*>(row + e) = *reinterpret_cast<const float4*>(line + e);
    else
      row[e] = line[e];
  }
}

// Whether the routes' rows are streamed past the caches: once they outgrow the
// 256 MiB memory-side cache.  Measured at K = 4096, top-8 (permute, then
// unpermute): 8,192 tokens (537 MB) 225 us streamed against 264, 4,096 tokens
// 119 against 145; 2,048 tokens (134 MB), whose rows the second call finds in the
// cache, 61 against 56, and 64 tokens 29 against 23.
// Every route counts as placed, since the host does not know how many are.  Three
// quarters of them elsewhere, the same calls and the weighted sum's gradient:
// 4,096 tokens (67 MB placed) 46 us streamed against 44 and 41 against 33, 8,192
// tokens (133 MB) 82 against 81 and 74 against 79, 16,384 156 against 172 and 145
// against 158.
bool streams(const RowsArgs& a, int64_t pitch) {
  return a.T * (a.top_k + a.n_shared) * pitch > (int64_t(192) << 20);
}

// workgroups of a token's row: its vectors and the elements behind them
int col_blocks(int64_t pitch, int es) {
  return (int)((pitch / 16 + pitch % 16 / es + kThreads - 1) / kThreads);
}

// Runs f<alignment of a row's vectors, STREAM>: 16 bytes where the pitch keeps
// it, else the element's (A < 16, never streamed.  8,192 tokens, top-8, bf16,
// permute and unpermute: K = 4100 282 us streamed against 280, K = 4099 300
// against 281; 2,048 tokens 113 against 88 and 119 against 92).
template <int ES, class F>
hipError_t by_pitch(const RowsArgs& a, int64_t pitch, F f) {
  typedef std::integral_constant<int, 16> whole;
  typedef std::integral_constant<int, ES> element;
  if (pitch % 16) f(element{}, std::false_type{});
  else if (streams(a, pitch)) f(whole{}, std::true_type{});
  else f(whole{}, std::false_type{});
  return hipGetLastError();
}

template <int ELEM, int A, bool STREAM>
void unpermute_backward(const RowsArgs& a, const void* d_out, const void* rows, void* d_rows,
                        float* d_w, hipStream_t stream) {
  constexpr int JB = 8;
  const int JG = (int)(((int64_t)a.top_k + a.n_shared + JB - 1) / JB);
  const dim3 grid((unsigned)(a.T * JG + (a.cap + kPadRows - 1) / kPadRows));
  auto g = static_cast<const uint8_t*>(d_out);
  auto y = static_cast<const uint8_t*>(rows);
  auto d = static_cast<uint8_t*>(d_rows);
  if (d_w)
    hipLaunchKernelGGL((k_unpermute_backward<ELEM, A, JB, true, STREAM>), grid, dim3(kThreads), 0,
                       stream, a, g, y, d, d_w, JG);
  else
    hipLaunchKernelGGL((k_unpermute_backward<ELEM, A, JB, false, STREAM>), grid, dim3(kThreads), 0,
                       stream, a, g, y, d, d_w, JG);
}

template <int ES>
hipError_t permute(const RowsArgs& a, const void* x, void* rows, hipStream_t stream) {
  const int64_t pitch = a.K * ES;
  const int CB = col_blocks(pitch, ES);
  const dim3 grid((unsigned)(a.T * CB + (a.cap + kPadRows - 1) / kPadRows));
  if (grid.x == 0) return hipSuccess;
  return by_pitch<ES>(a, pitch, [&](auto A, auto STREAM) {
    hipLaunchKernelGGL((k_permute<ES, A(), STREAM()>), grid, dim3(kThreads), 0, stream, a,
                       static_cast<const uint8_t*>(x), static_cast<uint8_t*>(rows), pitch, CB);
  });
}

template <int ELEM>
hipError_t unpermute(const RowsArgs& a, const void* rows, void* out, hipStream_t stream) {
  constexpr int ES = elem_bytes(ELEM);
  const int64_t pitch = a.K * ES;
  const int CB = col_blocks(pitch, ES);
  const dim3 grid((unsigned)(a.T * CB));
  if (grid.x == 0) return hipSuccess;
  return by_pitch<ES>(a, pitch, [&](auto A, auto STREAM) {
    hipLaunchKernelGGL((k_unpermute<ELEM, A(), STREAM()>), grid, dim3(kThreads), 0, stream, a,
                       static_cast<const uint8_t*>(rows), static_cast<uint8_t*>(out), CB);
  });
}

}  // namespace

hipError_t launch_route_rows(const int32_t* ids, const RowsArgs& a, int E, int32_t* row,
                             hipStream_t stream) {
  const int64_t n = a.cap > a.T * a.top_k ? a.cap : a.T * a.top_k;
  if (n == 0) return hipSuccess;
  hipLaunchKernelGGL(k_route_rows, dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads),
                     0, stream, ids, a, E, row);
  return hipGetLastError();
}

hipError_t launch_permute(int elem, const RowsArgs& a, const void* x, void* rows,
                          hipStream_t stream) {
  if (elem == ELEM_F32) return permute<4>(a, x, rows, stream);
  if (elem == ELEM_U8) return permute<1>(a, x, rows, stream);
  return permute<2>(a, x, rows, stream);
}

hipError_t launch_unpermute(int elem, const RowsArgs& a, const void* rows, void* out,
                            hipStream_t stream) {
  if (elem == ELEM_F32) return unpermute<ELEM_F32>(a, rows, out, stream);
  if (elem == ELEM_F16) return unpermute<ELEM_F16>(a, rows, out, stream);
  return unpermute<ELEM_BF16>(a, rows, out, stream);
}

hipError_t launch_unpermute_backward(int elem, const RowsArgs& a, const void* d_out,
                                     const void* rows, void* d_rows, float* d_w,
                                     hipStream_t stream) {
  if (a.T == 0 && a.cap == 0) return hipSuccess;
  auto run = [&](auto ELEM) {
    constexpr int ES = elem_bytes(ELEM());
    return by_pitch<ES>(a, a.K * ES, [&](auto A, auto STREAM) {
      unpermute_backward<ELEM(), A(), STREAM()>(a, d_out, rows, d_rows, d_w, stream);
    });
  };
  if (elem == ELEM_F32) return run(std::integral_constant<int, ELEM_F32>{});
  if (elem == ELEM_F16) return run(std::integral_constant<int, ELEM_F16>{});
  return run(std::integral_constant<int, ELEM_BF16>{});
}

hipError_t launch_route_backward(const int32_t* ids, const float* w, const float* dw,
                                 float* d_logits, int64_t T, int E, int top_k,
                                 hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const dim3 grid((unsigned)((T + kThreads / 64 - 1) / (kThreads / 64)));
  if (E % 4 == 0)
    hipLaunchKernelGGL(k_route_backward<16>, grid, dim3(kThreads), 0, stream, ids, w, dw, d_logits,
                       T, E, top_k);
  else
    hipLaunchKernelGGL(k_route_backward<4>, grid, dim3(kThreads), 0, stream, ids, w, dw, d_logits,
                       T, E, top_k);
  return hipGetLastError();
}
