// route.hip -- the general router: softmax or sigmoid scores, a bias for
// balance, groups of experts, the top k, their weights; and its gradient.
//
// With l the logits of a token, masked where they are -inf or NaN:
//   s_e = softmax(l)_e or 1 / (1 + exp(-l_e)), 0 where masked
//   c_e = s_e + bias_e, the score that chooses
//   a group's score: the sum of its best one or two c; the topk_group best
//   groups keep their experts; the top_k largest c among those are chosen;
//   weights: s (not c) of the chosen, divided by their sum if wanted, times scale
// The choice compares c in 64 bits: scores of different experts often lie
// within fp32's last bits of each other (8,192 tokens of 256 experts: a pair at
// the border of the choice in about every eighth call), and a choice must not
// depend on how a 32-bit exponential rounds.
#include "device.h"
#include "ops.h"

namespace {

constexpr int kThreads = 256;  // four waves, a token each
typedef unsigned long long u64;

template <int ELEM>
__device__ __forceinline__ float load_as_f32(const void* p, int64_t i) {
  if constexpr (ELEM == ELEM_F32) return static_cast<const float*>(p)[i];
  if constexpr (ELEM == ELEM_F16) return (float)static_cast<const _Float16*>(p)[i];
  return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}

template <int ELEM>
__device__ __forceinline__ void store_f32(void* p, int64_t i, float v) {
  if constexpr (ELEM == ELEM_F32) static_cast<float*>(p)[i] = v;
  else if constexpr (ELEM == ELEM_F16) static_cast<_Float16*>(p)[i] = (_Float16)v;
  else static_cast<uint16_t*>(p)[i] = f32_to_bf16(v);
}

__device__ __forceinline__ float wave_max_f32(float v) {
  v = wave_max16(v);
  const int i = __float_as_int(v);
  return __builtin_fmaxf(
      __builtin_fmaxf(__int_as_float(__builtin_amdgcn_readlane(i, 0)),
                      __int_as_float(__builtin_amdgcn_readlane(i, 16))),
      __builtin_fmaxf(__int_as_float(__builtin_amdgcn_readlane(i, 32)),
                      __int_as_float(__builtin_amdgcn_readlane(i, 48))));
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// Largest 32-bit value over the wave, in a scalar register.
template <int CTRL>
__device__ __forceinline__ uint32_t umax_dpp(uint32_t v) {
  const uint32_t u = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
  return v > u ? v : u;
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  v = umax_dpp<0xB1>(v);   // quad_perm [1, 0, 3, 2]
  v = umax_dpp<0x4E>(v);   // quad_perm [2, 3, 0, 1]
  v = umax_dpp<0x124>(v);  // row_ror 4
  v = umax_dpp<0x128>(v);  // row_ror 8
  const uint32_t a = __builtin_amdgcn_readlane((int)v, 0), b = __builtin_amdgcn_readlane((int)v, 16);
  const uint32_t c = __builtin_amdgcn_readlane((int)v, 32), d = __builtin_amdgcn_readlane((int)v, 48);
  const uint32_t ab = a > b ? a : b, cd = c > d ? c : d;
  return ab > cd ? ab : cd;
}

// A double's bits in an order that unsigned comparison follows; 0 for none (only
// a NaN would come out as 0).
__device__ __forceinline__ u64 order_key(double c) {
  const u64 b = __builtin_bit_cast(u64, c);
  return b ^ ((b >> 63) ? ~0ull : 0x8000000000000000ull);
}

// A logit, or -inf where it is masked; +inf counts as fp32's largest, so that a
// softmax over it stays defined.
__device__ __forceinline__ float clean_logit(float l) {
  return l > -INFINITY ? __builtin_fminf(l, 3.402823466e38f) : -INFINITY;
}

// One wave a token; lane holds experts lane, lane + 64, .. in NV registers.
template <int ELEM, int NV, bool SIGMOID, bool GROUPED>
__global__ void __launch_bounds__(kThreads)
k_route_topk(RouteArgs a, int32_t* __restrict__ ids, float* __restrict__ weights) {
  __shared__ double lds[GROUPED ? kThreads / 64 : 1][GROUPED ? NV * 64 : 1];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int64_t t = (int64_t)blockIdx.x * (kThreads / 64) + wave;
  if (t >= a.T) return;
  const int E = a.E;
  float l[NV];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 64 * i;
    l[i] = e < E ? clean_logit(load_as_f32<ELEM>(a.logits, t * E + e)) : -INFINITY;
    top = __builtin_fmaxf(top, l[i]);
  }
  double s[NV];
  double total = 0.0, inv = 1.0;
  if constexpr (!SIGMOID) {
    top = wave_max_f32(top);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      s[i] = l[i] > -INFINITY ? exp((double)l[i] - (double)top) : 0.0;
      total += s[i];
    }
    total = wave_sum_f64(total);
    inv = total > 0.0 ? 1.0 / total : 0.0;
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] = 1.0 / (1.0 + exp(-(double)l[i]));
  }
  u64 key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 64 * i;
    double c = s[i] * inv;
    if (a.bias && e < E) c += (double)a.bias[e];
    if (!(l[i] > -INFINITY) || !(c > -INFINITY)) c = -INFINITY;
    key[i] = c > -INFINITY ? order_key(c) : 0;
    if constexpr (GROUPED) lds[wave][e] = c;
  }
  if constexpr (GROUPED) {
    // P lanes share a group: each finds the best two of every P-th expert, then
    // the lanes' are merged.  P = 64 / (n_group rounded up to a power of two).
    wave_lds_fence();
    const int G = a.n_group, S = E / G;
    int lg = 0;
    while ((1 << lg) < G) ++lg;
    const int P = 64 >> lg, grp = lane / P;
    double b1 = -INFINITY, b2 = -INFINITY;
    if (grp < G)
      for (int j = lane % P; j < S; j += P) {
        const double c = lds[wave][grp * S + j];
        if (c > b1) { b2 = b1; b1 = c; }
        else if (c > b2) b2 = c;
      }
    for (int d = 1; d < P; d <<= 1) {
      const double o1 = __shfl_xor(b1, d), o2 = __shfl_xor(b2, d);
      const double lo = b1 > o1 ? o1 : b1;
      b1 = b1 > o1 ? b1 : o1;
      const double hi2 = b2 > o2 ? b2 : o2;
      b2 = lo > hi2 ? lo : hi2;
    }
    if (a.group_top == 2 && b2 > -INFINITY) b1 += b2;
    // a group is kept if fewer than topk_group groups come before it
    int before = 0;
    for (int g = 0; g < G; ++g) {
      const double o = __shfl(b1, g * P);
      before += (o > b1) || (o == b1 && g < grp);
    }
    u64 kept = 0;
    const u64 mine = __ballot(grp < G && before < a.topk_group);
    for (int g = 0; g < G; ++g) kept |= ((mine >> (g * P)) & 1ull) << g;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !((kept >> (e / S)) & 1ull)) key[i] = 0;
    }
  }
  // top_k times the largest key; equal keys go to the lowest expert
  int id = -1;
  for (int j = 0; j < a.top_k; ++j) {
    u64 best = 0;
    int slot = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (key[i] > best) { best = key[i]; slot = i; }
    const uint32_t hi = (uint32_t)(best >> 32), top_hi = wave_umax(hi);
    if (top_hi == 0) break;  // no candidate is left (every score's key has a high half above 0)
    u64 who = __ballot(hi == top_hi);
    if (who & (who - 1)) {
      const uint32_t lo = hi == top_hi ? (uint32_t)best : 0u, top_lo = wave_umax(lo);
      who = __ballot(hi == top_hi && lo == top_lo);
      if (who & (who - 1)) {
        const uint32_t e = (who >> lane) & 1ull ? 0xFFFFu - (uint32_t)(lane + 64 * slot) : 0u;
        const uint32_t first = wave_umax(e);
        who = __ballot(e == first);
      }
    }
    const int win = __builtin_ctzll(who);
    const int e = win + 64 * __builtin_amdgcn_readlane(slot, win);
    if (lane == j) id = e;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane == win && slot == i) key[i] = 0;
  }
  // lane j: the weight of the j-th chosen
  double w = 0.0;
  const float lj = id >= 0 ? clean_logit(load_as_f32<ELEM>(a.logits, t * E + id)) : -INFINITY;
  if constexpr (SIGMOID) {
    if (id >= 0) w = 1.0 / (1.0 + exp(-(double)lj));
    if (a.renormalize) {
      const double sum = wave_sum_f64(w);
      w = sum > 0.0 ? w / sum : 0.0;
    }
  } else if (a.renormalize) {
    // the softmax over the chosen ones
    const float m = wave_max_f32(lj);
    if (id >= 0) w = exp((double)lj - (double)m);
    const double sum = wave_sum_f64(w);
    w = sum > 0.0 ? w / sum : 0.0;
  } else if (id >= 0) {
    w = exp((double)lj - (double)top) * inv;
  }
  if (lane < a.top_k) {
    ids[t * a.top_k + lane] = id;
    weights[t * a.top_k + lane] = (float)(w * (double)a.scale);
  }
}

// Gradient.  With g_j = scale (dw_j - <p, dw>) / S for renormalised weights (p_j =
// s_j / S, S the chosen scores' sum) and scale dw_j otherwise,
//   sigmoid  dl_e = g_e s_e (1 - s_e)          of the chosen e, else 0
//   softmax  dl_e = s_e (g_e - sum_j g_j s_j); renormalised, the sum is 0 and the
//            unchosen have no gradient
// One wave a token; a row is put together in LDS.  Lanes below top_k hold the
// chosen; an id outside [0, E) takes no part.
template <int ELEM, bool SIGMOID, bool DENSE>
__global__ void __launch_bounds__(kThreads)
k_route_topk_backward(RouteArgs a, const int32_t* __restrict__ ids, const float* __restrict__ dw,
                      void* __restrict__ d_logits) {
  __shared__ float lds[kThreads / 64][kRouteMaxExperts];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int64_t t = (int64_t)blockIdx.x * (kThreads / 64) + wave;
  if (t >= a.T) return;
  const int E = a.E;
  float* line = lds[wave];
  for (int e = lane; e < E; e += 64) line[e] = 0.f;
  int id = -1;
  double g = 0.0;
  float l = -INFINITY;
  if (lane < a.top_k) {
    id = ids[t * a.top_k + lane];
    if ((unsigned)id >= (unsigned)E) id = -1;
    if (id >= 0) {
      g = (double)dw[t * a.top_k + lane] * (double)a.scale;
      l = clean_logit(load_as_f32<ELEM>(a.logits, t * E + id));
    }
  }
  double d = 0.0;  // this lane's term
  float top = -INFINITY, inv = 0.f;
  if constexpr (SIGMOID) {
    const double z = exp(-(double)l), s = id >= 0 ? 1.0 / (1.0 + z) : 0.0;
    const double rest = id >= 0 ? 1.0 / (1.0 + exp((double)l)) : 0.0;  // 1 - s
    if (a.renormalize) {
      const double sum = wave_sum_f64(s);
      const double p = sum > 0.0 ? s / sum : 0.0;
      d = p * rest * (g - wave_sum_f64(p * g));
    } else {
      d = s * rest * g;
    }
  } else if constexpr (!DENSE) {
    const float m = wave_max_f32(l);
    const double x = l > -INFINITY ? exp((double)l - (double)m) : 0.0;
    const double sum = wave_sum_f64(x);
    const double p = sum > 0.0 ? x / sum : 0.0;
    d = p * (g - wave_sum_f64(p * g));
  } else {
    double sum = 0.0;
    for (int e = lane; e < E; e += 64)
      top = __builtin_fmaxf(top, clean_logit(load_as_f32<ELEM>(a.logits, t * E + e)));
    top = wave_max_f32(top);
    for (int e = lane; e < E; e += 64) {
      const float v = clean_logit(load_as_f32<ELEM>(a.logits, t * E + e));
      if (v > -INFINITY) sum += exp((double)v - (double)top);
    }
    sum = wave_sum_f64(sum);
    const double s = l > -INFINITY ? exp((double)l - (double)top) / sum : 0.0;
    d = g;
    const double mean = wave_sum_f64(g * s);
    inv = sum > 0.0 ? (float)(1.0 / sum) : 0.f;
    g = mean;
  }
  // an id that occurs more than once gets its terms' sum, in their order
  double mine = 0.0;
  for (int j = 0; j < a.top_k; ++j) {
    const int ij = __shfl(id, j);
    const double dj = __shfl(d, j);
    if (id == ij) mine += dj;
  }
  wave_lds_fence();
  if (id >= 0) line[id] = (float)mine;
  wave_lds_fence();
  for (int e = lane; e < E; e += 64) {
    float v = line[e];
    if constexpr (DENSE) {
      const float x = clean_logit(load_as_f32<ELEM>(a.logits, t * E + e));
      v = x > -INFINITY ? (float)(exp((double)x - (double)top) * (double)inv * ((double)v - g)) : 0.f;
    }
    store_f32<ELEM>(d_logits, t * E + e, v);
  }
}

template <int ELEM, int NV>
void route(const RouteArgs& a, int32_t* ids, float* w, hipStream_t stream) {
  const dim3 grid((unsigned)((a.T + kThreads / 64 - 1) / (kThreads / 64)));
  const bool sig = a.scoring == SCORE_SIGMOID, grouped = a.topk_group < a.n_group;
  auto go = [&](auto SIG, auto GRP) {
    hipLaunchKernelGGL((k_route_topk<ELEM, NV, SIG(), GRP()>), grid, dim3(kThreads), 0, stream, a, ids, w);
  };
  if (sig && grouped) go(std::true_type{}, std::true_type{});
  else if (sig) go(std::true_type{}, std::false_type{});
  else if (grouped) go(std::false_type{}, std::true_type{});
  else go(std::false_type{}, std::false_type{});
}

template <class F>
void by_elem(int elem, F f) {
  if (elem == ELEM_F32) f(std::integral_constant<int, ELEM_F32>{});
  else if (elem == ELEM_F16) f(std::integral_constant<int, ELEM_F16>{});
  else f(std::integral_constant<int, ELEM_BF16>{});
}

}  // namespace

hipError_t launch_route_topk(const RouteArgs& a, int32_t* ids, float* weights, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  by_elem(a.elem, [&](auto ELEM) {
    if (a.E <= 128) route<ELEM(), 2>(a, ids, weights, stream);
    else if (a.E <= 256) route<ELEM(), 4>(a, ids, weights, stream);
    else if (a.E <= 320) route<ELEM(), 5>(a, ids, weights, stream);
    else if (a.E <= 512) route<ELEM(), 8>(a, ids, weights, stream);
    else route<ELEM(), 16>(a, ids, weights, stream);
  });
  return hipGetLastError();
}

hipError_t launch_route_topk_backward(const RouteArgs& a, const int32_t* ids, const float* d_weights,
                                      void* d_logits, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  const dim3 grid((unsigned)((a.T + kThreads / 64 - 1) / (kThreads / 64)));
  by_elem(a.elem, [&](auto ELEM) {
    auto go = [&](auto SIG, auto DENSE) {
      hipLaunchKernelGGL((k_route_topk_backward<ELEM(), SIG(), DENSE()>), grid, dim3(kThreads), 0,
                         stream, a, ids, d_weights, d_logits);
    };
    if (a.scoring == SCORE_SIGMOID) go(std::true_type{}, std::false_type{});
    else if (a.renormalize) go(std::false_type{}, std::false_type{});
    else go(std::false_type{}, std::true_type{});
  });
  return hipGetLastError();
}
