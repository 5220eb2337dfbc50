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
#include <type_traits>

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

// Four at i, a multiple of four.
template <int ELEM>
__device__ __forceinline__ void store4_f32(void* p, int64_t i, float4 v) {
  if constexpr (ELEM == ELEM_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = v;
  } else {
    auto bits = [](float x) -> uint32_t {
      if constexpr (ELEM == ELEM_F16) return __builtin_bit_cast(uint16_t, (_Float16)x);
      else return f32_to_bf16(x);
    };
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) =
        make_uint2(bits(v.x) | bits(v.y) << 16, bits(v.z) | bits(v.w) << 16);
  }
}

// The value lane movement CTRL (a DPP control) brings in.
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  const u64 b = __builtin_bit_cast(u64, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)b, CTRL, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, true);
  return __builtin_bit_cast(double, (u64)hi << 32 | lo);
}
constexpr int kSwap1 = 0xB1, kSwap2 = 0x4E;         // quad_perm: lanes 1 and 2 apart
constexpr int kMirror8 = 0x141, kMirror16 = 0x140;  // row_half_mirror, row_mirror

__device__ __forceinline__ double read_f64(double v, int lane) {
  const u64 b = __builtin_bit_cast(u64, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, (u64)hi << 32 | lo);
}

// Sum over each 16 lanes, in all of them: the pairs of mirrored lanes hold equal
// sums of equal parts.
__device__ __forceinline__ double sum16_f64(double v) {
  v += dpp_f64<kSwap1>(v);
  v += dpp_f64<kSwap2>(v);
  v += dpp_f64<kMirror8>(v);
  return v + dpp_f64<kMirror16>(v);
}
__device__ __forceinline__ double wave_sum_f64(double v) {
  v = sum16_f64(v);
  return (read_f64(v, 0) + read_f64(v, 16)) + (read_f64(v, 32) + read_f64(v, 48));
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

template <int CTRL>
__device__ __forceinline__ uint32_t umax_dpp(uint32_t v) {
  const uint32_t u = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
  return v > u ? v : u;
}
// Largest value over the wave, in a scalar register.
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  v = umax_dpp<kSwap1>(v);
  v = umax_dpp<kSwap2>(v);
  v = umax_dpp<kMirror8>(v);
  v = umax_dpp<kMirror16>(v);
  const uint32_t a = __builtin_amdgcn_readlane((int)v, 0), b = __builtin_amdgcn_readlane((int)v, 16);
  const uint32_t c = __builtin_amdgcn_readlane((int)v, 32), d = __builtin_amdgcn_readlane((int)v, 48);
  const uint32_t ab = a > b ? a : b, cd = c > d ? c : d;
  return ab > cd ? ab : cd;
}

// e^x in 64 bits, within 2 units in the last place: x = n ln 2 + r with ln 2 in two
// parts (Cody and Waite's reduction with the parts of fdlibm's e_exp.c: the first has 32
// bits, so that n times it is exact), the Taylor polynomial of e^r to r^13 (|r| <= ln 2 /
// 2: the next term is below 2^-57), and 2^n.  Infinite past 709.8, 0 below -745.2; no NaN.
__device__ __forceinline__ double exp_f64(double x) {
  x = __builtin_fmin(__builtin_fmax(x, -800.0), 800.0);
  const double n = __builtin_rint(x * 1.4426950408889634074);
  double r = __builtin_fma(n, -6.93147180369123816490e-01, x);
  r = __builtin_fma(n, -1.90821492927058770002e-10, r);
  double p = 1.0 / 6227020800.0;
  p = __builtin_fma(p, r, 1.0 / 479001600.0);
  p = __builtin_fma(p, r, 1.0 / 39916800.0);
  p = __builtin_fma(p, r, 1.0 / 3628800.0);
  p = __builtin_fma(p, r, 1.0 / 362880.0);
  p = __builtin_fma(p, r, 1.0 / 40320.0);
  p = __builtin_fma(p, r, 1.0 / 5040.0);
  p = __builtin_fma(p, r, 1.0 / 720.0);
  p = __builtin_fma(p, r, 1.0 / 120.0);
  p = __builtin_fma(p, r, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_ldexp(p, (int)n);
}

__device__ __forceinline__ double sigmoid_f64(float l) { return 1.0 / (1.0 + exp_f64(-(double)l)); }

// A double's bits in an order that unsigned comparison follows; every number's
// high half is above 0.
__device__ __forceinline__ u64 order_key(double c) {
  const u64 b = __builtin_bit_cast(u64, c);
  return b ^ ((b >> 63) ? ~0ull : 0x8000000000000000ull);
}

// A logit, or -inf where it is masked; +inf counts as fp32's largest, so that a
// softmax over it stays defined.
__device__ __forceinline__ float clean_logit(float l) {
  return l > -INFINITY ? __builtin_fminf(l, 3.402823466e38f) : -INFINITY;
}

// (b1, b2), a lane's best two, merged with those of the lane that CTRL brings in.
template <int CTRL>
__device__ __forceinline__ void merge_top2(double& b1, double& b2) {
  const double o1 = dpp_f64<CTRL>(b1), o2 = dpp_f64<CTRL>(b2);
  b2 = __builtin_fmax(__builtin_fmin(b1, o1), __builtin_fmax(b2, o2));
  b1 = __builtin_fmax(b1, o1);
}

// One wave a token.  The lanes are shared out to the groups, P = 2^lp for each, and
// a group's experts to its lanes in turn: lane holds slots i = 0 .. NV - 1, expert
// (lane / P) S + lane % P + P i of S a group.  (No groups: P = 64, S = E.)  So a
// group's best two meet in the row of lanes that hold it, and dropping a group is
// a lane's own business.
//
// The k-th best is found k times, by the high halves of the scores' keys: one
// maximum over the wave in 32 bits.  Where more than one expert has that high half
// (20 bits of the fraction), the low halves decide, then the experts' numbers.
//
// Each of the k rounds looks through all NV slots, so NV is the least of 2, 4, 5, 8, 16,
// 32 that holds a lane's experts.  8192 tokens, top-8, sigmoid, us by NV: 128 experts in 8
// groups 2: 9.5, 4: 11.9; 256 4: 12.1, 5: 13.4, 8: 17.0; 288 5: 13.5, 8: 17.1, 16: 27.5; 8 tokens
// of 256 4: 5.0, 5: 5.4.  Without groups: 256 experts 9.4 (softmax 10.9), 512, top-16, 8: 19.1, 16:
// 33.9; 1024 16: 24.4, 32: 59.3.
//
// 8192 tokens, 288 experts in 8 groups, top-8, sigmoid: 14 us, of which the launch and
// the loads are 5, the selection 4.7, the scores 2.3, the groups 1.1 and the weights 1:
// vector instructions and chains of lane movements, not bytes (9.5 MB, 2 us).  8 tokens:
// 5.1, one such chain.
template <int ELEM, int NV, bool SIGMOID, bool GROUPED>
__global__ void __launch_bounds__(kThreads)
k_route_topk(RouteArgs a, int lp, int32_t* __restrict__ ids, float* __restrict__ weights) {
  __shared__ double picked[kThreads / 64][kRouteMaxTopK];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int64_t t = (int64_t)blockIdx.x * (kThreads / 64) + wave;
  if (t >= a.T) return;
  const int E = a.E, G = GROUPED ? a.n_group : 1, S = GROUPED ? E / G : E, P = GROUPED ? 1 << lp : 64;
  const int grp = GROUPED ? lane >> lp : 0, sub = GROUPED ? lane & (P - 1) : lane;
  const int first = grp * S + sub;  // this lane's first expert
  float l[NV];
  double s[NV], c[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool here = sub + P * i < S && (!GROUPED || grp < G);
    l[i] = here ? load_as_f32<ELEM>(a.logits, t * E + first + P * i) : -INFINITY;
    c[i] = a.bias && here ? (double)a.bias[first + P * i] : 0.0;
  }
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    l[i] = clean_logit(l[i]);
    top = __builtin_fmaxf(top, l[i]);
  }
  double inv = 1.0;
  if constexpr (SIGMOID) {
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] = sigmoid_f64(l[i]);
  } else {
    top = wave_max_f32(top);
    double total = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      s[i] = l[i] > -INFINITY ? exp_f64((double)l[i] - (double)top) : 0.0;
      total += s[i];
    }
    total = wave_sum_f64(total);
    inv = total > 0.0 ? 1.0 / total : 0.0;
  }
  u64 key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if constexpr (!SIGMOID) s[i] *= inv;
    c[i] += s[i];
    if (!(l[i] > -INFINITY) || !(c[i] > -INFINITY)) c[i] = -INFINITY;
    key[i] = c[i] > -INFINITY ? order_key(c[i]) : 0;
  }
  if constexpr (GROUPED) {
    double b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      b2 = __builtin_fmax(b2, __builtin_fmin(b1, c[i]));
      b1 = __builtin_fmax(b1, c[i]);
    }
    if (lp > 0) merge_top2<kSwap1>(b1, b2);
    if (lp > 1) merge_top2<kSwap2>(b1, b2);
    if (lp > 2) merge_top2<kMirror8>(b1, b2);
    if (lp > 3) merge_top2<kMirror16>(b1, b2);
    if (lp > 4) {  // two groups
      const double o1 = __shfl_xor(b1, 16), o2 = __shfl_xor(b2, 16);
      b2 = __builtin_fmax(__builtin_fmin(b1, o1), __builtin_fmax(b2, o2));
      b1 = __builtin_fmax(b1, o1);
    }
    if (a.group_top == 2 && b2 > -INFINITY) b1 += b2;
    // a group is kept if fewer than topk_group groups come before it
    int before = 0;
    for (int g = 0; g < G; ++g) {
      const double o = read_f64(b1, g << lp);
      before += (int)(o > b1) + (int)(o == b1 && g < grp);
    }
    if (before >= a.topk_group) {
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] = 0;
    }
  }
  int id = -1;
  for (int j = 0; j < a.top_k; ++j) {
    uint32_t hi = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) hi = max(hi, (uint32_t)(key[i] >> 32));
    const uint32_t most = wave_umax(hi);
    if (most == 0) break;  // no candidate is left
    u64 who[NV];
    int n = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      who[i] = __ballot((uint32_t)(key[i] >> 32) == most);
      n += __builtin_popcountll(who[i]);
    }
    if (n > 1) {
      uint32_t lo = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if ((uint32_t)(key[i] >> 32) == most) lo = max(lo, (uint32_t)key[i]);
      lo = wave_umax(lo);
      uint32_t e = 0;  // 65535 - the lowest expert
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (key[i] == ((u64)most << 32 | lo)) e = max(e, 65535u - (uint32_t)(first + P * i));
      e = 65535u - wave_umax(e);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        who[i] = __ballot(key[i] == ((u64)most << 32 | lo) && (uint32_t)(first + P * i) == e);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (who[i]) {
        const int win = __builtin_ctzll(who[i]);
        const int e = __builtin_amdgcn_readlane(first, win) + P * i;
        if (lane == j) id = e;
        if (lane == win) {
          key[i] = 0;
          picked[wave][j] = s[i];
        }
      }
  }
  // lane j: the weight of the j-th chosen
  wave_lds_fence();
  double w = id >= 0 ? picked[wave][lane & (kRouteMaxTopK - 1)] : 0.0;
  if (a.renormalize) {
    if constexpr (!SIGMOID) {
      // the softmax over the chosen ones, which holds also where the others dwarf them
      const float lj = id >= 0 ? clean_logit(load_as_f32<ELEM>(a.logits, t * E + id)) : -INFINITY;
      const float m = wave_max_f32(lj);
      if (id >= 0) w = exp_f64((double)lj - (double)m);
    }
    const double sum = read_f64(sum16_f64(w), 0);  // the first 16 lanes
    w = sum > 0.0 ? w / sum : 0.0;
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
// One wave a token.  Lanes below top_k hold the chosen; an id outside [0, E) takes no
// part.  The sparse forms put a row together in LDS.  The dense form holds expert lane
// + 64 i in slot i; LDS has a byte for each expert, which of the chosen it is, and their
// terms in 64 bits: where one expert has nearly all of the softmax, its g and the sum
// differ by little, and either of them rounded to fp32 first would be most of the
// difference.  (A row of doubles in LDS instead: as fast to 512 experts, 27.3 us for
// 23.3 at 1000.)
// 8192 tokens, 288 experts, fp32: 6.8 us, the launch and then the writes (9.4 MB; the
// sparse forms read the chosen logits only, 5.6 MB of lines); dense, 10.
template <int ELEM, bool SIGMOID, bool DENSE, int NV>
__global__ void __launch_bounds__(kThreads)
k_route_topk_backward(RouteArgs a, const int32_t* __restrict__ ids, const float* __restrict__ dw,
                      void* __restrict__ d_logits) {
  using cell_t = std::conditional_t<DENSE, uint8_t, float>;
  constexpr int PER = 4 / sizeof(cell_t) * 4;  // of 16 bytes
  __shared__ __align__(16) cell_t lds[kThreads / 64][kRouteMaxExperts];
  __shared__ double terms[DENSE ? kThreads / 64 : 1][kRouteMaxTopK + 1];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int64_t t = (int64_t)blockIdx.x * (kThreads / 64) + wave;
  if (t >= a.T) return;
  const int E = a.E;
  cell_t* line = lds[wave];
  for (int e = lane * PER; e < E; e += 64 * PER) *reinterpret_cast<uint4*>(line + e) = make_uint4(0, 0, 0, 0);
  float x[NV];
  if constexpr (DENSE) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      x[i] = lane + 64 * i < E ? load_as_f32<ELEM>(a.logits, t * E + lane + 64 * i) : -INFINITY;
  }
  int id = -1;
  double g = 0.0;
  float l = -INFINITY;
  if (lane < a.top_k) {
    id = ids[t * a.top_k + lane];
    const float w = dw[t * a.top_k + lane];
    if ((unsigned)id >= (unsigned)E) id = -1;
    if (id >= 0) {
      g = (double)w * (double)a.scale;
      l = clean_logit(load_as_f32<ELEM>(a.logits, t * E + id));
    }
  }
  // sums over the chosen: the first 16 lanes hold them
  auto sum_of = [](double v) { return read_f64(sum16_f64(v), 0); };
  double d = 0.0;  // this lane's term
  float top = -INFINITY;
  double inv = 0.0, mean = 0.0, s[NV];
  if constexpr (SIGMOID) {
    const double v = id >= 0 ? sigmoid_f64(l) : 0.0;
    const double rest = id >= 0 ? sigmoid_f64(-l) : 0.0;  // 1 - s
    if (a.renormalize) {
      const double sum = sum_of(v);
      const double p = sum > 0.0 ? v / sum : 0.0;
      d = p * rest * (g - sum_of(p * g));
    } else {
      d = v * rest * g;
    }
  } else if constexpr (!DENSE) {
    const float m = wave_max_f32(l);
    const double x = l > -INFINITY ? exp_f64((double)l - (double)m) : 0.0;
    const double sum = sum_of(x);
    const double p = sum > 0.0 ? x / sum : 0.0;
    d = p * (g - sum_of(p * g));
  } else {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i] = clean_logit(x[i]);
      top = __builtin_fmaxf(top, x[i]);
    }
    top = wave_max_f32(top);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      s[i] = x[i] > -INFINITY ? exp_f64((double)x[i] - (double)top) : 0.0;
      sum += s[i];
    }
    sum = wave_sum_f64(sum);
    inv = sum > 0.0 ? 1.0 / sum : 0.0;
    const double p = l > -INFINITY ? exp_f64((double)l - (double)top) * inv : 0.0;
    d = g;
    mean = sum_of(g * p);
  }
  // an id that occurs more than once gets its terms' sum, in their order
  double mine = 0.0;
  for (int j = 0; j < a.top_k; ++j) {
    const int ij = __builtin_amdgcn_readlane(id, j);
    const double dj = read_f64(d, j);
    if (id == ij) mine += dj;
  }
  wave_lds_fence();
  if constexpr (DENSE) {
    if (id >= 0) line[id] = (uint8_t)(lane + 1);
    if (lane <= kRouteMaxTopK) terms[wave][(lane + 1) % (kRouteMaxTopK + 1)] = lane < a.top_k ? mine : 0.0;
  } else {
    if (id >= 0) line[id] = (float)mine;
  }
  wave_lds_fence();
  if constexpr (DENSE) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 64 * i;
      if (e < E) store_f32<ELEM>(d_logits, t * E + e, (float)(s[i] * inv * (terms[wave][line[e]] - mean)));
    }
  } else if ((E & 3) == 0) {
    for (int e = lane * 4; e < E; e += 256) store4_f32<ELEM>(d_logits, t * E + e, *reinterpret_cast<const float4*>(line + e));
  } else {
    for (int e = lane; e < E; e += 64) store_f32<ELEM>(d_logits, t * E + e, line[e]);
  }
}

template <int ELEM, int NV>
void route(const RouteArgs& a, int lp, int32_t* ids, float* w, hipStream_t stream) {
  const dim3 grid((unsigned)((a.T + kThreads / 64 - 1) / (kThreads / 64)));
  const bool sig = a.scoring == SCORE_SIGMOID, grouped = lp < 6;
  auto go = [&](auto SIG, auto GRP) {
    hipLaunchKernelGGL((k_route_topk<ELEM, NV, SIG(), GRP()>), grid, dim3(kThreads), 0, stream, a, lp, ids, w);
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
  // lanes of a group, 2^lp; groups that are all kept are none
  int lp = 6;
  if (a.topk_group < a.n_group)
    while ((64 >> lp) < a.n_group) --lp;
  const int S = lp < 6 ? a.E / a.n_group : a.E, slots = (S + (1 << lp) - 1) >> lp;
  by_elem(a.elem, [&](auto ELEM) {
    if (slots <= 2) route<ELEM(), 2>(a, lp, ids, weights, stream);
    else if (slots <= 4) route<ELEM(), 4>(a, lp, ids, weights, stream);
    else if (slots <= 5) route<ELEM(), 5>(a, lp, ids, weights, stream);
    else if (slots <= 8) route<ELEM(), 8>(a, lp, ids, weights, stream);
    else if (slots <= 16) route<ELEM(), 16>(a, lp, ids, weights, stream);
    else route<ELEM(), 32>(a, lp, ids, weights, stream);
  });
  return hipGetLastError();
}

hipError_t launch_route_topk_backward(const RouteArgs& a, const int32_t* ids, const float* d_weights,
                                      void* d_logits, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  const dim3 grid((unsigned)((a.T + kThreads / 64 - 1) / (kThreads / 64)));
  by_elem(a.elem, [&](auto ELEM) {
    auto go = [&](auto SIG, auto DENSE, auto NV) {
      hipLaunchKernelGGL((k_route_topk_backward<ELEM(), SIG(), DENSE(), NV()>), grid, dim3(kThreads), 0,
                         stream, a, ids, d_weights, d_logits);
    };
    typedef std::integral_constant<int, 1> none;
    if (a.scoring == SCORE_SIGMOID) go(std::true_type{}, std::false_type{}, none{});
    else if (a.renormalize) go(std::false_type{}, std::false_type{}, none{});
    else if (a.E <= 256) go(std::false_type{}, std::true_type{}, std::integral_constant<int, 4>{});
    else if (a.E <= 512) go(std::false_type{}, std::true_type{}, std::integral_constant<int, 8>{});
    else go(std::false_type{}, std::true_type{}, std::integral_constant<int, 16>{});
  });
  return hipGetLastError();
}
