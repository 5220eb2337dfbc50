// w4.hip -- products of a few tokens with 4-bit weights: y[r] = W[e] x for
// every route r of expert e, optionally with SwiGLU over the two halves of
// the outputs.
//
// Weights of one row n lie along the contraction, two a byte, with a scale for
// each group of it:  W = (q - z) s (whole q, z in 0..15; z = 8 when no zero
// points are given), or e2m1(q) 2^(c - 127) for each 32 (microscaling).  A few
// tokens leave the weights' bytes as the bound, so the weights are read once
// per expert, straight from their plain row-major layout into registers, and
// turned into bf16 there with about one instruction per weight:
//   int4: (v & 0x000F000F) | 0x43004300 holds 128 + q of two nibbles, exactly.
//         The group's sum of (128 + q) x minus (128 + z) times the group's sum
//         of x, times s, is the group's part; both sums are fp32, the second
//         one from the same matrix instruction with ones for weights.  The
//         offset costs about five of fp32's 24 bits, against the 8 or 11 of
//         the output.
//   e2m1: the hardware's conversion, scale included; e2m1 times a power of
//         two is a bf16, so this is exact too.
// Activations are bf16 operands: bf16 ones as they are, fp16 and fp32 ones as
// two bf16 parts hi + lo (exact for fp16, 2^-17 for fp32).
//
// A 16x16x32 matrix instruction takes 16 tokens (A rows) and 16 weight rows (B
// columns); a lane (n = l % 16, g = l / 16) reads 16 bytes of row n in each
// 128-wide step of K: elements 32 g .. 32 g + 31.  Where a scale covers the
// whole step, dword d of the four lane groups feeds instruction d as it is
// (the contraction's order is free as long as the tokens use the same).  Groups
// of 32 and 64 need the elements of one instruction to lie in one group: the
// four dwords of the four lane groups are transposed by lane-row swaps.
//
// A workgroup has 8 waves on the same 16 or 32 weight rows; wave w takes the
// steps w, w + 8, ... of K, and the waves' sums are added through LDS at the
// end.  The tokens' part of K lies in LDS, in the order the weights need.
#include "device.h"
#include "ops.h"

namespace {

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;
constexpr int kTile = 16;               // tokens of one pass over the weights
constexpr int kUnit = kWaves * 128;     // K elements of one step of every wave
constexpr int kPad = 8;                 // elements behind each token's row in LDS
constexpr int kDepth = 4;               // steps a wave requests ahead

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <int XE>
constexpr int parts() { return XE == ELEM_BF16 ? 1 : 2; }

__device__ __forceinline__ float bits_to_f32(uint32_t u16, int elem) {
  return elem == ELEM_F16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)u16)
                          : __uint_as_float(u16 << 16);
}

__device__ __forceinline__ int buf_loadu16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
  return (int)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)voff, (int)soff, 0);
}

// 8 int4 codes of one dword as bf16 128 + q, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ bf16x8 int4_to_bf16(uint32_t v) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = ((v >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
  return __builtin_bit_cast(bf16x8, o);
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// 8 e2m1 codes of one dword times a power of two, in order.
__device__ __forceinline__ bf16x8 e2m1_to_bf16(uint32_t v, float scale) {
  bf16x2 p[4];
  p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 0);
  p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 1);
  p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 2);
  p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 3);
  bf16x8 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[2 * i] = p[i][0], o[2 * i + 1] = p[i][1];
  return o;
}

// Dword d of lane group g <-> dword g of lane group d: halves, then quarters.
__device__ __forceinline__ void transpose4(uint4& c) {
  u32x2 a = __builtin_amdgcn_permlane32_swap(c.x, c.z, false, false);
  u32x2 b = __builtin_amdgcn_permlane32_swap(c.y, c.w, false, false);
  u32x2 e = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  u32x2 f = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  c = make_uint4(e[0], e[1], f[0], f[1]);
}

// bf16 bits of 8 consecutive activations: part 0 the nearest bf16, part 1 what is left.
template <int XE>
__device__ __forceinline__ void split8(const uint8_t* p, uint32_t (&b)[parts<XE>()][8]) {
  if constexpr (XE == ELEM_BF16) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) b[0][2 * i] = d[i] & 0xFFFFu, b[0][2 * i + 1] = d[i] >> 16;
  } else {
    float f[8];
    if constexpr (XE == ELEM_F16) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = bits_to_f32(d[i] & 0xFFFFu, ELEM_F16);
        f[2 * i + 1] = bits_to_f32(d[i] >> 16, ELEM_F16);
      }
    } else {
      const float4 v = *reinterpret_cast<const float4*>(p);
      const float4 u = *reinterpret_cast<const float4*>(p + 16);
      f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
      f[4] = u.x, f[5] = u.y, f[6] = u.z, f[7] = u.w;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      b[0][i] = f32_to_bf16(f[i]);
      b[1][i] = f32_to_bf16(f[i] - __uint_as_float(b[0][i] << 16));
    }
  }
}

__device__ __forceinline__ void store_out(void* out, size_t at, float v, int elem) {
  if (elem == ELEM_F32) static_cast<float*>(out)[at] = v;
  else if (elem == ELEM_F16) static_cast<_Float16*>(out)[at] = (_Float16)v;
  else static_cast<uint16_t*>(out)[at] = f32_to_bf16(v);
}

// GM: scale groups in a 128-wide step (int4: 1, 2, 4).  NT: 16-row weight
// tiles of a workgroup; with SWIGLU the gate's and the up's.
// Grid: x the output tile; y the route whose expert to take (R <= E; only the
// expert's first route works), the expert (R > E; y = E: the routes without an
// expert here), or the block of `tile` tokens (no ids).
template <int FMT, int XE, int GM, int NT, bool SWIGLU>
__global__ void __launch_bounds__(kThreads)
k_w4(W4Args a, int tile, int x_bytes) {
  constexpr int P = parts<XE>();
  extern __shared__ __align__(16) uint8_t smem[];
  uint16_t* xs = reinterpret_cast<uint16_t*>(smem);
  float* red = reinterpret_cast<float*>(smem);  // after the tokens' last use
  uint16_t* list = reinterpret_cast<uint16_t*>(smem + x_bytes);
  __shared__ int wave_count[kWaves];

  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  const int n16 = lane & 15, g = lane >> 4;
  const int out_n = SWIGLU ? a.N / 2 : a.N;
  constexpr int kCols = SWIGLU ? 16 : 16 * NT;
  const int col0 = blockIdx.x * kCols;

  // the workgroup's expert and the routes it works on
  int e = 0, count, first = 0;
  if (!a.ids) {
    first = blockIdx.y * tile;
    count = min(tile, a.R - first);
  } else {
    const int y = blockIdx.y;
    e = a.R <= a.E ? a.ids[y] : y < a.E ? y : -1;
    if ((unsigned)e >= (unsigned)a.E) e = -1;
    count = 0;
    for (int base = 0; base < a.R; base += kThreads) {
      const int r = base + tid;
      int id = -2;
      if (r < a.R) {
        id = a.ids[r];
        if ((unsigned)id >= (unsigned)a.E) id = -1;
      }
      const unsigned long long m = __ballot(id == e);
      if (lane == 0) wave_count[wave] = __popcll(m);
      __syncthreads();
      int at = count;
      for (int v = 0; v < kWaves; ++v) {
        if (v < wave) at += wave_count[v];
        count += wave_count[v];
      }
      if (id == e) list[at + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)r;
      __syncthreads();
    }
    if (count == 0 || (a.R <= a.E && list[0] != y)) return;
    if (e < 0) {  // routes without an expert here: zeros
      for (int i = tid; i < count * kCols; i += kThreads) {
        const int c = col0 + i % kCols;
        if (c < out_n) store_out(a.out, (size_t)list[i / kCols] * out_n + c, 0.f, a.oelem);
      }
      return;
    }
  }

  const int KS = (a.K + 127) / 128, KG = a.K / a.group;
  const uint32_t pitch = (uint32_t)a.K / 2;
  const __amdgpu_buffer_rsrc_t rw =
      make_rsrc(a.w + (size_t)e * a.N * pitch, (uint32_t)a.N * pitch);
  constexpr int SB = FMT == W4_MX ? 1 : 2;  // bytes of a scale
  const __amdgpu_buffer_rsrc_t rs =
      make_rsrc(static_cast<const uint8_t*>(a.scale) + (size_t)e * a.N * KG * SB,
                (uint32_t)a.N * KG * SB);
  const bool has_zero = FMT == W4_INT && a.zero;
  const __amdgpu_buffer_rsrc_t rz =
      make_rsrc(has_zero ? a.zero + (size_t)e * a.N * KG : a.w, (uint32_t)a.N * KG);
  uint32_t wrow[NT], srow[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    int n = SWIGLU ? t * out_n + min(col0 + n16, out_n - 1) : min(col0 + 16 * t + n16, a.N - 1);
    wrow[t] = (uint32_t)n * pitch + 16 * g;
    srow[t] = (uint32_t)n * KG;
  }
  constexpr uint32_t kNone = 0xFFFFFFF0u;  // past every buffer: the load returns 0

  for (int m0 = 0; m0 < count; m0 += tile) {
    const int nt = min(tile, count - m0);
    // as much of K at a time as the LDS holds for these tokens
    int kc = (x_bytes / (P * nt * 2) - kPad) / kUnit * kUnit;
    kc = min(kc, (a.K + kUnit - 1) / kUnit * kUnit);
    const int xrow = kc + kPad;
    const uint16_t* xa = xs + (size_t)(n16 < nt ? n16 : 0) * xrow;
    f32x4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};

    for (int k0 = 0; k0 < a.K; k0 += kc) {
      const int S = kc / kUnit;  // steps of each wave in this part of K
      uint4 wq[kDepth][NT];
      uint32_t sq[kDepth][NT][GM], zq[kDepth][NT][GM];
      auto request = [&](int slot, int i) {
        const int step = (k0 / 128) + i * kWaves + wave;
        if (step >= KS) return;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          // the whole offset in the checked one: behind the last row's end it reads 0
          wq[slot][t] = buf_load16(rw, wrow[t] + (uint32_t)step * 64, 0);
          if constexpr (FMT == W4_MX) {
            const int c = step * 4 + g;
            sq[slot][t][0] = (uint32_t)buf_loadu8(rs, c < KG ? srow[t] + c : kNone, 0);
          } else {
#pragma unroll
            for (int q = 0; q < GM; ++q) {
              const int c = GM > 1 ? step * GM + q : a.group == 128 ? step : 0;
              sq[slot][t][q] = (uint32_t)buf_loadu16(rs, c < KG ? (srow[t] + c) * 2 : kNone, 0);
              zq[slot][t][q] =
                  has_zero ? (uint32_t)buf_loadu8(rz, c < KG ? srow[t] + c : kNone, 0) : 8u;
            }
          }
        }
      };
#pragma unroll
      for (int u = 0; u < kDepth; ++u)
        if (u < S) request(u, u);

      if (m0 || k0) __syncthreads();  // the earlier part is read
      const int per = kc / 8;
      for (int u = tid; u < nt * per; u += kThreads) {
        const int m = u / per, k = k0 + (u - m * per) * 8;
        uint32_t b[P][8];
        if (k < a.K) {
          const int r = a.ids ? list[m0 + m] : first + m0 + m;
          const int row = a.x_per_route ? r : r / a.top_k;
          split8<XE>(static_cast<const uint8_t*>(a.x) +
                         ((size_t)row * a.K + k) * elem_bytes(XE), b);
        } else {
#pragma unroll
          for (int p = 0; p < P; ++p)
#pragma unroll
            for (int i = 0; i < 8; ++i) b[p][i] = 0;
        }
#pragma unroll
        for (int p = 0; p < P; ++p) {
          uint4 v;
          if constexpr (FMT == W4_MX)
            v = make_uint4(b[p][0] | b[p][1] << 16, b[p][2] | b[p][3] << 16,
                           b[p][4] | b[p][5] << 16, b[p][6] | b[p][7] << 16);
          else
            v = make_uint4(b[p][0] | b[p][4] << 16, b[p][1] | b[p][5] << 16,
                           b[p][2] | b[p][6] << 16, b[p][3] | b[p][7] << 16);
          *reinterpret_cast<uint4*>(xs + (size_t)(p * nt + m) * xrow + (k - k0)) = v;
        }
      }
      __syncthreads();

      for (int i0 = 0; i0 < S; i0 += kDepth) {
#pragma unroll
        for (int u = 0; u < kDepth; ++u) {
          const int i = i0 + u;
          if (i >= S || (k0 / 128) + i * kWaves + wave >= KS) continue;
          const uint16_t* xp = xa + (i * kWaves + wave) * 128;
          bf16x8 xf[P][4];
#pragma unroll
          for (int p = 0; p < P; ++p)
#pragma unroll
            for (int d = 0; d < 4; ++d)
              xf[p][d] = *reinterpret_cast<const bf16x8*>(
                  xp + (size_t)p * nt * xrow + (GM == 1 ? 32 * g + 8 * d : 32 * d + 8 * g));
          if constexpr (FMT == W4_MX) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const uint32_t c = sq[u][t][0];
              // 2^(c - 127) as a float: c in the exponent field, 0 subnormal, 255 NaN
              const float s = __uint_as_float(c == 255 ? 0x7FC00000u : c ? c << 23 : 0x00400000u);
              const uint32_t q[4] = {wq[u][t].x, wq[u][t].y, wq[u][t].z, wq[u][t].w};
#pragma unroll
              for (int d = 0; d < 4; ++d) {
                const bf16x8 b = e2m1_to_bf16(q[d], s);
#pragma unroll
                for (int p = 0; p < P; ++p)
                  acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[p][d], b, acc[t], 0, 0, 0);
              }
            }
          } else {
            const bf16x8 ones = __builtin_bit_cast(bf16x8, make_uint4(0x3F803F80u, 0x3F803F80u,
                                                                     0x3F803F80u, 0x3F803F80u));
            constexpr int DG = 4 / GM;  // instructions of one group
            f32x4 sx[GM];
#pragma unroll
            for (int q = 0; q < GM; ++q) {
              sx[q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int d = q * DG; d < (q + 1) * DG; ++d)
#pragma unroll
                for (int p = 0; p < P; ++p)
                  sx[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[p][d], ones, sx[q], 0, 0, 0);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              if constexpr (GM > 1) transpose4(wq[u][t]);
              const uint32_t q4[4] = {wq[u][t].x, wq[u][t].y, wq[u][t].z, wq[u][t].w};
#pragma unroll
              for (int q = 0; q < GM; ++q) {
                f32x4 v = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int d = q * DG; d < (q + 1) * DG; ++d) {
                  const bf16x8 b = int4_to_bf16(q4[d]);
#pragma unroll
                  for (int p = 0; p < P; ++p)
                    v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[p][d], b, v, 0, 0, 0);
                }
                const float s = bits_to_f32(sq[u][t][q], a.scale_elem);
                const float z = 128.f + (float)zq[u][t][q];
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[t][j] += s * (v[j] - z * sx[q][j]);
              }
            }
          }
          if (i + kDepth < S) request(u, i + kDepth);
        }
      }
    }

    // the waves' sums, then one thread per output
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t)
      *reinterpret_cast<f32x4*>(red + ((wave * NT + t) * 64 + lane) * 4) = acc[t];
    __syncthreads();
    auto total = [&](int t, int m, int c) {
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < kWaves; ++v)
        s += red[((v * NT + t) * 64 + c + 16 * (m >> 2)) * 4 + (m & 3)];
      return s;
    };
    for (int o = tid; o < nt * kCols; o += kThreads) {
      const int m = o / kCols, c = o % kCols;
      if (col0 + c >= out_n) continue;
      const int r = a.ids ? list[m0 + m] : first + m0 + m;
      const float v = SWIGLU ? swiglu(total(0, m, c), total(NT - 1, m, c)) : total(c / 16, m, c % 16);
      store_out(a.out, (size_t)r * out_n + col0 + c, v, a.oelem);
    }
  }
}

constexpr int kCombineThreads = 256;

__global__ void __launch_bounds__(kCombineThreads)
k_w4_combine(const float* __restrict__ y, const int32_t* __restrict__ ids,
             const float* __restrict__ w, void* __restrict__ out, int oelem, int top_k, int K,
             int E) {
  const int t = blockIdx.y, c = (blockIdx.x * kCombineThreads + threadIdx.x) * 4;
  if (c >= K) return;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int j = 0; j < top_k; ++j) {
    const int r = t * top_k + j;
    if ((unsigned)ids[r] >= (unsigned)E) continue;
    const float wr = w[r];
    const float4 v = *reinterpret_cast<const float4*>(y + (size_t)r * K + c);
    s.x += wr * v.x, s.y += wr * v.y, s.z += wr * v.z, s.w += wr * v.w;
  }
  const size_t at = (size_t)t * K + c;
  store_out(out, at, s.x, oelem);
  store_out(out, at + 1, s.y, oelem);
  store_out(out, at + 2, s.z, oelem);
  store_out(out, at + 3, s.w, oelem);
}

// LDS of the tokens: a few tokens' whole K, or 1,024 elements of kTile tokens
// (half as many of two parts).
constexpr int kTokenLds = 33 * 1024;
static_assert(kTile * (kUnit + kPad) * 2 <= kTokenLds, "one step of a full tile fits");
static_assert(kWaves * 2 * 64 * 16 <= kTokenLds, "the waves' sums fit");

template <int FMT, int XE, int GM, int NT, bool SWIGLU>
hipError_t launch_one(const W4Args& a, hipStream_t stream) {
  // tokens of one pass: 16, or 8 of two parts so that the LDS stays small
  const int most = parts<XE>() == 1 ? kTile : kTile / 2;
  const int tokens = a.R / a.top_k;
  const int tile = tokens < most ? tokens : most;
  const int out_n = SWIGLU ? a.N / 2 : a.N, cols = SWIGLU ? 16 : 16 * NT;
  const int lists = a.ids ? (a.R * 2 + 15) / 16 * 16 : 0;
  const int y = !a.ids ? (a.R + tile - 1) / tile : a.R <= a.E ? a.R : a.E + 1;
  hipLaunchKernelGGL((k_w4<FMT, XE, GM, NT, SWIGLU>), dim3((out_n + cols - 1) / cols, y),
                     dim3(kThreads), kTokenLds + lists, stream, a, tile, kTokenLds);
  return hipGetLastError();
}

template <int FMT, int XE, int GM>
hipError_t launch_shape(const W4Args& a, hipStream_t stream) {
  if constexpr (XE != ELEM_F32)
    if (a.swiglu) return launch_one<FMT, XE, GM, 2, true>(a, stream);
  return launch_one<FMT, XE, GM, 1, false>(a, stream);
}

template <int XE>
hipError_t launch_format(int format, const W4Args& a, hipStream_t stream) {
  if (format == W4_MX) return launch_shape<W4_MX, XE, 1>(a, stream);
  if (a.group == 32) return launch_shape<W4_INT, XE, 4>(a, stream);
  if (a.group == 64) return launch_shape<W4_INT, XE, 2>(a, stream);
  return launch_shape<W4_INT, XE, 1>(a, stream);
}

}  // namespace

hipError_t launch_w4(int format, const W4Args& a, hipStream_t stream) {
  if (a.R == 0) return hipSuccess;
  if (a.xelem == ELEM_F32) return launch_format<ELEM_F32>(format, a, stream);
  if (a.xelem == ELEM_F16) return launch_format<ELEM_F16>(format, a, stream);
  return launch_format<ELEM_BF16>(format, a, stream);
}

hipError_t launch_w4_combine(const float* y, const int32_t* ids, const float* w, void* out,
                             int oelem, int T, int top_k, int K, int E, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  hipLaunchKernelGGL(k_w4_combine, dim3((K / 4 + kCombineThreads - 1) / kCombineThreads, T),
                     dim3(kCombineThreads), 0, stream, y, ids, w, out, oelem, top_k, K, E);
  return hipGetLastError();
}
