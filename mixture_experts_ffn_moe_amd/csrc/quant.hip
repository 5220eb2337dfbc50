// quant.hip -- values into e4m3 with a scale for each 128: along rows (what a
// product over the columns takes), along columns with the result transposed
// (what a product over the rows takes: the gradient of weights), both in one
// pass, and weights in 128 x 128 blocks with their transpose (the gradient of a
// layer's input).
//
//   scale = amax / 448 in fp32 (as amax times fp32(1 / 448)), or as e8m0 the
//   smallest power of two at or above amax / 448, so that nothing saturates;
//   q = e4m3(x * (1 / scale)), round to nearest even.
// amax is floored at 1e-30, not at the forward's 1e-10: gradients are
// quantized too, and groups of 1e-12 are ordinary there; at 1e-30 the scale, its
// inverse and the products of two scales' inverses with values stay normal
// numbers.  A group that holds an infinity or a NaN comes out as NaN (scale NaN
// or infinite, e8m0 255).
#include <type_traits>

#include "device.h"
#include "ops.h"

namespace {

constexpr int kThreads = 256;
constexpr float kAmaxFloor = 1e-30f;

// Eight consecutive values as the bits of fp32 or as they are held.
template <int ELEM>
struct Eight {
  uint4 v[ELEM == ELEM_F32 ? 2 : 1];
};

template <int ELEM>
__device__ __forceinline__ Eight<ELEM> load8(const void* p, int64_t i) {
  Eight<ELEM> r;
  if constexpr (ELEM == ELEM_F32) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
    r.v[0] = q[0];
    r.v[1] = q[1];
  } else {
    r.v[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
  }
  return r;
}

template <int ELEM>
__device__ __forceinline__ Eight<ELEM> zero8() {
  Eight<ELEM> r;
  for (auto& x : r.v) x = make_uint4(0, 0, 0, 0);
  return r;
}

template <int ELEM>
__device__ __forceinline__ float value(const Eight<ELEM>& r, int j) {
  if constexpr (ELEM == ELEM_F32) {
    const uint4& q = r.v[j >> 2];
    return __uint_as_float((j & 3) == 0 ? q.x : (j & 3) == 1 ? q.y : (j & 3) == 2 ? q.z : q.w);
  } else {
    const uint4& q = r.v[0];
    const uint32_t d = (j >> 1) == 0 ? q.x : (j >> 1) == 1 ? q.y : (j >> 1) == 2 ? q.z : q.w;
    if constexpr (ELEM == ELEM_BF16) return __uint_as_float((j & 1) ? d & 0xFFFF0000u : d << 16);
    const uint16_t h = (uint16_t)((j & 1) ? d >> 16 : d);
    return (float)__builtin_bit_cast(_Float16, h);
  }
}

// |x| as bits: their unsigned order is the values', infinities and NaN on top,
// so a NaN is kept where a maximum of floats would drop it.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <int CTRL>
__device__ __forceinline__ uint32_t umax_dpp(uint32_t v) {
  return umax(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true));
}
// over the 16 lanes sharing l / 16
__device__ __forceinline__ uint32_t umax16(uint32_t v) {
  v = umax_dpp<0xB1>(v);
  v = umax_dpp<0x4E>(v);
  v = umax_dpp<0x124>(v);
  return umax_dpp<0x128>(v);
}

// A group's inverse scale, and the scale as it is held.
template <int SCALE>
__device__ __forceinline__ float group_scale(uint32_t amax_bits, uint32_t& held) {
  const float amax = __uint_as_float(umax(amax_bits, __float_as_uint(kAmaxFloor)));
  if constexpr (SCALE == SCALE_F32) {
    const float s = amax * (1.0f / 448.0f);
    held = __float_as_uint(s);
    return 1.0f / s;
  } else {
    const uint32_t b = __float_as_uint(amax);
    if (b >= 0x7F800000u) {  // infinity or NaN
      held = 255;
      return __uint_as_float(0x7FC00000u);
    }
    // amax = m 2^k, 448 = 1.75 2^8: 2^(k - 8), twice that where m > 1.75
    const uint32_t e = (b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    held = e;
    return __uint_as_float((254u - e) << 23);
  }
}

template <int SCALE>
__device__ __forceinline__ void store_scale(void* p, int64_t i, uint32_t held) {
  if constexpr (SCALE == SCALE_F32) static_cast<uint32_t*>(p)[i] = held;
  else static_cast<uint8_t*>(p)[i] = (uint8_t)held;
}

// Four values, scaled, as e4m3 bytes.  |x| <= amax, so x / scale is at most 448 and
// a few ulp: nothing to saturate.  A NaN becomes a NaN code.
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

// Rows: 16 lanes a group of 128, eight values each.  A thread has U groups
// requested before it uses the first.  Bound by HBM where it is large (8192 x 4096
// bf16: 20 us, 5.1 TB/s), by the launch where it is small (32 x 4096: 2.5).
constexpr int kGroups = kThreads / 16;  // groups of one pass of a workgroup

template <int ELEM, int SCALE, int U>
__global__ void __launch_bounds__(kThreads)
k_quant_rows(QuantArgs a, uint32_t G, uint32_t total) {
  const int sub = threadIdx.x & 15;
  Eight<ELEM> v[U];
  uint32_t row[U], k[U];
  const uint32_t M = (uint32_t)(a.ntp ? min((int64_t)max(*a.ntp, 0), a.M) : a.M), K = (uint32_t)a.K;
  const uint32_t first = blockIdx.x * (kGroups * U) + (threadIdx.x >> 4);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = first + u * kGroups;
    row[u] = i < total ? i / G : M;
    k[u] = (i - row[u] * G) * 128 + sub * 8;
    v[u] = row[u] < M && k[u] < K ? load8<ELEM>(a.x, (int64_t)row[u] * K + k[u]) : zero8<ELEM>();
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = umax(m, abs_bits(value<ELEM>(v[u], j)));
    m = umax16(m);
    uint32_t held;
    const float inv = group_scale<SCALE>(m, held);
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = value<ELEM>(v[u], j) * inv;
    if (row[u] < M) {
      if (k[u] < K)
        *reinterpret_cast<uint2*>(a.q + (int64_t)row[u] * K + k[u]) =
            make_uint2(pack4(f[0], f[1], f[2], f[3]), pack4(f[4], f[5], f[6], f[7]));
      if (sub == 0) store_scale<SCALE>(a.qs, first + u * kGroups, held);
    }
  }
}

// Tiles of 128 rows x 128 columns: thread (r, c) = (tid / 16, tid % 16) holds rows
// [8r, 8r + 8) of columns [8c, 8c + 8).  The columns' bytes are turned in LDS, so
// that whole 128-byte lines of a column are written.
// BLOCK: one scale for the tile (weights; blockIdx.z the expert), q and, with COLS,
// its transpose.  Else ROWS and COLS with scales of their own.
// x is read once for both forms.  Bound by HBM: weights 8 x 4096 x 4096 fp32 in 149
// us, 5.4 TB/s (a plain conversion of these bytes, two read for one written: 137); rows and columns of 8192 x 4096 bf16 in 31, 4.3 TB/s, where the
// conversions of both forms take turns with the loads.
//
// In LDS a column is 128 bytes and every access 8 or 16.  A wave writes 8 bytes of 16
// columns 8 apart; so that these fall on all banks, chunk q of column 8 c + j lies at
// chunk q ^ (c % 8) of column 8 c + (j ^ (c / 8)).
__device__ __forceinline__ int turned(int c, int j, int byte) {
  return ((8 * c + (j ^ (c >> 3))) << 7) + (byte ^ ((c & 7) << 4));
}

// Largest over the wave's lanes l % 16: both halves, both rows of each half.
__device__ __forceinline__ uint32_t umax_rows(uint32_t v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  v = umax(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return umax(b[0], b[1]);
}

template <int ELEM, int SCALE, bool ROWS, bool COLS, bool BLOCK>
__global__ void __launch_bounds__(kThreads)
k_quant_tile(QuantArgs a, int64_t Mp, int64_t KB) {
  __shared__ __align__(16) uint8_t turn[COLS ? 128 * 128 : 16];
  __shared__ __align__(16) uint32_t part[4][BLOCK ? 4 : 128];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int64_t m0 = (int64_t)blockIdx.y * 128, k0 = (int64_t)blockIdx.x * 128;
  const int64_t M = a.ntp ? min((int64_t)max(*a.ntp, 0), a.M) : a.M;
  if (m0 >= M) return;  // columns: groups behind the rows in use are left alone
  const int64_t z = blockIdx.z;  // expert
  const int64_t xbase = z * a.M * a.K, k = k0 + 8 * c;
  Eight<ELEM> v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t m = m0 + 8 * r + i;
    v[i] = m < M && k < a.K ? load8<ELEM>(a.x, xbase + m * a.K + k) : zero8<ELEM>();
  }
  float inv_block = 0.f;
  uint32_t held;
  if constexpr (BLOCK) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = umax(m, abs_bits(value<ELEM>(v[i], j)));
    m = umax_rows(umax16(m));
    if ((threadIdx.x & 63) == 0) part[0][threadIdx.x >> 6] = m;
    __syncthreads();
    m = umax(umax(part[0][0], part[0][1]), umax(part[0][2], part[0][3]));
    inv_block = group_scale<SCALE>(m, held);
    if (threadIdx.x == 0) {
      const int64_t NB = (a.M + 127) / 128;
      store_scale<SCALE>(a.qs, (z * NB + blockIdx.y) * KB + blockIdx.x, held);
      if constexpr (COLS) store_scale<SCALE>(a.qts, (z * KB + blockIdx.x) * NB + blockIdx.y, held);
    }
  }
  if constexpr (ROWS) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t m = m0 + 8 * r + i;
      float inv = inv_block;
      if constexpr (!BLOCK) {
        uint32_t x = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) x = umax(x, abs_bits(value<ELEM>(v[i], j)));
        inv = group_scale<SCALE>(umax16(x), held);
        if (c == 0 && m < M) store_scale<SCALE>(a.qs, m * KB + blockIdx.x, held);
      }
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = value<ELEM>(v[i], j) * inv;
      if (m < M && k < a.K)
        *reinterpret_cast<uint2*>(a.q + xbase + m * a.K + k) =
            make_uint2(pack4(f[0], f[1], f[2], f[3]), pack4(f[4], f[5], f[6], f[7]));
    }
  }
  if constexpr (COLS) {
    float inv[8];
    if constexpr (BLOCK) {
#pragma unroll
      for (int j = 0; j < 8; ++j) inv[j] = inv_block;
    } else {
      uint32_t x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j] = umax(x[j], abs_bits(value<ELEM>(v[i], j)));
        x[j] = umax_rows(x[j]);
      }
      if ((threadIdx.x & 63) < 16) {
        uint4* to = reinterpret_cast<uint4*>(&part[threadIdx.x >> 6][8 * c]);
        to[0] = make_uint4(x[0], x[1], x[2], x[3]);
        to[1] = make_uint4(x[4], x[5], x[6], x[7]);
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4* from = reinterpret_cast<const uint4*>(&part[i][8 * c]);
        const uint4 p = from[0], q = from[1];
        x[0] = umax(x[0], p.x), x[1] = umax(x[1], p.y), x[2] = umax(x[2], p.z), x[3] = umax(x[3], p.w);
        x[4] = umax(x[4], q.x), x[5] = umax(x[5], q.y), x[6] = umax(x[6], q.z), x[7] = umax(x[7], q.w);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        inv[j] = group_scale<SCALE>(x[j], held);
        if (r == 0 && k + j < a.K) store_scale<SCALE>(a.qts, (k + j) * (Mp / 128) + blockIdx.y, held);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = value<ELEM>(v[i], j) * inv[j];
      *reinterpret_cast<uint2*>(turn + turned(c, j, 8 * r)) =
          make_uint2(pack4(f[0], f[1], f[2], f[3]), pack4(f[4], f[5], f[6], f[7]));
    }
    __syncthreads();
    // 8 threads a column of 128 bytes; weights' rows end at M, tokens' columns are padded
    const int64_t end = BLOCK ? a.M : Mp;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int col = (threadIdx.x >> 3) + 32 * u, at = (threadIdx.x & 7) * 16;
      if (k0 + col < a.K && m0 + at < end)
        *reinterpret_cast<uint4*>(a.qt + z * a.M * a.K * (BLOCK ? 1 : 0) + (k0 + col) * end + m0 + at) =
            *reinterpret_cast<const uint4*>(turn + turned(col >> 3, col & 7, at));
    }
  }
}

template <class F>
void by_types(int elem, int scale_type, F f) {
  auto with = [&](auto SCALE) {
    if (elem == ELEM_F32) f(std::integral_constant<int, ELEM_F32>{}, SCALE);
    else if (elem == ELEM_F16) f(std::integral_constant<int, ELEM_F16>{}, SCALE);
    else f(std::integral_constant<int, ELEM_BF16>{}, SCALE);
  };
  if (scale_type == SCALE_F32) with(std::integral_constant<int, SCALE_F32>{});
  else with(std::integral_constant<int, SCALE_E8M0>{});
}

}  // namespace

hipError_t launch_quant(const QuantArgs& a, hipStream_t stream) {
  if (a.M == 0) return hipSuccess;
  const int64_t G = (a.K + 127) / 128, Mp = (a.M + 127) / 128 * 128;
  by_types(a.elem, a.scale_type, [&](auto ELEM, auto SCALE) {
    if (!a.qt) {
      // one group for 16 lanes where the call is small, four where there are many
      // workgroups: more requests in flight (bf16, one / four groups, us: 1024 x 4096
      // 3.7 / 3.9, 2048 x 7168 8.8 / 8.6, 8192 x 4096 20.9 / 20.1)
      const int64_t total = a.M * G;
      auto go = [&](auto U) {
        constexpr int64_t per = kGroups * U();
        hipLaunchKernelGGL((k_quant_rows<ELEM(), SCALE(), U()>), dim3((unsigned)((total + per - 1) / per)),
                           dim3(kThreads), 0, stream, a, (uint32_t)G, (uint32_t)total);
      };
      if (total <= 2048 * kGroups) go(std::integral_constant<int, 1>{});
      else go(std::integral_constant<int, 4>{});
      return;
    }
    const dim3 grid((unsigned)G, (unsigned)(Mp / 128));
    if (a.q)
      hipLaunchKernelGGL((k_quant_tile<ELEM(), SCALE(), true, true, false>), grid, dim3(kThreads), 0,
                         stream, a, Mp, G);
    else
      hipLaunchKernelGGL((k_quant_tile<ELEM(), SCALE(), false, true, false>), grid, dim3(kThreads), 0,
                         stream, a, Mp, G);
  });
  return hipGetLastError();
}

hipError_t launch_quant_weights(const void* w, int64_t E, int64_t N, int64_t K, int elem,
                                int scale_type, uint8_t* q, void* qs, uint8_t* qt, void* qts,
                                hipStream_t stream) {
  if (E == 0) return hipSuccess;
  QuantArgs a{w, nullptr, q, qs, qt, qts, N, K, elem, scale_type};
  const int64_t KB = (K + 127) / 128;
  const dim3 grid((unsigned)KB, (unsigned)((N + 127) / 128), (unsigned)E);
  by_types(elem, scale_type, [&](auto ELEM, auto SCALE) {
    if (qt)
      hipLaunchKernelGGL((k_quant_tile<ELEM(), SCALE(), true, true, true>), grid, dim3(kThreads), 0,
                         stream, a, N, KB);
    else
      hipLaunchKernelGGL((k_quant_tile<ELEM(), SCALE(), true, false, true>), grid, dim3(kThreads), 0,
                         stream, a, N, KB);
  });
  return hipGetLastError();
}
