// fp8_linear.hip -- products of e4m3 values with a scale for each 128 of the
// contraction: linear layers (dense, or block by block of a plan with each
// block's expert) and the gradient of their weights.
//
//   out[m, n] = sum_g sx[m, g] sw[n, g] sum_{k in group g} X[m, k] W[n, k]
//
// W is the matrix instruction's A operand and X its B operand, so that a lane
// ends with one row m and four consecutive n.  With fp32 scales a group's sum
// leaves the instruction and is added in fp32 with its scale; e8m0 scales go into
// the instruction, which then adds up all groups by itself.
#include <type_traits>

#include "device.h"
#include "ops.h"

namespace {

__device__ __forceinline__ uint32_t f32_to_f16(float v) {
  return __builtin_bit_cast(uint16_t, (_Float16)v);
}

template <int OELEM>
__device__ __forceinline__ uint32_t to_elem(float v) {
  if constexpr (OELEM == ELEM_F16) return f32_to_f16(v);
  else return f32_to_bf16(v);
}

template <int SCALE>
__device__ __forceinline__ float scale_at(const void* p, int64_t i) {
  if constexpr (SCALE == SCALE_F32) return static_cast<const float*>(p)[i];
  return 0.f;
}

// What a workgroup works on: rows [m0, m1) of X and of the output (below it
// the output's row offset), weights of one expert, and the steps of k.
struct Part {
  int64_t m0;      // first row
  int rows;        // rows from m0 on that exist
  int64_t k0;      // first column of both operands (a multiple of 128)
  int64_t k1;      // one past the last
  int e;           // expert, or -1: the rows are zeros
  bool none;       // nothing to do
};

// Blocks of expert e (a plan's blocks lie in the experts' order).  Every thread of
// the workgroup calls this.
__device__ __forceinline__ void blocks_of(const Fp8Args& a, int e, int& first, int& count) {
  __shared__ int lo, n;
  if (threadIdx.x == 0) {
    lo = 0x7FFFFFFF;
    n = 0;
  }
  __syncthreads();
  const int nb = min(max(*a.ntp, 0) / a.block_m, a.n_blocks);
  int mine = 0, least = 0x7FFFFFFF;
  for (int b = threadIdx.x; b < nb; b += blockDim.x)
    if (a.experts[b] == e) {
      ++mine;
      least = min(least, b);
    }
  if (mine) {
    atomicAdd(&n, mine);
    atomicMin(&lo, least);
  }
  __syncthreads();
  first = __builtin_amdgcn_readfirstlane(lo);
  count = __builtin_amdgcn_readfirstlane(n);
}

// The part of tile `mt` of BM rows (layer), or of expert z (gradient).
template <bool DW>
__device__ __forceinline__ Part part_of(const Fp8Args& a, int64_t mt, int BM, int z) {
  Part p;
  p.m0 = mt * BM;
  p.k0 = 0;
  p.k1 = a.K;
  p.e = 0;
  p.none = false;
  int64_t end = a.M;
  if constexpr (DW) {
    p.e = z;
    if (a.experts) {
      int first, count;
      blocks_of(a, z, first, count);
      p.k0 = count ? (int64_t)first * a.block_m : 0;
      p.k1 = min(p.k0 + (int64_t)count * a.block_m, a.K);
    }
  } else if (a.experts) {
    const int64_t ntp = min((int64_t)max(*a.ntp, 0), a.M);
    const int64_t b = p.m0 / a.block_m;
    end = min((b + 1) * a.block_m, ntp);  // a tile lies in one block
    if (p.m0 >= ntp) {
      p.none = true;
      return p;
    }
    p.e = a.experts[b];
    if ((unsigned)p.e >= (unsigned)a.E) p.e = -1;
  }
  p.rows = (int)min(end - p.m0, (int64_t)BM);
  p.none = p.rows <= 0;
  return p;
}

// Four values of row m at columns n .. n + 3.
template <int OELEM>
__device__ __forceinline__ void store4(void* out, int64_t row, int64_t n, int64_t N, const f32x4& v) {
  uint16_t* o = static_cast<uint16_t*>(out) + row * N + n;
  if ((N & 3) == 0 && n + 4 <= N) {
    *reinterpret_cast<uint2*>(o) = make_uint2(to_elem<OELEM>(v[0]) | to_elem<OELEM>(v[1]) << 16,
                                              to_elem<OELEM>(v[2]) | to_elem<OELEM>(v[3]) << 16);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) o[i] = (uint16_t)to_elem<OELEM>(v[i]);
  }
}

// A workgroup of kW waves: 16 rows of W, 16 * NT rows of X; the waves take the
// steps of k in turn and add their sums in LDS, in a fixed order.
constexpr int kW = 8;

template <int OELEM, int SCALE, int NT, bool DW>
__global__ void __launch_bounds__(kW * 64)
k_fp8_rows(Fp8Args a) {
  __shared__ f32x4 sums[kW][NT][64];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int g = lane >> 4, r16 = lane & 15;
  const int64_t n0 = (int64_t)blockIdx.y * 16;
  const Part p = part_of<DW>(a, blockIdx.x, 16 * NT, blockIdx.z);
  if (p.none) return;
  f32x4 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int wrows = (int)min((int64_t)16, a.N - n0);
  const int64_t GK = (a.K + 127) / 128;  // groups of a row
  if (p.e >= 0) {
    const int64_t we = DW ? 0 : p.e;
    const uint8_t* wp = a.w + (we * a.N + n0) * a.K + p.k0;
    const uint8_t* xp = a.x + p.m0 * a.K + p.k0;
    const int steps = (int)((p.k1 - p.k0 + 127) / 128);
    for (int ks = wave; ks < steps; ks += kW) {
      const int64_t k = (int64_t)ks * 128 + 32 * g;
      const int64_t left = p.k1 - p.k0 - k;  // 16-byte chunks: K is a multiple of 16
      const uint4 zero = make_uint4(0, 0, 0, 0);
      Frag<KIND_FP8B> fw;
      const bool wr = r16 < wrows;
      const uint8_t* wl = wp + (int64_t)r16 * a.K + k;
      fw.c[0] = wr && left > 0 ? *reinterpret_cast<const uint4*>(wl) : zero;
      fw.c[1] = wr && left > 16 ? *reinterpret_cast<const uint4*>(wl + 16) : zero;
      const int64_t gk = p.k0 / 128 + ks;
      float sw[4];
      int ew = 127;
      if constexpr (DW) {
        if constexpr (SCALE == SCALE_F32) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            sw[i] = 4 * g + i < wrows ? scale_at<SCALE>(a.ws, (n0 + 4 * g + i) * GK + gk) : 0.f;
        } else {
          ew = wr ? static_cast<const uint8_t*>(a.ws)[(n0 + r16) * GK + gk] : 127;
        }
      } else {
        const int64_t at = (we * ((a.N + 127) / 128) + n0 / 128) * GK + gk;
        if constexpr (SCALE == SCALE_F32) sw[0] = sw[1] = sw[2] = sw[3] = scale_at<SCALE>(a.ws, at);
        else ew = static_cast<const uint8_t*>(a.ws)[at];
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int m = 16 * t + r16;
        const bool xr = m < p.rows;
        const uint8_t* xl = xp + (int64_t)m * a.K + k;
        Frag<KIND_FP8B> fx;
        fx.c[0] = xr && left > 0 ? *reinterpret_cast<const uint4*>(xl) : zero;
        fx.c[1] = xr && left > 16 ? *reinterpret_cast<const uint4*>(xl + 16) : zero;
        const int64_t at = (p.m0 + m) * GK + gk;
        if constexpr (SCALE == SCALE_F32) {
          const float sx = xr ? scale_at<SCALE>(a.xs, at) : 0.f;
          const f32x4 d = mfma_step<KIND_FP8B>(fw, fx, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_fmaf(d[i], sx * sw[i], acc[t][i]);
        } else {
          const int ex = xr ? static_cast<const uint8_t*>(a.xs)[at] : 127;
          acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              as_i32x8(fw.c[0], fw.c[1]), as_i32x8(fx.c[0], fx.c[1]), acc[t], 0, 0, 0, ew, 0, ex);
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) sums[wave][t][lane] = acc[t];
  __syncthreads();
  for (int t = wave; t < NT; t += kW) {
    f32x4 v = sums[0][t][lane];
#pragma unroll
    for (int w = 1; w < kW; ++w) v += sums[w][t][lane];
    const int m = 16 * t + r16;
    const int64_t row = (DW ? p.e * a.M : 0) + p.m0 + m;
    if (m < p.rows) store4<OELEM>(a.out, row, n0 + 4 * g, a.N, v);
  }
}

template <class F>
void by_types(const Fp8Args& a, F f) {
  auto with = [&](auto OELEM) {
    if (a.scale_type == SCALE_F32) f(OELEM, std::integral_constant<int, SCALE_F32>{});
    else f(OELEM, std::integral_constant<int, SCALE_E8M0>{});
  };
  if (a.oelem == ELEM_F16) with(std::integral_constant<int, ELEM_F16>{});
  else with(std::integral_constant<int, ELEM_BF16>{});
}

template <int OELEM, int SCALE, int NT, bool DW>
void rows_kernel(const Fp8Args& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.M + 16 * NT - 1) / (16 * NT)), (unsigned)((a.N + 15) / 16),
                  (unsigned)(DW ? a.E : 1));
  hipLaunchKernelGGL((k_fp8_rows<OELEM, SCALE, NT, DW>), grid, dim3(kW * 64), 0, stream, a);
}

}  // namespace

hipError_t launch_fp8_linear(const Fp8Args& a, hipStream_t stream) {
  if (a.M == 0) return hipSuccess;
  by_types(a, [&](auto OELEM, auto SCALE) {
    if (a.dw) rows_kernel<OELEM(), SCALE(), 4, true>(a, stream);
    else if (a.experts ? a.block_m == 16 : a.M <= 16) rows_kernel<OELEM(), SCALE(), 1, false>(a, stream);
    else if (a.experts ? a.block_m == 32 : a.M <= 32) rows_kernel<OELEM(), SCALE(), 2, false>(a, stream);
    else rows_kernel<OELEM(), SCALE(), 4, false>(a, stream);
  });
  return hipGetLastError();
}
