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

// ---- many rows: tiles staged in LDS ------------------------------------------
//
// A workgroup computes BM rows of X by BN rows of W; a wave TM x 64 of them.  One
// 128-wide step of both operands is a stage of LDS, brought there by direct loads
// NS - 1 steps ahead.  LDS rows are 128 bytes, chunk q of a row stored at q ^ key
// so that the 16 rows of a fragment read spread over the banks.
//
// A wave's four subtiles of W interleave: row r of subtile s is W's row 16 (r / 4) +
// 4 s + r % 4 of the wave's 64, so that a lane ends with 16 consecutive n of one row.
constexpr int kRow = 128;
constexpr uint32_t kOut = 0xC0000000u;  // an offset past every buffer: loads zeros

__device__ __forceinline__ int x_key(int r) { return r & 7; }
__device__ __forceinline__ int w_key(int r) { return (r & 3) | ((r >> 4) & 1) << 2; }

template <int BM, int BN, int TM, int NS, int SCALE, bool DW>
struct Tile {
  static constexpr int MI = TM / 16, NI = 4;
  static constexpr int WN = BN / 64, WM = BM / TM, NW = WM * WN;
  static constexpr int X = BM * kRow, W = BN * kRow;
  static constexpr int SX = SCALE == SCALE_F32 ? BM * 4 : 0;  // row scales of a stage
  static constexpr int SW = SCALE == SCALE_F32 && DW ? BN * 4 : 0;
  static constexpr int STAGE = X + W + SX + SW;
  static constexpr int XI = X / 1024 / NW, WI = W / 1024 / NW;  // 16-byte loads a wave and stage
  static constexpr int SI = (SX + SW) / 256;                    // 4-byte loads, one a wave
  static_assert(X % (1024 * NW) == 0 && W % (1024 * NW) == 0 && SI <= NW);
  static constexpr int THREADS = NW * 64;
};

__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's LDS reads are done
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Four steps' e8m0 scales from byte i on; n bytes in all (at least four).
__device__ __forceinline__ uint32_t scales4(const uint8_t* p, int64_t i, int64_t n) {
  typedef uint32_t u32_any __attribute__((aligned(1)));
  const int64_t at = i + 4 <= n ? i : n - 4;
  return *reinterpret_cast<const u32_any*>(p + at) >> (8 * (int)(i - at));
}

template <int OELEM, int SCALE, bool DW, int BM, int BN, int TM, int NS>
__global__ void __launch_bounds__((Tile<BM, BN, TM, NS, SCALE, DW>::THREADS))
k_fp8_tiles(Fp8Args a, int mtiles, int ntiles) {
  using C = Tile<BM, BN, TM, NS, SCALE, DW>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NS * C::STAGE];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int g = lane >> 4, r16 = lane & 15;
  const int wm = wave / C::WN, wn = wave % C::WN;
  // consecutive tiles on one XCD; groups of four row tiles walk the columns together
  int valid = mtiles;
  if (!DW && a.experts) valid = min((min(max(*a.ntp, 0), (int)a.M) + BM - 1) / BM, mtiles);
  const int total = valid * ntiles;
  const int per = (total + 7) / 8, j = blockIdx.x / 8;
  const int tile = (blockIdx.x % 8) * per + j;
  if (j >= per || tile >= total) return;
  const int band = tile / (4 * ntiles), inb = tile - band * 4 * ntiles;
  const int tall = min(4, valid - 4 * band);
  const int mt = 4 * band + inb % tall, nt = inb / tall;
  const Part p = part_of<DW>(a, mt, BM, blockIdx.y);
  if (p.none) return;
  const int64_t n0 = (int64_t)nt * BN;
  const int wrows = (int)min((int64_t)BN, a.N - n0);
  const int64_t K = a.K, GK = (K + 127) / 128;
  const int64_t we = DW ? 0 : max(p.e, 0);
  const int steps = p.e < 0 ? 0 : (int)((p.k1 - p.k0 + 127) / 128);
  const int tail = (int)(p.k1 - p.k0) & 127;  // bytes of a last step that is not whole

  const desc_t rx = make_desc(a.x + p.m0 * K + p.k0, (uint32_t)(p.rows * K - p.k0));
  const desc_t rw = make_desc(a.w + (we * a.N + n0) * K + p.k0, (uint32_t)(wrows * K - p.k0));
  uint32_t xo[C::XI], wo[C::WI];
  bool xt[C::XI], wt[C::WI];  // this lane's chunk lies behind the tail
#pragma unroll
  for (int t = 0; t < C::XI; ++t) {
    const int slot = (wave + C::NW * t) * 64 + lane, row = slot / 8, q = (slot % 8) ^ x_key(row);
    xo[t] = (uint32_t)row * (uint32_t)K + q * 16;
    xt[t] = q * 16 >= tail;
  }
#pragma unroll
  for (int t = 0; t < C::WI; ++t) {
    const int slot = (wave + C::NW * t) * 64 + lane, row = slot / 8, q = (slot % 8) ^ w_key(row);
    wo[t] = (uint32_t)row * (uint32_t)K + q * 16;
    wt[t] = q * 16 >= tail;
  }
  const uint32_t lds0 = lds_addr(smem);
  // row scales: wave w brings rows [64 w, 64 w + 64) of X, then of W
  desc_t rs = rx;
  uint32_t so = 0;
  if constexpr (SCALE == SCALE_F32) {
    constexpr int XS = C::SX / 256;
    const bool isx = wave < XS;
    const int64_t first = isx ? p.m0 : n0;
    const int rows = isx ? p.rows : wrows;
    rs = make_desc(static_cast<const float*>(isx ? a.xs : a.ws) + first * GK, (uint32_t)(rows * GK * 4));
    so = (uint32_t)((isx ? wave : wave - XS) * 64 + lane) * (uint32_t)(GK * 4);
  }
  const uint32_t g0 = (uint32_t)(p.k0 / 128);
  auto load = [&](int i) {
    const uint32_t st = lds0 + (uint32_t)(i % NS) * C::STAGE, k = (uint32_t)i * kRow;
    const bool cut = tail && i == steps - 1;
#pragma unroll
    for (int t = 0; t < C::XI; ++t) dma16(rx, st + (wave + C::NW * t) * 1024, cut && xt[t] ? kOut : xo[t], k);
#pragma unroll
    for (int t = 0; t < C::WI; ++t)
      dma16(rw, st + C::X + (wave + C::NW * t) * 1024, cut && wt[t] ? kOut : wo[t], k);
    if constexpr (SCALE == SCALE_F32)
      if (wave < C::SI) dma4(rs, st + C::X + C::W + wave * 256, so, (g0 + i) * 4);
  };
  f32x4 acc[C::MI][C::NI];
#pragma unroll
  for (int mi = 0; mi < C::MI; ++mi)
#pragma unroll
    for (int ni = 0; ni < C::NI; ++ni) acc[mi][ni] = f32x4{0.f, 0.f, 0.f, 0.f};

  // e8m0: four steps' scales of this lane's rows, and the next four's, requested in
  // the fourth step ahead of its operand loads (a wait for them after those
  // would wait for those too)
  uint32_t ex[C::MI], ew[C::NI], exn[C::MI], ewn[C::NI];
  auto load_e8 = [&](int i) {
    const int64_t gk = g0 + i;
#pragma unroll
    for (int mi = 0; mi < C::MI; ++mi) {
      const int64_t m = min(p.m0 + wm * TM + 16 * mi + r16, a.M - 1);
      exn[mi] = scales4(static_cast<const uint8_t*>(a.xs), m * GK + gk, a.M * GK);
    }
    if constexpr (DW) {
#pragma unroll
      for (int ni = 0; ni < C::NI; ++ni) {
        const int64_t n = min(n0 + wn * 64 + (r16 >> 2) * 16 + ni * 4 + (r16 & 3), a.N - 1);
        ewn[ni] = scales4(static_cast<const uint8_t*>(a.ws), n * GK + gk, a.N * GK);
      }
    } else {
      const int64_t NB = (a.N + 127) / 128, nb = min((n0 + wn * 64) / 128, NB - 1);
      ewn[0] = scales4(static_cast<const uint8_t*>(a.ws), (we * NB + nb) * GK + gk, a.E * NB * GK);
    }
  };
  const float* wsc = nullptr;  // fp32 layer: the scales of the wave's block of W
  if constexpr (SCALE == SCALE_F32 && !DW) {
    const int64_t NB = (a.N + 127) / 128, nb = min((n0 + wn * 64) / 128, NB - 1);
    wsc = static_cast<const float*>(a.ws) + (we * NB + nb) * GK;
  }

  if constexpr (SCALE == SCALE_E8M0)
    if (steps) load_e8(0);
#pragma unroll
  for (int i = 0; i < NS - 1; ++i)
    if (i < steps) load(i);
  for (int i = 0; i < steps; ++i) {
    wait_vmcnt<0>();
    lds_barrier();
    if constexpr (SCALE == SCALE_E8M0) {
      if ((i & 3) == 0) {
#pragma unroll
        for (int mi = 0; mi < C::MI; ++mi) ex[mi] = exn[mi];
#pragma unroll
        for (int ni = 0; ni < (DW ? C::NI : 1); ++ni) ew[ni] = ewn[ni];
      }
      if ((i & 3) == 3 && i + 1 < steps) load_e8(i + 1);
    }
    if (i + NS - 1 < steps) load(i + NS - 1);
    const uint8_t* st = smem + (i % NS) * C::STAGE;
    Frag<KIND_FP8B> fw[C::NI];
#pragma unroll
    for (int ni = 0; ni < C::NI; ++ni) {
      const int row = wn * 64 + (r16 >> 2) * 16 + ni * 4 + (r16 & 3);
      const uint8_t* q = st + C::X + row * kRow;
      fw[ni].c[0] = *reinterpret_cast<const uint4*>(q + ((g ^ w_key(row)) << 4));
      fw[ni].c[1] = *reinterpret_cast<const uint4*>(q + (((4 + g) ^ w_key(row)) << 4));
    }
    float sw[C::NI][4];
    if constexpr (SCALE == SCALE_F32) {
      if constexpr (DW) {
        const float* q = reinterpret_cast<const float*>(st + C::X + C::W + C::SX);
#pragma unroll
        for (int ni = 0; ni < C::NI; ++ni)
#pragma unroll
          for (int c = 0; c < 4; ++c) sw[ni][c] = q[wn * 64 + g * 16 + ni * 4 + c];
      } else {
        sw[0][0] = wsc[i];
      }
    }
#pragma unroll
    for (int mi = 0; mi < C::MI; ++mi) {
      const int row = wm * TM + 16 * mi + r16;
      const uint8_t* q = st + row * kRow;
      Frag<KIND_FP8B> fx;
      fx.c[0] = *reinterpret_cast<const uint4*>(q + ((g ^ x_key(row)) << 4));
      fx.c[1] = *reinterpret_cast<const uint4*>(q + (((4 + g) ^ x_key(row)) << 4));
      if constexpr (SCALE == SCALE_F32) {
        float sx = reinterpret_cast<const float*>(st + C::X + C::W)[row];
        if constexpr (!DW) sx *= sw[0][0];
#pragma unroll
        for (int ni = 0; ni < C::NI; ++ni) {
          const f32x4 d = mfma_step<KIND_FP8B>(fw[ni], fx, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int c = 0; c < 4; ++c)
            acc[mi][ni][c] = __builtin_fmaf(d[c], DW ? sx * sw[ni][c] : sx, acc[mi][ni][c]);
        }
      } else {
#pragma unroll
        for (int ni = 0; ni < C::NI; ++ni)
          acc[mi][ni] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              as_i32x8(fw[ni].c[0], fw[ni].c[1]), as_i32x8(fx.c[0], fx.c[1]), acc[mi][ni], 0, 0, 0,
              (int)ew[DW ? ni : 0], 0, (int)ex[mi]);
        ex[mi] >>= 8;
      }
    }
    if constexpr (SCALE == SCALE_E8M0) {
#pragma unroll
      for (int ni = 0; ni < (DW ? C::NI : 1); ++ni) ew[ni] >>= 8;
    }
  }
  // a lane: row m, 16 consecutive n
  const int64_t n = n0 + wn * 64 + g * 16;
#pragma unroll
  for (int mi = 0; mi < C::MI; ++mi) {
    const int m = wm * TM + 16 * mi + r16;
    if (m >= p.rows) continue;
    uint16_t* o = static_cast<uint16_t*>(a.out) + ((DW ? p.e * a.M : 0) + p.m0 + m) * a.N + n;
    uint32_t v[8];
#pragma unroll
    for (int ni = 0; ni < 4; ++ni)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        v[2 * ni + c] = to_elem<OELEM>(acc[mi][ni][2 * c]) | to_elem<OELEM>(acc[mi][ni][2 * c + 1]) << 16;
    if ((a.N & 7) == 0 && n + 16 <= a.N) {
      reinterpret_cast<uint4*>(o)[0] = make_uint4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<uint4*>(o)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int c = 0; c < 16; ++c)
        if (n + c < a.N) o[c] = (uint16_t)(c & 1 ? v[c / 2] >> 16 : v[c / 2]);
    }
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

template <int OELEM, int SCALE, bool DW, int BM, int BN, int TM, int NS>
void tile_kernel(const Fp8Args& a, hipStream_t stream) {
  const int mt = (int)((a.M + BM - 1) / BM), nt = (int)((a.N + BN - 1) / BN);
  const unsigned tiles = ((unsigned)(mt * nt) + 7) / 8 * 8;
  hipLaunchKernelGGL((k_fp8_tiles<OELEM, SCALE, DW, BM, BN, TM, NS>), dim3(tiles, (unsigned)(DW ? a.E : 1)),
                     dim3(Tile<BM, BN, TM, NS, SCALE, DW>::THREADS), 0, stream, a, mt, nt);
}

}  // namespace

hipError_t launch_fp8_linear(const Fp8Args& a, hipStream_t stream) {
  if (a.M == 0) return hipSuccess;
  by_types(a, [&](auto OELEM, auto SCALE) {
    constexpr int O = OELEM(), S = SCALE();
    const int64_t rows = a.experts && !a.dw ? a.block_m : a.M;
    if (a.dw) {
      if (a.M > 64 && a.N > 64) tile_kernel<O, S, true, 256, 256, 128, 2>(a, stream);
      else rows_kernel<O, S, 4, true>(a, stream);
    } else if (rows <= 16) {
      rows_kernel<O, S, 1, false>(a, stream);
    } else if (rows <= 32) {
      rows_kernel<O, S, 2, false>(a, stream);
    } else if (rows <= 64) {
      rows_kernel<O, S, 4, false>(a, stream);
    } else if (rows <= 128) {
      tile_kernel<O, S, false, 128, 128, 64, 2>(a, stream);
    } else {
      tile_kernel<O, S, false, 256, 256, 128, 2>(a, stream);
    }
  });
  return hipGetLastError();
}
