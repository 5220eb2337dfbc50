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
// 128-wide step of both operands and of their rows' scales is a stage of LDS,
// brought there by direct loads one step ahead; there are two.  LDS rows are 128
// bytes, chunk q of a row stored at q ^ key so that the 16 rows of a fragment read
// spread over the banks.  Workgroups stay and take tile after tile: the last step
// of one requests the first of the next, which so arrives while the sums are
// written.
//
// A wave's four subtiles of W interleave: row r of subtile s is W's row 32 (s / 2) +
// 8 (r / 4) + 4 (s % 2) + r % 4 of the wave's 64, so that a lane ends with eight
// consecutive n of one row, twice, and four lanes with 64 bytes of it.
constexpr int kRow = 128;
constexpr uint32_t kOut = 0xC0000000u;  // an offset past every buffer: loads zeros
constexpr int kMaxPlanExperts = kFp8MaxPlanExperts;
constexpr int kMaxPlanBlocks = 4096;    // of a layer over a plan whose blocks are put together

__device__ __forceinline__ int x_key(int r) { return r & 7; }
__device__ __forceinline__ int w_key(int r) { return (r & 3) | ((r >> 3) & 1) << 2; }

constexpr int w_sub(int ni) { return (ni >> 1) * 32 + (ni & 1) * 4; }

template <int BM, int BN, int TM>
struct Tile {
  static constexpr int MI = TM / 16, NI = 4;
  static constexpr int WN = BN / 64, WM = BM / TM, NW = WM * WN;
  static constexpr int X = BM * kRow, W = BN * kRow;
  static constexpr int S = NW * 256;  // scales: 64 rows a wave, X's then W's
  static constexpr int STAGE = X + W + S;
  static constexpr int XI = X / 1024 / NW, WI = W / 1024 / NW;  // 16-byte loads a wave and stage
  static constexpr int LROWS = NW * 8;                          // rows of one such load
  static_assert(X % (1024 * NW) == 0 && W % (1024 * NW) == 0 && (BM + BN) / 64 <= NW && BM % 64 == 0);
  static constexpr int PER = (XI + WI + MI - 1) / MI;  // loads beside each row subtile's products
  static constexpr int THREADS = NW * 64;
};

__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's LDS reads are done
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// A byte a lane, as a dword, to LDS.
__device__ __forceinline__ void dma1(desc_t r, uint32_t m0, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_ubyte %1, %2, %3 offen lds"
               :: "s"(__builtin_amdgcn_readfirstlane(m0)), "v"(voff), "s"(r),
                  "s"(__builtin_amdgcn_readfirstlane(soff)) : "memory");
}

template <int OELEM>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 v = {lo, hi};
  if constexpr (OELEM == ELEM_F16) {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
  } else {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
  }
}

// Where a tile's operands lie, all wave-uniform.
struct Source {
  const uint8_t* x;   // first row of X, first step
  const uint8_t* w;
  const uint8_t* s;   // this wave's 64 rows of scales
  int xn, wn, sn;     // bytes from there to the last row's end
  int steps;
};

// Row tiles of a plan: of each run of blocks with one expert every `per`-th (a power
// of two) begins a tile.  tab[t] = block + 2 kMaxPlanBlocks * expert (kNoExpert for one
// that is elsewhere); tab[tiles] = nb.  Returns the tiles.  Every thread calls this;
// nb <= kMaxPlanBlocks.
constexpr int kNoExpert = (1 << 30) / kMaxPlanBlocks - 1;

template <int NW>
__device__ __forceinline__ int join_blocks(const Fp8Args& a, int nb, int per, int* tab) {
  __shared__ int last[NW], cnt[NW];
  const int lane = threadIdx.x & 63, wave = wave_id();
  int run = 0, tiles = 0;  // where the last run began, tiles so far
  for (int base = 0; base < nb; base += NW * 64) {
    const int b = base + threadIdx.x;
    const int e = b < nb ? a.experts[b] : -1;
    const bool begins = b < nb && (b == 0 || a.experts[b - 1] != e);
    int at = begins ? b : -1;  // the last beginning up to here
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(at, d);
      if (lane >= d) at = max(at, o);
    }
    if (lane == 63) last[wave] = at;
    __syncthreads();
    int before = run;
    for (int w = 0; w < NW; ++w) {
      if (w < wave) before = max(before, last[w]);
      run = max(run, last[w]);
    }
    at = max(at, before);
    const bool lead = b < nb && ((b - at) & (per - 1)) == 0;
    const uint64_t who = __ballot(lead);
    if (lane == 0) cnt[wave] = __builtin_popcountll(who);
    __syncthreads();
    int to = tiles;
    for (int w = 0; w < NW; ++w) {
      if (w < wave) to += cnt[w];
      tiles += cnt[w];
    }
    to += __builtin_popcountll(who & ((1ull << lane) - 1));
    if (lead) tab[to] = b + 2 * kMaxPlanBlocks * ((unsigned)e < (unsigned)a.E ? e : kNoExpert);
    __syncthreads();
  }
  if (threadIdx.x == 0) tab[tiles] = nb;
  __syncthreads();
  return tiles;
}

template <int OELEM, int SCALE, bool DW, bool PLAN, int BM, int BN, int TM>
__global__ void __launch_bounds__((Tile<BM, BN, TM>::THREADS))
k_fp8_tiles(Fp8Args a, int mtiles, int ntiles) {
  using C = Tile<BM, BN, TM>;
  constexpr int SB = SCALE == SCALE_F32 ? 4 : 1;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * C::STAGE];
  __shared__ int tab[!PLAN ? 1 : DW ? 2 * kMaxPlanExperts : kMaxPlanBlocks + 1];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int g = lane >> 4, r16 = lane & 15;
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int K = (int)a.K, GK = (K + 127) / 128;

  // plan: the row tiles there are, and (gradient) each expert's blocks
  int valid = mtiles;
  int64_t M = a.M;
  bool joined = false;
  if constexpr (PLAN && !DW) {
    M = min((int64_t)max(*a.ntp, 0), a.M);
    valid = (int)((M + a.block_m - 1) / a.block_m);
    // Blocks that follow each other with one expert are put together into tiles of up
    // to BM rows: tab[t] is tile t's first block and, above, its expert.  More
    // blocks than fit are tiles of their own.
    joined = a.block_m < BM && valid <= kMaxPlanBlocks && a.E < kNoExpert;
    if (joined) valid = join_blocks<C::NW>(a, valid, BM / a.block_m, tab);
  }
  if constexpr (PLAN && DW) {
    int* first = tab;
    int* count = tab + kMaxPlanExperts;
    for (int e = threadIdx.x; e < a.E; e += C::THREADS) {
      first[e] = 0x7FFFFFFF;
      count[e] = 0;
    }
    __syncthreads();
    const int nb = min(max(*a.ntp, 0) / a.block_m, a.n_blocks);
    for (int b = threadIdx.x; b < nb; b += C::THREADS) {
      const int e = a.experts[b];
      if ((unsigned)e < (unsigned)a.E) {
        atomicAdd(&count[e], 1);
        atomicMin(&first[e], b);
      }
    }
    __syncthreads();
  }
  // consecutive tiles on one XCD, which its workgroups walk together; in bands of
  // four row tiles by all columns
  const int per_e = valid * ntiles, total = DW ? per_e * a.E : per_e;
  const int per = (total + 7) / 8, here = gridDim.x / 8;
  const int tile0 = (blockIdx.x % 8) * per, tile_end = min(tile0 + per, total);
  int tile = tile0 + blockIdx.x / 8;

  // a tile: its place, and where its operands lie.  rows = 0: nothing to do
  struct At {
    int64_t m0, n0, out;
    int rows, e;
  };
  auto place = [&](int t, Source& src) {
    At p;
    const int z = DW ? t / per_e : 0;
    const int u = t - z * per_e;
    constexpr int BAND = 4;
    const int band = u / (BAND * ntiles), inb = u - band * BAND * ntiles;
    const int tall = min(BAND, valid - BAND * band);
    const int mt = BAND * band + inb % tall;
    p.n0 = (int64_t)(inb / tall) * BN;
    p.m0 = (int64_t)mt * BM;
    p.e = z;
    int64_t end = M, k0 = 0, k1 = a.K;
    if constexpr (PLAN && DW) {
      const int count = __builtin_amdgcn_readfirstlane(tab[kMaxPlanExperts + z]);
      k0 = count ? (int64_t)__builtin_amdgcn_readfirstlane(tab[z]) * a.block_m : 0;
      k1 = min(k0 + (int64_t)count * a.block_m, a.K);
    } else if constexpr (PLAN) {
      int first = mt, past = mt + 1;
      if (joined) {
        const int at = __builtin_amdgcn_readfirstlane(tab[mt]);
        first = at & (2 * kMaxPlanBlocks - 1);
        past = __builtin_amdgcn_readfirstlane(tab[mt + 1]) & (2 * kMaxPlanBlocks - 1);
        p.e = at / (2 * kMaxPlanBlocks);
      } else {
        p.e = __builtin_amdgcn_readfirstlane(a.experts[mt]);
      }
      if ((unsigned)p.e >= (unsigned)a.E) p.e = -1;
      p.m0 = (int64_t)first * a.block_m;
      end = min((int64_t)past * a.block_m, M);
    }
    p.rows = (int)max(min(end - p.m0, (int64_t)BM), (int64_t)0);
    p.out = (DW ? z * a.M : 0) + p.m0;
    const int64_t we = DW ? 0 : max(p.e, 0);
    const int wrows = (int)min((int64_t)BN, a.N - p.n0);
    src.x = a.x + p.m0 * K + k0;
    src.w = a.w + (we * a.N + p.n0) * K + k0;
    src.xn = (int)(p.rows * K - k0);
    src.wn = (int)(wrows * K - k0);
    src.steps = p.e < 0 || p.rows == 0 ? 0 : (int)((k1 - k0 + 127) / 128);
    // scales: this wave's 64 rows of X, of W, or of nothing
    const int r = wave * 64;
    const uint8_t* ws = static_cast<const uint8_t*>(a.ws);
    if (r < BM) {
      src.s = static_cast<const uint8_t*>(a.xs) + ((p.m0 + r) * GK + k0 / 128) * SB;
      src.sn = (int)(((p.rows - r) * (int64_t)GK - k0 / 128) * SB);
    } else if constexpr (DW) {
      src.s = ws + ((p.n0 + r - BM) * GK + k0 / 128) * SB;
      src.sn = (int)(((wrows - (r - BM)) * (int64_t)GK - k0 / 128) * SB);
    } else {
      // the rows of a block of W share a scale (every lane loads it)
      const int64_t NB = (a.N + 127) / 128, nb = min((p.n0 + r - BM) / 128, NB - 1);
      src.s = ws + (we * NB + nb) * GK * SB;
      src.sn = r < BM + BN ? GK * SB : 0;
    }
    return p;
  };

  // this lane's chunks: load t adds t * LROWS rows.  In a last step that is not
  // whole, chunks behind K load zeros
  const int tail = K & 127;
  const int slot0 = wave * 64 + lane, row0 = slot0 / 8;
  const int xq = (slot0 % 8) ^ x_key(row0), wq = (slot0 % 8) ^ w_key(row0);
  const uint32_t xo = (uint32_t)row0 * (uint32_t)K + xq * 16, wo = (uint32_t)row0 * (uint32_t)K + wq * 16;
  const uint32_t xo_last = tail && xq * 16 >= tail ? kOut : xo, wo_last = tail && wq * 16 >= tail ? kOut : wo;
  const uint32_t so = !DW && wave * 64 >= BM ? 0 : (uint32_t)lane * (uint32_t)(GK * SB);
  const uint32_t lds0 = lds_addr(smem);

  // requests load t of a step into stage `slot`; t < 0: the scales
  auto load1 = [&](const Source& s, int step, int slot, int t) {
    const uint32_t st = lds0 + (uint32_t)(slot * C::STAGE);
    const bool last = step == s.steps - 1;
    const int k = step * kRow;
    if (t < 0) {
      const desc_t r = make_desc(s.s + step * SB, (uint32_t)max(s.sn - step * SB, 0));
      if constexpr (SCALE == SCALE_F32) dma4(r, st + C::X + C::W + wave * 256, so, 0);
      else dma1(r, st + C::X + C::W + wave * 256, so, 0);
    } else if (t < C::WI) {
      const int d = t * C::LROWS * K + k;
      dma16(make_desc(s.w + d, (uint32_t)max(s.wn - d, 0)), st + C::X + (wave + C::NW * t) * 1024,
            last ? wo_last : wo, 0);
    } else {
      const int d = (t - C::WI) * C::LROWS * K + k;
      dma16(make_desc(s.x + d, (uint32_t)max(s.xn - d, 0)), st + (wave + C::NW * (t - C::WI)) * 1024,
            last ? xo_last : xo, 0);
    }
  };

  f32x4 acc[C::MI][C::NI];
  Source cur, nxt;
  At p, q;
  nxt.steps = 0;
  if (tile >= tile_end) return;
  p = place(tile, cur);
  if (cur.steps) {
#pragma unroll
    for (int t = -1; t < C::WI + C::XI; ++t) load1(cur, 0, 0, t);
  }
  int slot = 0;
  bool stores = false;  // a whole tile's stores may be under way
  for (;;) {
    const int after = tile + here;
    const bool more = after < tile_end;
    if (more) q = place(after, nxt);
    if (!more) nxt.steps = 0;
#pragma unroll
    for (int mi = 0; mi < C::MI; ++mi)
#pragma unroll
      for (int ni = 0; ni < C::NI; ++ni) acc[mi][ni] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < cur.steps; ++i) {
      // the stage has landed (stores behind it may be pending), and every wave
      // is done with the other
      if (stores) wait_vmcnt<2 * C::MI>();
      else wait_vmcnt<0>();
      stores = false;
      lds_barrier();
      // what to request: the next step, or the next tile's first
      const bool end = i + 1 == cur.steps;
      Source f;
      f.x = end ? nxt.x : cur.x;
      f.w = end ? nxt.w : cur.w;
      f.s = end ? nxt.s : cur.s;
      const bool none = end && nxt.steps == 0;
      f.xn = none ? 0 : end ? nxt.xn : cur.xn;
      f.wn = none ? 0 : end ? nxt.wn : cur.wn;
      f.sn = none ? 0 : end ? nxt.sn : cur.sn;
      f.steps = end ? nxt.steps : cur.steps;
      const int fstep = end ? 0 : i + 1;
      if (none) f.x = cur.x, f.w = cur.w, f.s = cur.s;
      const uint8_t* st = smem + slot * C::STAGE;
      const uint8_t* xr = st + (wm * TM + r16) * kRow + ((g ^ x_key(r16)) << 4);
      const uint8_t* xr2 = st + (wm * TM + r16) * kRow + (((4 + g) ^ x_key(r16)) << 4);
      const int wrow = wn * 64 + (r16 >> 2) * 8 + (r16 & 3);
      const uint8_t* wr = st + C::X + wrow * kRow + ((g ^ w_key(wrow)) << 4);
      const uint8_t* wr2 = st + C::X + wrow * kRow + (((4 + g) ^ w_key(wrow)) << 4);
      const uint32_t* sc = reinterpret_cast<const uint32_t*>(st + C::X + C::W);
      Frag<KIND_FP8B> fx[2], fw[C::NI];
      uint32_t sx[2];
      auto read_x = [&](int mi) {
        fx[mi & 1].c[0] = *reinterpret_cast<const uint4*>(xr + mi * 16 * kRow);
        fx[mi & 1].c[1] = *reinterpret_cast<const uint4*>(xr2 + mi * 16 * kRow);
        sx[mi & 1] = sc[wm * TM + r16 + 16 * mi];
      };
      read_x(0);
      float sw[DW ? C::NI : 1][4];
      uint32_t ew[DW ? C::NI : 1];
      if constexpr (SCALE == SCALE_F32) {
        if constexpr (DW) {
#pragma unroll
          for (int ni = 0; ni < C::NI; ++ni) {
            const float4 v = *reinterpret_cast<const float4*>(sc + BM + wn * 64 + g * 8 + w_sub(ni));
            sw[ni][0] = v.x, sw[ni][1] = v.y, sw[ni][2] = v.z, sw[ni][3] = v.w;
          }
        } else {
          sw[0][0] = __uint_as_float(sc[BM + wn * 64]);
        }
      } else {
#pragma unroll
        for (int ni = 0; ni < (DW ? C::NI : 1); ++ni) ew[ni] = sc[BM + wrow + w_sub(ni)];
      }
#pragma unroll
      for (int ni = 0; ni < C::NI; ++ni) {
        fw[ni].c[0] = *reinterpret_cast<const uint4*>(wr + w_sub(ni) * kRow);
        fw[ni].c[1] = *reinterpret_cast<const uint4*>(wr2 + w_sub(ni) * kRow);
      }
      load1(f, fstep, slot ^ 1, -1);
#pragma unroll
      for (int mi = 0; mi < C::MI; ++mi) {
        if (mi + 1 < C::MI) read_x(mi + 1);
#pragma unroll
        for (int u = 0; u < C::PER; ++u)
          if (mi * C::PER + u < C::XI + C::WI) load1(f, fstep, slot ^ 1, mi * C::PER + u);
        const Frag<KIND_FP8B>& x = fx[mi & 1];
        if constexpr (SCALE == SCALE_F32) {
          float s = __uint_as_float(sx[mi & 1]);
          if constexpr (!DW) s *= sw[0][0];
#pragma unroll
          for (int ni = 0; ni < C::NI; ++ni) {
            const f32x4 d = mfma_step<KIND_FP8B>(fw[ni], x, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int c = 0; c < 4; ++c)
              acc[mi][ni][c] = __builtin_fmaf(d[c], DW ? s * sw[DW ? ni : 0][c] : s, acc[mi][ni][c]);
          }
        } else {
#pragma unroll
          for (int ni = 0; ni < C::NI; ++ni)
            acc[mi][ni] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                as_i32x8(fw[ni].c[0], fw[ni].c[1]), as_i32x8(x.c[0], x.c[1]), acc[mi][ni], 0, 0, 0,
                (int)ew[DW ? ni : 0], 0, (int)sx[mi & 1]);
        }
      }
      slot ^= 1;
    }
    if (cur.steps == 0 && nxt.steps) {  // no step has requested the next tile's first
#pragma unroll
      for (int t = -1; t < C::WI + C::XI; ++t) load1(nxt, 0, slot, t);
    }
    // a lane: row m, n to n + 7 and n + 32 to n + 39
    const int64_t n = p.n0 + wn * 64 + g * 8;
    const bool whole = p.rows == BM && p.n0 + BN <= a.N && (a.N & 7) == 0;
#pragma unroll
    for (int mi = 0; mi < C::MI; ++mi) {
      typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
      u32x4 v[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          v[h][c] = pack2<OELEM>(acc[mi][2 * h + c / 2][2 * (c & 1)], acc[mi][2 * h + c / 2][2 * (c & 1) + 1]);
      if (whole) {
        // lanes r and r + 8 trade halves, so that a store writes whole lines: eight
        // rows of 128 bytes
        const bool low = r16 < 8;
        u32x4 first, second;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t give = low ? v[1][c] : v[0][c];
          const uint32_t got = (uint32_t)__builtin_amdgcn_mov_dpp((int)give, 0x128, 0xF, 0xF, true);  // row_ror 8
          first[c] = low ? v[0][c] : got;
          second[c] = low ? got : v[1][c];
        }
        const int from = ((lane & 3) * 16 + (lane >> 3) + 8 * ((lane >> 2) & 1)) * 4;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          first[c] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)first[c]);
          second[c] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)second[c]);
        }
        uint16_t* o = static_cast<uint16_t*>(a.out) + (p.out + wm * TM + 16 * mi + (lane >> 3)) * a.N + p.n0 +
                      wn * 64 + 8 * (lane & 7);
        __builtin_nontemporal_store(first, reinterpret_cast<u32x4*>(o));
        __builtin_nontemporal_store(second, reinterpret_cast<u32x4*>(o + 8 * a.N));
      } else {
        const int m = wm * TM + 16 * mi + r16;
        uint16_t* o = static_cast<uint16_t*>(a.out) + (p.out + m) * a.N + n;
        if (m < p.rows) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < 8; ++c)
              if (n + 32 * h + c < a.N) o[32 * h + c] = (uint16_t)(c & 1 ? v[h][c / 2] >> 16 : v[h][c / 2]);
        }
      }
    }
    asm volatile("" ::: "memory");
    stores = whole;
    if (!more) break;
    tile = after;
    cur = nxt;
    p = q;
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

// workgroups that run at once on the current device: one a CU
int cus() {
  int dev = 0, n = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 8)
    return 256;
  return n / 8 * 8;
}

template <int OELEM, int SCALE, bool DW, int BM, int BN, int TM>
void tile_kernel(const Fp8Args& a, hipStream_t stream) {
  using C = Tile<BM, BN, TM>;
  const int64_t rows = a.experts && !DW ? a.block_m : BM;  // at most as many tiles as blocks
  const int64_t mt = (a.M + rows - 1) / rows, nt = (a.N + BN - 1) / BN, tiles = mt * nt * (DW ? a.E : 1);
  const int64_t fit = (int64_t)cus() * (2 * C::STAGE <= 80 * 1024 ? 2 : 1);
  const int64_t grid = tiles < fit ? (tiles + 7) / 8 * 8 : fit;
  if (a.experts)
    hipLaunchKernelGGL((k_fp8_tiles<OELEM, SCALE, DW, true, BM, BN, TM>), dim3((unsigned)grid),
                       dim3(C::THREADS), 0, stream, a, (int)mt, (int)nt);
  else
    hipLaunchKernelGGL((k_fp8_tiles<OELEM, SCALE, DW, false, BM, BN, TM>), dim3((unsigned)grid),
                       dim3(C::THREADS), 0, stream, a, (int)mt, (int)nt);
}

}  // namespace

hipError_t launch_fp8_linear(const Fp8Args& a, hipStream_t stream) {
  if (a.M == 0) return hipSuccess;
  by_types(a, [&](auto OELEM, auto SCALE) {
    constexpr int O = OELEM(), S = SCALE();
    const int64_t rows = a.experts && !a.dw ? a.block_m : a.M;
    if (a.dw) {
      if (a.M > 64 && a.N > 64) tile_kernel<O, S, true, 256, 256, 128>(a, stream);
      else rows_kernel<O, S, 4, true>(a, stream);
    } else if (rows <= 16) {
      rows_kernel<O, S, 1, false>(a, stream);
    } else if (rows <= 32) {
      rows_kernel<O, S, 2, false>(a, stream);
    } else if (rows <= 64) {
      rows_kernel<O, S, 4, false>(a, stream);
    } else if (!a.experts && rows <= 128) {
      tile_kernel<O, S, false, 128, 128, 64>(a, stream);
    } else {
      tile_kernel<O, S, false, 256, 256, 128>(a, stream);
    }
  });
  return hipGetLastError();
}
