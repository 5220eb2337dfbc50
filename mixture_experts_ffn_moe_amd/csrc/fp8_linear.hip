// fp8_linear.hip -- products of e4m3 values with a scale for each 128 of the
// contraction: linear layers (dense, or block by block of a plan with each
// block's expert) and the gradient of their weights.
//
//   out[m, n] = sum_g sx[m, g] sw[n, g] sum_{k in group g} X[m, k] W[n, k]
//
// W is the matrix instruction's A operand and X its B operand, so that a lane
// ends with one row m and four consecutive n.  With fp32 scales a group's sum
// leaves the instruction and is added in fp32 with its scale; e8m0 scales go into
// the instruction, which then adds up all groups by itself, the running sum in fp32.
// Inside 128 the instruction by itself cuts each product off below 2^-13 of the largest
// of its eight consecutive k; the output's rounding, 2^-8 or 2^-11 of a value, is coarser
// unless one of each eight outweighs the rest.
#include <type_traits>

#include "device.h"
#include "ops.h"

namespace {

// Two sums, rounded to the output's type.
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

// ---- few rows: weights streamed into registers --------------------------------
//
// A workgroup of KW waves: 16 * MW rows of W by 16 * NT rows of X.  The waves take
// the steps of k in turn, each with two steps requested ahead (the weights' bytes set
// the time), and add their sums in LDS in a fixed order.  Rows and chunks that do not
// exist load zeros past the buffers' ends.  One token, 4096 x 7168: 9.3 us from HBM (3.2
// TB/s), 7.5 where the 29 MB lie in the last-level cache; 64 tokens, top-6 of 64 experts
// of 4096 x 4096: 181 us, 5.9 TB/s.
constexpr uint32_t kOut = 0xC0000000u;  // an offset past every buffer

template <int SCALE>
__device__ __forceinline__ uint32_t load_scale(__amdgpu_buffer_rsrc_t r, uint32_t i) {
  if constexpr (SCALE == SCALE_F32) return __float_as_uint(buf_loadf(r, i * 4, 0));
  else return (uint32_t)buf_loadu8(r, i, 0);
}

// Four values of row m at columns n .. n + 3.
template <int OELEM>
__device__ __forceinline__ void store4(void* out, int64_t row, int64_t n, int64_t N, const f32x4& v) {
  uint16_t* o = static_cast<uint16_t*>(out) + row * N + n;
  const uint32_t lo = pack2<OELEM>(v[0], v[1]), hi = pack2<OELEM>(v[2], v[3]);
  if ((N & 3) == 0 && n + 4 <= N) {
    *reinterpret_cast<uint2*>(o) = make_uint2(lo, hi);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) o[i] = (uint16_t)((i < 2 ? lo : hi) >> (16 * (i & 1)));
  }
}

template <int OELEM, int SCALE, int NT, int MW, int KW>
__global__ void __launch_bounds__(KW * 64)
k_fp8_rows(Fp8Args a) {
  constexpr int SB = SCALE == SCALE_F32 ? 4 : 1;
  __shared__ f32x4 sums[KW][MW * NT][64];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int g = lane >> 4, r16 = lane & 15;
  // a row tile's columns follow each other: the workgroups that run together read
  // one expert's weights as they lie
  const uint32_t ntiles = (uint32_t)((a.N + 16 * MW - 1) / (16 * MW)), mt = blockIdx.x / ntiles;
  const int64_t n0 = (int64_t)(blockIdx.x - mt * ntiles) * (16 * MW), m0 = (int64_t)mt * (16 * NT);
  int64_t end = a.M;
  int e = 0;
  if (a.experts) {  // a row tile is a block
    end = min((int64_t)max(*a.ntp, 0), a.M);
    if (m0 >= end) return;
    e = a.experts[mt];
    if ((unsigned)e >= (unsigned)a.E) e = -1;
  }
  const int rows = (int)min(end - m0, (int64_t)(16 * NT));
  f32x4 acc[MW][NT];
#pragma unroll
  for (int j = 0; j < MW; ++j)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[j][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (e >= 0) {
    const int wrows = (int)min((int64_t)(16 * MW), a.N - n0);
    const int K = (int)a.K, GK = (K + 127) / 128;
    const auto rw = make_rsrc(a.w + ((int64_t)e * a.N + n0) * K, (uint32_t)(wrows * K));
    const auto rx = make_rsrc(a.x + m0 * K, (uint32_t)(rows * K));
    const auto rsx = make_rsrc(static_cast<const uint8_t*>(a.xs) + m0 * GK * SB, (uint32_t)(rows * GK * SB));
    const int64_t block = (int64_t)e * ((a.N + 127) / 128) + n0 / 128;  // of the weights' scales
    const auto rsw = make_rsrc(static_cast<const uint8_t*>(a.ws) + block * GK * SB, (uint32_t)(GK * SB));
    struct Step {
      uint4 w[MW][2], x[NT][2];
      uint32_t sw, sx[NT];
    };
    auto load = [&](Step& f, int ks) {
      if (ks >= GK) return;
      const int k = ks * 128 + 32 * g;
      const uint32_t o0 = k < K ? 0u : kOut, o1 = k + 16 < K ? 0u : kOut;
#pragma unroll
      for (int j = 0; j < MW; ++j) {
        const uint32_t wo = (uint32_t)((16 * j + r16) * K + k);
        f.w[j][0] = buf_load16(rw, wo | o0, 0);
        f.w[j][1] = buf_load16(rw, (wo + 16) | o1, 0);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint32_t xo = (uint32_t)((16 * t + r16) * K + k);
        f.x[t][0] = buf_load16(rx, xo | o0, 0);
        f.x[t][1] = buf_load16(rx, (xo + 16) | o1, 0);
        f.sx[t] = load_scale<SCALE>(rsx, (uint32_t)((16 * t + r16) * GK + ks));
      }
      f.sw = load_scale<SCALE>(rsw, (uint32_t)ks);
    };
    auto add = [&](const Step& f) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const i32x8 fx = as_i32x8(f.x[t][0], f.x[t][1]);
        const float s = __uint_as_float(f.sx[t]) * __uint_as_float(f.sw);
#pragma unroll
        for (int j = 0; j < MW; ++j) {
          const i32x8 fw = as_i32x8(f.w[j][0], f.w[j][1]);
          if constexpr (SCALE == SCALE_F32) {
            const f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                fw, fx, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][t][i] = __builtin_fmaf(d[i], s, acc[j][t][i]);
          } else {
            acc[j][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw, fx, acc[j][t], 0, 0, 0,
                                                                        (int)f.sw, 0, (int)f.sx[t]);
          }
        }
      }
    };
    constexpr int PD = 2;
    const int mine = (GK - wave + KW - 1) / KW;
    Step f[PD];
#pragma unroll
    for (int u = 0; u < PD; ++u) load(f[u], wave + u * KW);
    for (int i = 0; i < mine; i += PD) {
#pragma unroll
      for (int u = 0; u < PD; ++u) {
        if (i + u < mine) add(f[u]);
        load(f[u], wave + (i + u + PD) * KW);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < MW; ++j)
#pragma unroll
    for (int t = 0; t < NT; ++t) sums[wave][j * NT + t][lane] = acc[j][t];
  __syncthreads();
  for (int u = wave; u < MW * NT; u += KW) {
    f32x4 v = sums[0][u][lane];
#pragma unroll
    for (int w = 1; w < KW; ++w) v += sums[w][u][lane];
    const int m = 16 * (u % NT) + r16;
    const int64_t n = n0 + 16 * (u / NT) + 4 * g;
    if (m < rows && n < a.N) store4<OELEM>(a.out, m0 + m, n, a.N, v);
  }
}

// ---- more rows: tiles staged in LDS --------------------------------------------
//
// A tile is BM rows of X by BN rows of W; a wave has TM x 64 of it.  One 128-wide step
// of both operands and of their rows' scales is a stage of LDS, brought there by
// direct loads.  LDS rows are 128 bytes, chunk q of a row stored at q ^ key so that
// the 16 rows of a fragment read spread over the banks.
//
// A wave's four subtiles of W interleave: row r of subtile s is W's row 32 (s / 2) +
// 8 (r / 4) + 4 (s % 2) + r % 4 of the wave's 64, so that a lane ends with eight
// consecutive n of one row, twice, and four lanes with 64 bytes of it.
//
// Two kernels run on such tiles.  k_fp8_stay (256 x 256, two stages): a workgroup a
// CU that stays and takes tile after tile; a tile's last step requests the next
// one's first, which arrives while the sums are written.  (8192 x 7168 by 4096, e8m0:
// 181 to 195 us, 2.5 to 2.65 PFLOP/s; the matrix pipes are busy 62% of the cycles, at the
// 1.9 to 2.0 GHz that this load holds.)  k_fp8_tile (smaller tiles
// where those would leave CUs idle): a workgroup a tile, KG groups of waves that
// take the steps in turn, each with D stages, and add up in the end.
constexpr int kRow = 128;
constexpr int kMaxPlanExperts = kFp8MaxPlanExperts;
constexpr int kMaxPlanBlocks = 2048;  // of a layer over a plan whose blocks are put together
constexpr int kNoExpert = (1 << 30) / kMaxPlanBlocks - 1;

__device__ __forceinline__ int x_key(int r) { return r & 7; }
__device__ __forceinline__ int w_key(int r) { return (r & 3) | ((r >> 3) & 1) << 2; }
constexpr int w_sub(int ni) { return (ni >> 1) * 32 + (ni & 1) * 4; }

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

// Row tiles of a plan: of each run of blocks with one expert every `per`-th (a power
// of two) begins a tile.  tab[t] = block + 2 kMaxPlanBlocks * expert (kNoExpert for one
// that is elsewhere); tab[tiles] = nb.  Returns the tiles.  Every thread calls this;
// nb <= kMaxPlanBlocks.
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

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Where a tile's operands lie, all wave-uniform.
struct Source {
  const uint8_t* x;   // first row of X, first step
  const uint8_t* w;
  const uint8_t* s;   // this wave's 64 rows of scales
  int xn, wn, sn;     // bytes from there to the last row's end
  int steps;
};

// A tile's place: rows [m0, m0 + rows) and columns from n0, `out` its first row of
// the output; expert e (-1: the rows are zeros).
struct At {
  int64_t m0, n0, out;
  int rows, e;
};

template <int OELEM, int SCALE, bool DW, bool PLAN, int BM, int BN, int TM, int KG, int D>
struct Tiles {
  static constexpr int MI = TM / 16, NI = 4;
  static constexpr int WN = BN / 64, WM = BM / TM, NW = WM * WN;  // waves of a group
  static constexpr int X = BM * kRow, W = BN * kRow;
  static constexpr int S = NW * 256;  // scales: 64 rows a wave, X's then W's
  static constexpr int STAGE = X + W + S, LDS = D * KG * STAGE;  // D stages a group
  static constexpr int XI = X / 1024 / NW, WI = W / 1024 / NW;  // 16-byte loads a wave and stage
  static constexpr int LOADS = XI + WI + 1;                     // with the scales
  static constexpr int LROWS = NW * 8;                          // rows of one 16-byte load
  static constexpr int PER = (XI + WI + MI - 1) / MI;           // loads beside a row subtile's products
  static constexpr int THREADS = NW * KG * 64;
  static constexpr int TAB = !PLAN ? 1 : DW ? 2 * kMaxPlanExperts : BM > 128 ? kMaxPlanBlocks + 1 : 1;
  static constexpr int SB = SCALE == SCALE_F32 ? 4 : 1;
  static_assert(X % (1024 * NW) == 0 && W % (1024 * NW) == 0 && (BM + BN) / 64 <= NW && BM % 64 == 0);
  static_assert(LDS <= 160 * 1024 && (KG == 1 || (KG - 1) * NW * MI * NI * 1024 <= LDS));

  const Fp8Args& a;
  uint8_t* smem;
  int* tab;
  int K, GK, lane, wave, g, r16, wm, wn;
  int64_t M;             // rows in use
  int valid, ntiles, per_e, total;
  bool joined;
  uint32_t xo, wo, xo_last, wo_last, so, lds0;

  __device__ __forceinline__ Tiles(const Fp8Args& args, uint8_t* lds, int* table, int mtiles, int nt)
      : a(args), smem(lds), tab(table) {
    lane = threadIdx.x & 63;
    wave = wave_id() % NW;
    g = lane >> 4;
    r16 = lane & 15;
    wm = wave / WN;
    wn = wave % WN;
    K = (int)a.K;
    GK = (K + 127) / 128;
    M = a.M;
    valid = mtiles;
    ntiles = nt;
    joined = false;
    if constexpr (PLAN && !DW) {
      M = min((int64_t)max(*a.ntp, 0), a.M);
      const int rows = min(a.block_m, BM);  // a block is a tile, or tiles of BM rows
      valid = (int)((M + rows - 1) / rows);
      // Blocks that follow each other with one expert are put together into tiles of up
      // to BM rows: tab[t] is tile t's first block and, above, its expert.  More
      // blocks than fit are tiles of their own.
      if constexpr (BM > 128) {
        joined = a.block_m < BM && valid <= kMaxPlanBlocks && a.E < kNoExpert;
        if (joined) valid = join_blocks<NW * KG>(a, valid, BM / a.block_m, tab);
      }
    }
    if constexpr (PLAN && DW) {  // each expert's blocks
      int* first = tab;
      int* count = tab + kMaxPlanExperts;
      for (int e = threadIdx.x; e < a.E; e += THREADS) {
        first[e] = 0x7FFFFFFF;
        count[e] = 0;
      }
      __syncthreads();
      const int nb = min((int)((summed() + a.block_m - 1) / a.block_m), a.n_blocks);
      for (int b = threadIdx.x; b < nb; b += THREADS) {
        const int e = a.experts[b];
        if ((unsigned)e < (unsigned)a.E) {
          atomicAdd(&count[e], 1);
          atomicMin(&first[e], b);
        }
      }
      __syncthreads();
    }
    per_e = valid * ntiles;
    total = DW ? per_e * a.E : per_e;
    // this lane's chunks: load t adds t * LROWS rows.  In a last step that is not
    // whole, chunks behind K load zeros
    const int tail = K & 127;
    const int slot0 = wave * 64 + lane, row0 = slot0 / 8;
    const int xq = (slot0 % 8) ^ x_key(row0), wq = (slot0 % 8) ^ w_key(row0);
    xo = (uint32_t)row0 * (uint32_t)K + xq * 16;
    wo = (uint32_t)row0 * (uint32_t)K + wq * 16;
    xo_last = tail && xq * 16 >= tail ? kOut : xo;
    wo_last = tail && wq * 16 >= tail ? kOut : wo;
    so = !DW && wave * 64 >= BM ? 0 : (uint32_t)lane * (uint32_t)(GK * SB);
    lds0 = lds_addr(smem);
  }

  // The rows in use that a plan's gradient sums over.
  __device__ __forceinline__ int64_t summed() const { return min((int64_t)max(*a.ntp, 0), a.K); }

  // Tile t in the order of the walk: bands of four row tiles by all columns, so that
  // the tiles that run together on one XCD share both operands in its L2
  __device__ __forceinline__ At place(int t, Source& src) const {
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
      k1 = min(k0 + (int64_t)count * a.block_m, summed());
    } else if constexpr (PLAN) {
      if (joined) {
        const int at = __builtin_amdgcn_readfirstlane(tab[mt]);
        const int past = __builtin_amdgcn_readfirstlane(tab[mt + 1]) & (2 * kMaxPlanBlocks - 1);
        p.e = at / (2 * kMaxPlanBlocks);
        p.m0 = (int64_t)(at & (2 * kMaxPlanBlocks - 1)) * a.block_m;
        end = min((int64_t)past * a.block_m, M);
      } else {
        const int rows = min(a.block_m, BM);
        p.e = __builtin_amdgcn_readfirstlane(a.experts[mt / (a.block_m / rows)]);
        p.m0 = (int64_t)mt * rows;
        end = min(p.m0 + rows, M);
      }
      if ((unsigned)p.e >= (unsigned)a.E) p.e = -1;
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
      src.sn = r < BM + BN ? (int)(((wrows - (r - BM)) * (int64_t)GK - k0 / 128) * SB) : 0;
    } else {
      // the rows of a block of W share a scale (every lane loads it)
      const int64_t NB = (a.N + 127) / 128, nb = min((p.n0 + r - BM) / 128, NB - 1);
      src.s = ws + (we * NB + nb) * GK * SB;
      src.sn = r < BM + BN ? GK * SB : 0;
    }
    return p;
  }

  // Requests load t of a step into stage `slot`; t < 0: the scales.
  __device__ __forceinline__ void load1(const Source& s, int step, int slot, int t) const {
    const uint32_t st = lds0 + (uint32_t)(slot * STAGE);
    const bool last = step == s.steps - 1;
    const int k = step * kRow;
    if (t < 0) {
      const desc_t r = make_desc(s.s + step * SB, (uint32_t)max(s.sn - step * SB, 0));
      if constexpr (SCALE == SCALE_F32) dma4(r, st + X + W + wave * 256, so, 0);
      else dma1(r, st + X + W + wave * 256, so, 0);
    } else if (t < WI) {
      const int d = t * LROWS * K + k;
      dma16(make_desc(s.w + d, (uint32_t)max(s.wn - d, 0)), st + X + (wave + NW * t) * 1024,
            last ? wo_last : wo, 0);
    } else {
      const int d = (t - WI) * LROWS * K + k;
      dma16(make_desc(s.x + d, (uint32_t)max(s.xn - d, 0)), st + (wave + NW * (t - WI)) * 1024,
            last ? xo_last : xo, 0);
    }
  }

  __device__ __forceinline__ void load(const Source& s, int step, int slot) const {
#pragma unroll
    for (int t = -1; t < WI + XI; ++t) load1(s, step, slot, t);
  }

  // Adds a stage's products, and requests step `fstep` of f beside them.
  __device__ __forceinline__ void add(int slot, f32x4 (&acc)[MI][NI], const Source& f, int fstep,
                                      int fslot) const {
    const uint8_t* st = smem + slot * STAGE;
    const uint8_t* xr = st + (wm * TM + r16) * kRow + ((g ^ x_key(r16)) << 4);
    const uint8_t* xr2 = st + (wm * TM + r16) * kRow + (((4 + g) ^ x_key(r16)) << 4);
    const int wrow = wn * 64 + (r16 >> 2) * 8 + (r16 & 3);
    const uint8_t* wr = st + X + wrow * kRow + ((g ^ w_key(wrow)) << 4);
    const uint8_t* wr2 = st + X + wrow * kRow + (((4 + g) ^ w_key(wrow)) << 4);
    const uint32_t* sc = reinterpret_cast<const uint32_t*>(st + X + W);
    Frag<KIND_FP8B> fx[2], fw[NI];
    uint32_t sx[2];
    auto read_x = [&](int mi) {
      fx[mi & 1].c[0] = *reinterpret_cast<const uint4*>(xr + mi * 16 * kRow);
      fx[mi & 1].c[1] = *reinterpret_cast<const uint4*>(xr2 + mi * 16 * kRow);
      sx[mi & 1] = sc[wm * TM + r16 + 16 * mi];
    };
    read_x(0);
    float sw[DW ? NI : 1][4];
    uint32_t ew[DW ? NI : 1];
    if constexpr (SCALE == SCALE_F32) {
      if constexpr (DW) {
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) {
          const float4 v = *reinterpret_cast<const float4*>(sc + BM + wn * 64 + g * 8 + w_sub(ni));
          sw[ni][0] = v.x, sw[ni][1] = v.y, sw[ni][2] = v.z, sw[ni][3] = v.w;
        }
      } else {
        sw[0][0] = __uint_as_float(sc[BM + wn * 64]);
      }
    } else {
#pragma unroll
      for (int ni = 0; ni < (DW ? NI : 1); ++ni) ew[ni] = sc[BM + wrow + w_sub(ni)];
    }
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) {
      fw[ni].c[0] = *reinterpret_cast<const uint4*>(wr + w_sub(ni) * kRow);
      fw[ni].c[1] = *reinterpret_cast<const uint4*>(wr2 + w_sub(ni) * kRow);
    }
    load1(f, fstep, fslot, -1);
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      if (mi + 1 < MI) read_x(mi + 1);
#pragma unroll
      for (int u = 0; u < PER; ++u)
        if (mi * PER + u < XI + WI) load1(f, fstep, fslot, mi * PER + u);
      const Frag<KIND_FP8B>& x = fx[mi & 1];
      if constexpr (SCALE == SCALE_F32) {
        float s = __uint_as_float(sx[mi & 1]);
        if constexpr (!DW) s *= sw[0][0];
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) {
          const f32x4 d = mfma_step<KIND_FP8B>(fw[ni], x, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int c = 0; c < 4; ++c)
            acc[mi][ni][c] = __builtin_fmaf(d[c], DW ? s * sw[DW ? ni : 0][c] : s, acc[mi][ni][c]);
        }
      } else {
#pragma unroll
        for (int ni = 0; ni < NI; ++ni)
          acc[mi][ni] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              as_i32x8(fw[ni].c[0], fw[ni].c[1]), as_i32x8(x.c[0], x.c[1]), acc[mi][ni], 0, 0, 0,
              (int)ew[DW ? ni : 0], 0, (int)sx[mi & 1]);
      }
    }
  }

  // Whether every store of the tile is a whole line.
  __device__ __forceinline__ bool whole(const At& p) const {
    return p.rows == BM && p.n0 + BN <= a.N && (a.N & 7) == 0;
  }

  // Eight values at row `row` of the tile, columns n .. n + 7, as far as they exist.
  __device__ __forceinline__ void store8(const At& p, int row, int64_t n, const u32x4& v) const {
    if (row >= p.rows || n >= a.N) return;
    uint16_t* o = static_cast<uint16_t*>(a.out) + (p.out + row) * a.N + n;
    if ((a.N & 7) == 0) {
      __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(o));
    } else if (n + 8 <= a.N) {
      typedef u32x4 u32x4_any __attribute__((aligned(2)));  // rows of any length: at the element's alignment
      *reinterpret_cast<u32x4_any*>(o) = v;
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (n + c < a.N) o[c] = (uint16_t)(v[c / 2] >> (16 * (c & 1)));
    }
  }

  // Rounds and writes the sums.  A lane has row m, n to n + 7 and n + 32 to n + 39 of
  // them; lanes r and r + 8 trade halves and the lanes change places, so that a store
  // writes eight rows of 128 bytes (32 experts' weights' gradients, 537 MB: 255 us
  // with 64 bytes of 16 rows, 200 so).  The stores go past the caches: what reads the
  // output next is another kernel, and it must not push the operands out (8192 x
  // 7168 x 4096 in e8m0: 200 us through the caches, 187 past them).
  __device__ __forceinline__ void store(const At& p, const f32x4 (&acc)[MI][NI]) const {
    const bool lines = whole(p), low = r16 < 8;
    const int from = ((lane & 3) * 16 + (lane >> 3) + 8 * ((lane >> 2) & 1)) * 4;
    const int row = wm * TM + (lane >> 3);
    const int64_t n = p.n0 + wn * 64 + 8 * (lane & 7);
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      u32x4 v[2], first, second;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          v[h][c] = pack2<OELEM>(acc[mi][2 * h + c / 2][2 * (c & 1)], acc[mi][2 * h + c / 2][2 * (c & 1) + 1]);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t give = low ? v[1][c] : v[0][c];
        const uint32_t got = (uint32_t)__builtin_amdgcn_mov_dpp((int)give, 0x128, 0xF, 0xF, true);  // row_ror 8
        first[c] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)(low ? v[0][c] : got));
        second[c] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)(low ? got : v[1][c]));
      }
      if (lines) {
        uint16_t* o = static_cast<uint16_t*>(a.out) + (p.out + row + 16 * mi) * a.N + n;
        __builtin_nontemporal_store(first, reinterpret_cast<u32x4*>(o));
        __builtin_nontemporal_store(second, reinterpret_cast<u32x4*>(o + 8 * a.N));
      } else {
        store8(p, row + 16 * mi, n, first);
        store8(p, row + 16 * mi + 8, n, second);
      }
    }
  }
};

template <class T>
__device__ __forceinline__ void zero(T& acc) {
  for (auto& r : acc)
    for (auto& v : r) v = f32x4{0.f, 0.f, 0.f, 0.f};
}

template <int OELEM, int SCALE, bool DW, bool PLAN>
using Stay = Tiles<OELEM, SCALE, DW, PLAN, 256, 256, 128, 1, 2>;

template <int OELEM, int SCALE, bool DW, bool PLAN>
__global__ void __launch_bounds__((Stay<OELEM, SCALE, DW, PLAN>::THREADS))
k_fp8_stay(Fp8Args a, int mtiles, int ntiles) {
  using C = Stay<OELEM, SCALE, DW, PLAN>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS];
  __shared__ int tab[C::TAB];
  const C c(a, smem, tab, mtiles, ntiles);
  // consecutive tiles on one XCD, which its workgroups walk together
  const int per = (c.total + 7) / 8, here = gridDim.x / 8;
  const int tile0 = (blockIdx.x % 8) * per, tile_end = min(tile0 + per, c.total);
  int tile = tile0 + blockIdx.x / 8;
  if (tile >= tile_end) return;
  f32x4 acc[C::MI][C::NI];
  Source cur, nxt;
  At p, q;
  nxt.steps = 0;
  p = c.place(tile, cur);
  if (cur.steps) c.load(cur, 0, 0);
  int slot = 0;
  bool stores = false;  // a whole tile's stores may be under way
  for (;;) {
    const int after = tile + here;
    const bool more = after < tile_end;
    if (more) q = c.place(after, nxt);
    if (!more) nxt.steps = 0;
    zero(acc);
    for (int i = 0; i < cur.steps; ++i) {
      // the stage has landed (stores behind it may be pending), and every wave
      // is done with the other
      if (stores) wait_vmcnt<2 * C::MI>();
      else wait_vmcnt<0>();
      stores = false;
      lds_barrier();
      // what to request: the next step, or the next tile's first, or no bytes
      const bool end = i + 1 == cur.steps;
      const bool none = end && nxt.steps == 0;
      Source f;
      f.x = end && !none ? nxt.x : cur.x;
      f.w = end && !none ? nxt.w : cur.w;
      f.s = end && !none ? nxt.s : cur.s;
      f.xn = none ? 0 : end ? nxt.xn : cur.xn;
      f.wn = none ? 0 : end ? nxt.wn : cur.wn;
      f.sn = none ? 0 : end ? nxt.sn : cur.sn;
      f.steps = end ? nxt.steps : cur.steps;
      c.add(slot, acc, f, end ? 0 : i + 1, slot ^ 1);
      slot ^= 1;
    }
    if (cur.steps == 0 && nxt.steps) c.load(nxt, 0, slot);  // no step has requested it
    c.store(p, acc);
    asm volatile("" ::: "memory");
    stores = c.whole(p);
    if (!more) break;
    tile = after;
    cur = nxt;
    p = q;
  }
  wait_vmcnt<0>();  // the last step's requests write LDS too
}

template <int OELEM, int SCALE, bool DW, bool PLAN, int BM, int BN, int TM, int KG, int D>
__global__ void __launch_bounds__((Tiles<OELEM, SCALE, DW, PLAN, BM, BN, TM, KG, D>::THREADS))
k_fp8_tile(Fp8Args a, int mtiles, int ntiles) {
  using C = Tiles<OELEM, SCALE, DW, PLAN, BM, BN, TM, KG, D>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS];
  __shared__ int tab[C::TAB];
  const C c(a, smem, tab, mtiles, ntiles);
  const int per = (c.total + 7) / 8, j = blockIdx.x / 8;
  const int tile = (blockIdx.x % 8) * per + j;
  if (j >= per || tile >= c.total) return;
  const int kg = wave_id() / C::NW;
  Source src;
  const At p = c.place(tile, src);
  f32x4 acc[C::MI][C::NI];
  zero(acc);
  // group kg's i-th step is KG i + kg; behind the last, requests of no bytes
  auto source = [&](int i) {
    Source f = src;
    if (i * KG + kg >= src.steps) f.xn = f.wn = f.sn = 0;
    return f;
  };
  const int rounds = (src.steps + KG - 1) / KG;
#pragma unroll
  for (int i = 0; i < D - 1; ++i) c.load(source(i), i * KG + kg, i * KG + kg);
  int slot = 0;
  for (int i = 0; i < rounds; ++i) {
    wait_vmcnt<C::LOADS * (D - 2)>();
    lds_barrier();
    const int ahead = i + D - 1, to = slot == 0 ? D - 1 : slot - 1;
    c.add(slot * KG + kg, acc, source(ahead), ahead * KG + kg, to * KG + kg);
    slot = slot + 1 == D ? 0 : slot + 1;
  }
  wait_vmcnt<0>();  // the last requests write LDS too
  if constexpr (KG > 1) {
    // the groups' sums, added in their order.  (A round behind the last step has
    // added zeros.)
    f32x4* part = reinterpret_cast<f32x4*>(smem);
    lds_barrier();
    if (kg > 0) {
      f32x4* to = part + ((kg - 1) * C::NW + c.wave) * C::MI * C::NI * 64 + c.lane;
#pragma unroll
      for (int mi = 0; mi < C::MI; ++mi)
#pragma unroll
        for (int ni = 0; ni < C::NI; ++ni) to[(mi * C::NI + ni) * 64] = acc[mi][ni];
    }
    __syncthreads();
    if (kg > 0) return;
#pragma unroll
    for (int k = 1; k < KG; ++k) {
      const f32x4* from = part + ((k - 1) * C::NW + c.wave) * C::MI * C::NI * 64 + c.lane;
#pragma unroll
      for (int mi = 0; mi < C::MI; ++mi)
#pragma unroll
        for (int ni = 0; ni < C::NI; ++ni) acc[mi][ni] += from[(mi * C::NI + ni) * 64];
    }
  }
  c.store(p, acc);
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

// CUs of the current device, a multiple of its eight XCDs
int cus() {
  int dev = 0, n = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 8)
    return 256;
  return n / 8 * 8;
}

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to; }

// row tiles of BM rows; of a plan's smaller blocks at most as many as blocks
template <bool DW>
int64_t row_tiles(const Fp8Args& a, int BM) {
  return up(a.M, a.experts && !DW && a.block_m < BM ? a.block_m : BM);
}

// Rows of a plan that are likely in use.  Its buffers have room for a block that is
// not whole with every expert; by shares of equal size, r, an expert has r rows and
// those to its block's end, and at least half a block of them where shares differ.
// (1506 tokens, 21 experts, top-3, blocks of 128, K = 2176, N = 1040: 22.6 us with the
// tiles that this gives, 128 x 128; 29.6 with 256 x 256, which all rows would give.)
int64_t rows_likely(const Fp8Args& a) {
  const int64_t room = (int64_t)a.E * (a.block_m - 1);
  if (a.M <= room + a.E) return a.M;
  const int64_t whole = a.E * up((a.M - room) / a.E, a.block_m) * a.block_m;
  return min(a.M, max(whole, a.M - room / 2));
}

template <int OELEM, int SCALE, bool DW>
void stay_kernel(const Fp8Args& a, hipStream_t stream) {
  const int64_t mt = row_tiles<DW>(a, 256), nt = up(a.N, 256), tiles = mt * nt * (DW ? a.E : 1);
  const int64_t fit = cus(), grid = tiles < fit ? up(tiles, 8) * 8 : fit;
  auto go = [&](auto PLAN) {
    hipLaunchKernelGGL((k_fp8_stay<OELEM, SCALE, DW, PLAN()>), dim3((unsigned)grid),
                       dim3(Stay<OELEM, SCALE, DW, PLAN()>::THREADS), 0, stream, a, (int)mt, (int)nt);
  };
  if (a.experts) go(std::true_type{});
  else go(std::false_type{});
}

template <int OELEM, int SCALE, bool DW, bool PLAN, int BM, int BN, int TM, int KG, int D>
void tile_kernel(const Fp8Args& a, hipStream_t stream) {
  const int64_t mt = row_tiles<DW>(a, BM), nt = up(a.N, BN), tiles = mt * nt * (DW ? a.E : 1);
  hipLaunchKernelGGL((k_fp8_tile<OELEM, SCALE, DW, PLAN, BM, BN, TM, KG, D>), dim3((unsigned)(up(tiles, 8) * 8)),
                     dim3(Tiles<OELEM, SCALE, DW, PLAN, BM, BN, TM, KG, D>::THREADS), 0, stream, a, (int)mt,
                     (int)nt);
}

template <int OELEM, int SCALE, int NT, int MW, int KW>
void rows_kernel(const Fp8Args& a, hipStream_t stream) {
  const int64_t grid = up(a.M, 16 * NT) * up(a.N, 16 * MW);
  hipLaunchKernelGGL((k_fp8_rows<OELEM, SCALE, NT, MW, KW>), dim3((unsigned)grid), dim3(KW * 64), 0, stream, a);
}

// Rows of W a workgroup: 64 where that leaves two workgroups a CU, since each brings
// the rows of X again (64 tokens, 64 experts, top-6, 4096 x 4096, blocks of 16: 181 us
// with 64 rows of W, 213 with 32, 292 with 16), else fewer (one token, 4096 x 7168: 7.7
// us with 16, 10.6 with 32; 16384 x 7168: 23.3 with 16, 22.2 with 32).  Blocks of 32 hold
// twice the sums and run with four waves (256 tokens of the same: 244 us, with eight
// 284).
template <int OELEM, int SCALE, int NT>
void few_rows(const Fp8Args& a, hipStream_t stream) {
  const int64_t mt = up(a.M, 16 * NT), wanted = 2 * cus();
  if (mt * up(a.N, 64) >= wanted) rows_kernel<OELEM, SCALE, NT, 4, NT == 1 ? 8 : 4>(a, stream);
  else if (mt * up(a.N, 32) >= wanted) rows_kernel<OELEM, SCALE, NT, 2, 8>(a, stream);
  else rows_kernel<OELEM, SCALE, NT, 1, 8>(a, stream);
}

// Tiles as large as still fill the CUs: a step of a large tile takes longer, but
// moves fewer bytes for its products.  Dense, K = 7168, N = 4096, fp32 scales, twelve
// layers' weights in turn, us for M = 128 / 512 / 1024 / 2048 / 2304 / 4352 / 8192:
//   64 x 64, two groups of three stages      24 / 41 / 79 / 157 /     /     /
//   64 x 128, two groups of three stages     31 / 30 / 57 / 111 /     /     /
//   128 x 128, two groups of two stages      48 / 46 / 45 /  88 / 111 / 188 / 318
//   128 x 128, one of two (two a CU)         65 / 62 / 60 /  82 / 114 / 179 / 294
//   256 x 256, staying                       93 / 96 / 96 /  94 /  93 / 193 / 220
// A weights' gradient over 8192 rows, us for N x K = 1024 x 1024 / 1024 x 2048 / 2048 x
// 2048 / 2816 x 2816 / 4096 x 4096 / 4352 x 4096, in the same order:
//   22 / 43 / 84 / 167,  32 / 34 / 66 / 128,  46 / 47 / 49 / 96 / 231 / 241,
//   61 / 61 / 62 / 91 / 192 / 244,  119 / 120 / 119 / 119 / 148 / 255
// and over a plan's 8 experts of 1024 rows each, 1024 x 1024 / 2048 x 2048: 42, 30, 22 / 83,
// 17 / 63, 22 / 49.  The plan's forward, 8 experts of 2048 x 4096, blocks of 128, for 512 /
// 1024 / 2048 / 4096 (of 4096 x 4096) tokens, top-2: 31 / 51 / 86 / 334, 28 / 42 / 66 / 242, 26 / 46 /
// 65 / 197, 30 / 39 / 63 / 181, 54 / 54 / 55 / 170.
// The rule counts tiles, not rounds of the CUs: just past a whole round of 256 x 256
// (4352 rows, 4352 x 4096) 128 x 128 is up to 7% faster with fp32 scales, as fast with
// e8m0; 2304 rows of 2048 by 8192 take 61 us with the rule's 256 x 256, 53 with 128 x 128.
template <int OELEM, int SCALE, bool DW, bool PLAN>
void tiles(const Fp8Args& a, hipStream_t stream) {
  const int64_t n = cus(), E = DW ? a.E : 1;
  Fp8Args likely = a;
  if constexpr (PLAN && !DW) likely.M = rows_likely(a);
  auto count = [&](int BM, int BN) { return row_tiles<DW>(likely, BM) * up(a.N, BN) * E; };
  if (count(64, 64) <= n) return tile_kernel<OELEM, SCALE, DW, PLAN, 64, 64, 16, 2, 3>(a, stream);
  if (count(64, 128) <= n) return tile_kernel<OELEM, SCALE, DW, PLAN, 64, 128, 32, 2, 3>(a, stream);
  // blocks of 64 rows: the weights' bytes are the time (512 tokens, 64 experts, top-6,
  // 4096 x 4096: 209 to 214 us; 64 x 64 tiles 252 to 278; of 512 x 4096, 29 and 27)
  if constexpr (PLAN && !DW)
    if (a.block_m == 64) return tile_kernel<OELEM, SCALE, DW, PLAN, 64, 128, 32, 1, 2>(a, stream);
  if (count(128, 128) <= n) return tile_kernel<OELEM, SCALE, DW, PLAN, 128, 128, 64, 2, 2>(a, stream);
  if (count(128, 128) <= 2 * n) return tile_kernel<OELEM, SCALE, DW, PLAN, 128, 128, 32, 1, 2>(a, stream);
  stay_kernel<OELEM, SCALE, DW>(a, stream);
}

}  // namespace

hipError_t launch_fp8_linear(const Fp8Args& a, hipStream_t stream) {
  if (a.M == 0) return hipSuccess;
  by_types(a, [&](auto OELEM, auto SCALE) {
    constexpr int O = OELEM(), S = SCALE();
    const int64_t rows = a.experts ? a.block_m : a.M;
    if (a.dw) {
      if (a.experts) tiles<O, S, true, true>(a, stream);
      else tiles<O, S, true, false>(a, stream);
    } else if (rows <= 16 || (!a.experts && up(a.M, 16) * up(a.N, 16) <= cus())) {
      // also where 16 x 16 pieces do not outnumber the CUs: a tile's LDS and its
      // groups' sums cost more than reading X and W once more (100 rows of 4096 by 512:
      // 6.6 us, tiles 10.0; by 1024, 448 pieces: 11.2 and 10.0).  16 rows of 7168 / 4096 /
      // 2048 by 4096 / 4096 / 8192: 10.9 / 7.1 / 6.8, with 32 rows a workgroup 12.7 / 8.5 /
      // 7.6, tiles 17.9 / 10.0 / 6.8
      few_rows<O, S, 1>(a, stream);
    } else if (rows <= 32) {
      // 17 rows of the same: 12.7 / 8.5 / 7.6, with 16 rows a workgroup 15.3 / 10.0 / 7.8,
      // tiles 17.9 / 10.0 / 6.8; 32 rows: 15.9 / 10.1 / 9.6, tiles 19.1 / 10.0 / 6.7; 33 rows:
      // 21.3 / 13.2 / 9.6 so, tiles 19.3 / 10.0 / 6.7.  (Short K by wide N is the side that
      // loses, up to 3 us.)
      few_rows<O, S, 2>(a, stream);
    } else if (a.experts) {
      tiles<O, S, false, true>(a, stream);
    } else {
      tiles<O, S, false, false>(a, stream);
    }
  });
  return hipGetLastError();
}
