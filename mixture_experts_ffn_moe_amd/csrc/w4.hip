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
//   int4: ((v << 3) & 0x00780078) | 0x41804180 holds 16 + q of two nibbles,
//         exactly.  The group's sum of (16 + q) x minus (16 + z) times the
//         group's sum of x, times s, is the group's part; both sums are fp32, the
//         second one from the same matrix instruction with ones for weights (the
//         vector units are the busier ones; sums taken once, as the tokens are
//         brought into LDS, cost 8 tokens of 4096 x 4096 10.2 us against 9.0).
//         The offset costs about two of fp32's 24 bits: 16 is the smallest one
//         that leaves the four bits of a code in one binade.  128, which saves the
//         shift of every fourth pair, costs five and is no more than 2% faster
//         (one token's FFN 22.7 us against 23.2, 32 tokens of 256 experts 397
//         against 402).
//         With fp16 activations the codes are fp16: 1024 + q in the same way,
//         then 1032 taken off again, exactly, by a packed subtraction.  1024 + q
//         itself, or q 2^-24 as a subnormal, would cost the matrix instruction's
//         sum eight bits more (measured: 2.3e-5 of the result against 3e-6).
//         Two bf16 parts of the activations, the alternative, are twice the matrix
//         instructions and LDS: 32 tokens of 4096 x 8192 51 us against 20.6.
//   e2m1: the hardware's conversion, scale included; e2m1 times a power of
//         two is a bf16, so this is exact too.
// Activations are operands as they are, except fp16 ones with e2m1 (whose scales
// are out of fp16's range): two bf16 parts hi + lo, which is exact.  The FFN's
// intermediate, an fp32 value, is written as three bf16 parts of eight bits each,
// which is exact too, in the order the second product reads.  Its tokens (up to
// eight) have two rows each in one instruction, a second instruction adds the
// third part to both by halves, and the two rows are added at the end: as many
// instructions as two parts would take.
//
// A 16x16x32 matrix instruction takes 16 tokens (A rows) and 16 weight rows (B
// columns); a lane (n = l % 16, g = l / 16) reads 16 bytes of row n in each
// 128-wide step of K: elements 32 g .. 32 g + 31.  Where a scale covers the
// whole step, dword d of the four lane groups feeds instruction d as it is
// (the contraction's order is free as long as the tokens use the same).  Groups
// of 32 and 64 need the elements of one instruction to lie in one group: the
// four dwords of the four lane groups are transposed by lane-row swaps.
//
// A workgroup has 4 waves on the same 16 or 32 weight rows; each takes a run of
// steps of K, D of them requested ahead with one load for the D steps' scales
// (a load of one step's touches 16 rows' lines for two bytes each, and costs the
// address unit as much as the weights'), and the waves' sums are added through
// LDS at the end.  The tokens' part of K lies in LDS, in the order the weights
// need.  Where there are many tiles a workgroup takes several in a row,
// requesting the next one's weights while it ends the last.
//
// Measured at K = 4096, I = 2048, 256 experts, top-6 (kernel times under the
// profiler): 32 tokens in e2m1 take 241 us for the first product (1.21 GB, 5.0
// TB/s) and 123 us for the second (4.9 TB/s); int4 with zero points 277 and 157
// us, its conversion keeping the vector units busy half of the time.  One token in
// int4 takes 14 us (53 MB) and 9 us: the launch, finding the expert and bringing
// the token in are half of that, the loads of all workgroups going out at once.
// Streaming the weights past the caches was slower (366 -> 381 us for the e2m1
// FFN): a line of 128 bytes is read in two steps.
#include <atomic>
#include <type_traits>

#include "device.h"
#include "ops.h"

namespace {

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * 64;
constexpr int kTile = 16;               // tokens of one pass over the weights
constexpr int kUnit = kWaves * 128;     // K elements of one step of every wave
constexpr int kPad = 8;                 // elements behind each token's row in LDS
constexpr int kBlocks = 4;              // 64-route blocks found without a barrier
// LDS of the tokens: a few tokens' whole K, or 1,024 elements of kTile tokens
// (half as many of more parts); and the most that the sums and the list leave.
template <int XE>
constexpr int least_token_lds() {
  return (XE == ELEM_PARTS ? kTile / 2 * 3 : kTile) * (2 * kUnit + kPad) * 2;
}
constexpr int kTokenLdsMost = 144 * 1024;
constexpr int kSumLds = (kWaves - 1) * 2 * 1024;  // the waves' sums of two tiles, at most
constexpr int kCUs = 256, kLds = 160 * 1024;      // of a CU

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// fp16 activations stay fp16 where the codes can be fp16 too.
template <int FMT, int XE>
constexpr bool half_ops() { return FMT == W4_INT && XE == ELEM_F16; }
// Operands of a product for each step of a token, and its rows in LDS.
template <int FMT, int XE>
constexpr int parts() { return XE == ELEM_BF16 || half_ops<FMT, XE>() ? 1 : 2; }
template <int FMT, int XE>
constexpr int lds_rows() { return XE == ELEM_PARTS ? 3 : parts<FMT, XE>(); }

__device__ __forceinline__ float bits_to_f32(uint32_t u16, int elem) {
  return elem == ELEM_F16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)u16)
                          : __uint_as_float(u16 << 16);
}

// The two constants of the int4 conversion, in registers: as literals the
// compiler takes an and and an or for each pair where one v_and_or does.
template <bool HALF>
struct Int4Bits {
  uint32_t mask = HALF ? 0x000F000Fu : 0x00780078u, bias = HALF ? 0x64006400u : 0x41804180u;
  __device__ __forceinline__ Int4Bits() { asm("" : "+s"(mask), "+v"(bias)); }
};

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
template <bool HALF>
using Operand = typename std::conditional<HALF, f16x8, bf16x8>::type;

__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// 8 int4 codes of one dword as bf16 16 + q or fp16 q - 8, in the order 0 4 1 5
// 2 6 3 7.
constexpr float kInt4Offset = 16.f;
template <bool HALF>
__device__ __forceinline__ Operand<HALF> int4_operand(uint32_t v, const Int4Bits<HALF>& c) {
  if constexpr (HALF) {
    const uint4 b = make_uint4((v & c.mask) | c.bias, ((v >> 4) & c.mask) | c.bias,
                               ((v >> 8) & c.mask) | c.bias, ((v >> 12) & c.mask) | c.bias);
    return __builtin_bit_cast(f16x8, b) - (_Float16)1032.f;
  } else {
    return __builtin_bit_cast(
        bf16x8, make_uint4(((v << 3) & c.mask) | c.bias, ((v >> 1) & c.mask) | c.bias,
                           ((v >> 5) & c.mask) | c.bias, ((v >> 9) & c.mask) | c.bias));
  }
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

// 8 consecutive activations of a lane: one 16-byte load, or one of each part.
template <int XE>
struct X8 {
  uint4 v[XE == ELEM_PARTS ? 3 : 1];
};

// From k of a row of K.
template <int XE>
__device__ __forceinline__ void load_tokens(X8<XE>& x, __amdgpu_buffer_rsrc_t r, uint32_t k,
                                            uint32_t K) {
  x.v[0] = buf_load16(r, k < K ? k * 2 : 0xFFFFFFF0u, 0);  // zeros past K
  if constexpr (XE == ELEM_PARTS) {
    x.v[1] = buf_load16(r, k < K ? (K + k) * 2 : 0xFFFFFFF0u, 0);
    x.v[2] = buf_load16(r, k < K ? (2 * K + k) * 2 : 0xFFFFFFF0u, 0);
  }
}

// The three parts of v that each lose nothing: v = p[0] + p[1] + 2 p[2], eight
// bits a part (the last one halved, see above; below 2^-133 bits go).  An infinity
// or NaN is whole in the first.
__device__ __forceinline__ void split_parts(float v, uint16_t (&p)[3]) {
  const uint32_t hi = __float_as_uint(v) & 0xFFFF0000u;
  const float r = __builtin_isfinite(v) ? v - __uint_as_float(hi) : 0.f;
  const uint32_t mid = __float_as_uint(r) & 0xFFFF0000u;
  p[0] = (uint16_t)(hi >> 16);
  p[1] = (uint16_t)(mid >> 16);
  p[2] = (uint16_t)(__float_as_uint(0.5f * (r - __uint_as_float(mid))) >> 16);
}

// The place of element i of a row in the order that the weights' codes come in:
// in each eight 0 4 1 5 2 6 3 7 for int4.
template <int FMT>
__device__ __forceinline__ int place_of(int i) {
  return FMT == W4_MX ? i : (i & ~7) | (i & 3) << 1 | (i >> 2 & 1);
}

__device__ __forceinline__ uint32_t lo_halves(uint32_t a, uint32_t b) { return (a & 0xFFFFu) | b << 16; }
__device__ __forceinline__ uint32_t hi_halves(uint32_t a, uint32_t b) { return a >> 16 | (b & 0xFFFF0000u); }

// Lanes of a 16-lane row that hold one scale group's 8-element shares (GM groups
// in the row's 128 elements): every lane gets their sum.
template <int GM>
__device__ __forceinline__ float group_sum(float v) {
  v = add_dpp<0xB1>(v);                         // neighbours
  v = add_dpp<0x4E>(v);                         // quads
  if constexpr (GM <= 2) v = add_dpp<0x141>(v);  // the half row's other quad
  if constexpr (GM == 1) v = add_dpp<0x140>(v);  // the row's other half
  return v;
}

__device__ __forceinline__ float pair_sum(uint32_t d) {
  return __uint_as_float(d << 16) + __uint_as_float(d & 0xFFFF0000u);
}

// 8 activations into LDS as bf16 in that order, each part `part` elements after
// the one before.  Returns their sum (int4 with bf16 operands; in fp32 as every sum
// here).
template <int FMT, int XE>
__device__ __forceinline__ float store_tokens(const X8<XE>& x, uint16_t* to, int part) {
  const uint32_t d[4] = {x.v[0].x, x.v[0].y, x.v[0].z, x.v[0].w};
  uint32_t b[3][4];  // pairs of elements
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    b[0][i] = d[i], b[1][i] = 0;
    if constexpr (XE == ELEM_F16 && !half_ops<FMT, XE>()) {
      const float f = bits_to_f32(d[i] & 0xFFFFu, ELEM_F16), h = bits_to_f32(d[i] >> 16, ELEM_F16);
      const uint32_t f0 = f32_to_bf16(f), h0 = f32_to_bf16(h);
      b[0][i] = f0 | h0 << 16;
      b[1][i] = (uint32_t)f32_to_bf16(f - __uint_as_float(f0 << 16)) |
                (uint32_t)f32_to_bf16(h - __uint_as_float(h0 << 16)) << 16;
    }
  }
  if constexpr (XE == ELEM_PARTS) {  // in order already
    b[1][0] = x.v[1].x, b[1][1] = x.v[1].y, b[1][2] = x.v[1].z, b[1][3] = x.v[1].w;
    b[2][0] = x.v[2].x, b[2][1] = x.v[2].y, b[2][2] = x.v[2].z, b[2][3] = x.v[2].w;
  }
  float sum = 0.f;
#pragma unroll
  for (int p = 0; p < lds_rows<FMT, XE>(); ++p) {
    uint4 v = make_uint4(b[p][0], b[p][1], b[p][2], b[p][3]);
    if constexpr (FMT != W4_MX && XE != ELEM_PARTS)
      v = make_uint4(lo_halves(b[p][0], b[p][2]), hi_halves(b[p][0], b[p][2]),
                     lo_halves(b[p][1], b[p][3]), hi_halves(b[p][1], b[p][3]));
    *reinterpret_cast<uint4*>(to + p * part) = v;
    if constexpr (FMT != W4_MX && !half_ops<FMT, XE>())
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += (p == 2 ? 2.f : 1.f) * pair_sum(b[p][i]);
  }
  return sum;
}

__device__ __forceinline__ void store_out(void* out, size_t at, float v, int elem) {
  if (elem == ELEM_F32) static_cast<float*>(out)[at] = v;
  else if (elem == ELEM_F16) static_cast<_Float16*>(out)[at] = (_Float16)v;
  else static_cast<uint16_t*>(out)[at] = f32_to_bf16(v);
}

// BYTES consecutive bytes of a table, as dwords.  RAG: at any address, from the
// dwords that cover them (a dword with a byte of the table in it can be read
// whole; one behind the buffer's end reads 0).
template <int BYTES, bool RAG>
struct Window {
  static constexpr int N = (BYTES + 3) / 4;
  uint32_t d[N + RAG];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int off, int soff) {
    const int at = RAG ? off & ~3 : off;
    constexpr int M = N + RAG;
    int i = 0;
#pragma unroll
    for (; i + 4 <= M; i += 4) {
      const uint4 v = buf_load16(r, (uint32_t)at + 4 * i, soff);
      d[i] = v.x, d[i + 1] = v.y, d[i + 2] = v.z, d[i + 3] = v.w;
    }
    if constexpr (M % 4 >= 2) {
      const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(r, at + 4 * (M / 4 * 4), soff, 0);
      d[M / 4 * 4] = v[0], d[M / 4 * 4 + 1] = v[1];
    }
    if constexpr (M % 2 == 1) d[M - 1] = __builtin_amdgcn_raw_buffer_load_b32(r, at + 4 * (M - 1), soff, 0);
  }
  __device__ __forceinline__ void align(int off) {
    if constexpr (RAG) {
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = __builtin_amdgcn_alignbyte(d[i + 1], d[i], off & 3);
    }
  }
  __device__ __forceinline__ uint32_t u16(int i) const { return d[i / 2] >> (16 * (i % 2)) & 0xFFFFu; }
  __device__ __forceinline__ uint32_t u8(int i) const { return d[i / 4] >> (8 * (i % 4)) & 0xFFu; }
};

// A buffer over `bytes` bytes from any address: its base is the dword that holds
// the first, `skip` bytes further.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t dword_rsrc(const uint8_t* p, uint32_t bytes,
                                                             int& skip) {
  skip = (int)(reinterpret_cast<uintptr_t>(p) & 3);
  return make_rsrc(p - skip, bytes ? (bytes + skip + 3) & ~3u : 0);
}

// The table's scales of a row in a step, and their bytes.
template <int FMT, int GM>
constexpr int step_scales() { return FMT == W4_MX ? 4 : GM; }
template <int FMT>
constexpr int scale_bytes() { return FMT == W4_MX ? 1 : 2; }

// Zero points of D steps: two are no whole dword, so they can lie anywhere too.
template <int D, int GM, bool RAG>
using ZeroWindow = Window<D * GM, RAG || D * GM % 4 != 0>;
template <int FMT, int D, int GM, bool RAG>
using ScaleWindow = Window<D * step_scales<FMT, GM>() * scale_bytes<FMT>(), RAG>;

// acc[t] += tokens x weights of one 128-wide step, the u-th of its window.
// xp: the lane's row at this step in LDS, its P operands `part` elements apart.
// valid: the scale groups of the step that the row has (RAG).  ONE: the product's
// first four rows add up to one token, whose sum over group q of the step is
// sx[q]; int4 adds them here, into the first.  SE: type of int4 scales.
template <int FMT, int GM, bool RAG, int P, int NT, int D, bool ONE, int SE, bool HALF>
__device__ __forceinline__ void step_product(f32x4 (&acc)[NT], const uint16_t* xp, int part,
                                             const float* sx,
                                             const uint4 (&wq)[NT],
                                             const ScaleWindow<FMT, D, GM, RAG> (&sc)[NT],
                                             const ZeroWindow<D, GM, RAG> (&zc)[NT], int u,
                                             int valid, bool one_scale, float z0,
                                             const Int4Bits<HALF>& bits) {
  const int g = (threadIdx.x & 63) >> 4;
  Operand<HALF> xf[P][4];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int d = 0; d < 4; ++d)
      xf[p][d] = *reinterpret_cast<const Operand<HALF>*>(
          xp + p * part + (GM == 1 ? 32 * g + 8 * d : 32 * d + 8 * g));
  if constexpr (FMT == W4_MX) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      // 2^(c - 127) as a float: c in the exponent field, 0 subnormal, 255 NaN;
      // past the row's end 0, as the tokens there
      const uint32_t c = sc[t].d[u] >> (8 * g) & 0xFFu;
      float s = __uint_as_float(c == 255 ? 0x7FC00000u : c ? c << 23 : 0x00400000u);
      if (RAG && g >= valid) s = 0.f;
      const uint32_t q[4] = {wq[t].x, wq[t].y, wq[t].z, wq[t].w};
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const bf16x8 b = e2m1_to_bf16(q[d], s);
#pragma unroll
        for (int p = 0; p < P; ++p)
          acc[t] = mma(xf[p][d], b, acc[t]);
      }
    }
  } else {
    constexpr int DG = 4 / GM;  // instructions of one group
    [[maybe_unused]] f32x4 xsum[GM];
    if constexpr (!ONE) {
      constexpr uint32_t one = HALF ? 0x3C003C00u : 0x3F803F80u;
      const auto ones = __builtin_bit_cast(Operand<HALF>, make_uint4(one, one, one, one));
#pragma unroll
      for (int q = 0; q < GM; ++q) {
        xsum[q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int d = q * DG; d < (q + 1) * DG; ++d)
#pragma unroll
          for (int p = 0; p < P; ++p)
            xsum[q] = mma(xf[p][d], ones, xsum[q]);
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      uint4 w = wq[t];
      if constexpr (GM > 1) transpose4(w);
      const uint32_t q4[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int q = 0; q < GM; ++q) {
        f32x4 v = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int d = q * DG; d < (q + 1) * DG; ++d) {
          const Operand<HALF> b = int4_operand<HALF>(q4[d], bits);
#pragma unroll
          for (int p = 0; p < P; ++p)
            v = mma(xf[p][d], b, v);
        }
        // a row of one scale has a window of its own (RAG)
        const int k = u * GM + q;
        float s = bits_to_f32(RAG && one_scale ? sc[t].u16(0) : sc[t].u16(k), SE);
        const float z = z0 + (float)(RAG && one_scale ? zc[t].u8(0) : zc[t].u8(k));
        if (RAG && !one_scale && q >= valid) s = 0.f;  // past the row's end
        if constexpr (ONE) {
          acc[t][0] += s * ((v[0] + v[1]) + (v[2] + v[3]) - z * sx[q]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[t][j] += s * (v[j] - z * xsum[q][j]);
        }
      }
    }
  }
}

constexpr int kNone = (int)0x80000000;  // past every buffer

// Lanes of a wave that hold sums (a token of three parts has two rows, the second
// one in the upper half), and the LDS for the sums of all waves but the first.
template <int XE>
constexpr int sum_lanes() { return XE == ELEM_PARTS ? 32 : 64; }
template <int XE, int NT>
constexpr int sum_lds() { return (kWaves - 1) * NT * sum_lanes<XE>() * 16; }

// The bound on waves keeps every instantiation out of scratch memory, whose
// accesses the waits for the requested steps would count too.
// GM: scale groups in a 128-wide step (int4: 1, 2, 4).  RAG: K is no multiple of
// 512 or a row has one scale, so that the scales of D steps lie at any address,
// and a row may end inside a step.  NT: 16-row weight tiles taken together; with
// SWIGLU the gate's and the up's.  D: steps a wave requests ahead.  SE: type of
// int4 scales.
// Grid: x the first of `run` output tiles; y the route whose expert to take (R
// <= E; only the expert's first route works), the expert (R > E; y = E: the
// routes without an expert here), or the block of `tile` tokens (no ids).
template <int FMT, int XE, int SE, int GM, bool RAG, int NT, bool SWIGLU, int D>
__global__ void
__launch_bounds__(kThreads, XE == ELEM_PARTS ? (RAG && GM == 4 ? 2 : 3)
                            : GM > 1 ? 2
                            : NT == 2 && D == 4 && (RAG || parts<FMT, XE>() == 2) ? 3 : 4)
k_w4(W4Args a, int tile, int run, int token_lds) {
  constexpr int P = parts<FMT, XE>(), PR = lds_rows<FMT, XE>();
  constexpr bool HALF = half_ops<FMT, XE>();
  constexpr int kRowParts = XE == ELEM_PARTS ? 3 : 1;  // 16-bit rows of a token in memory
  constexpr int kSumLanes = sum_lanes<XE>();
  extern __shared__ __align__(16) uint8_t smem[];
  uint16_t* xs = reinterpret_cast<uint16_t*>(smem);
  float* red = reinterpret_cast<float*>(smem + token_lds);  // waves 1.. of each tile
  uint16_t* list = reinterpret_cast<uint16_t*>(smem + token_lds + sum_lds<XE, NT>());
  __shared__ int wave_count[kWaves];

  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  const int n16 = lane & 15, g = lane >> 4;
  const int out_n = SWIGLU ? a.N / 2 : a.N;
  constexpr int kCols = SWIGLU ? 16 : 16 * NT;
  const int tiles = (out_n + kCols - 1) / kCols;
  const int tile0 = blockIdx.x * run, tile1 = min(tiles, tile0 + run);

  // the workgroup's expert and the routes it works on
  int e = 0, count, first = 0, lead = -1;  // lead: the first of them
  const bool few = a.ids && a.R <= 64 * kBlocks;  // found by every wave alone
  if (!a.ids) {
    first = blockIdx.y * tile;
    count = min(tile, a.R - first);
  } else {
    const int y = blockIdx.y;
    e = a.R <= a.E ? a.ids[y] : y < a.E ? y : -1;
    if ((unsigned)e >= (unsigned)a.E) e = -1;
    count = 0;
    if (few) {
      int id[kBlocks];
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) id[b] = a.ids[min(64 * b + lane, a.R - 1)];
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        const bool valid = (unsigned)id[b] < (unsigned)a.E;
        const unsigned long long m =
            __ballot(64 * b + lane < a.R && (valid ? id[b] : -1) == e);
        if (lead < 0 && m) lead = 64 * b + __ffsll(m) - 1;
        if (wave == 0 && (m >> lane & 1))
          list[count + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)(64 * b + lane);
        count += __popcll(m);
      }
    } else {
      for (int base = 0; base < a.R; base += kThreads) {
        int id = -2;
        if (base + tid < a.R) {
          id = a.ids[base + tid];
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
        if (id == e) list[at + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)(base + tid);
        __syncthreads();
      }
      if (count) lead = list[0];
    }
    if (count == 0 || (a.R <= a.E && lead != y)) return;
    if (e < 0) {  // routes without an expert here: zeros (parts are not read)
      if (a.oelem == ELEM_PARTS) return;
      if (few) __syncthreads();
      const int c0 = tile0 * kCols, w = min(out_n, tile1 * kCols) - c0;
      for (int i = tid; i < count * w; i += kThreads)
        store_out(a.out, (size_t)list[i / w] * out_n + c0 + i % w, 0.f, a.oelem);
      return;
    }
  }
  // the m-th of them, m wave-uniform
  if (few && count > 1) __syncthreads();
  auto route = [&](int m) -> int {
    if (!a.ids) return first + m;
    return count == 1 ? lead : __builtin_amdgcn_readfirstlane((int)list[m]);
  };

  const int KS = (a.K + 127) / 128, KG = a.K / a.group;
  const int J = (KS + kWaves - 1) / kWaves, JP = (J + D - 1) / D * D;  // steps of a wave
  const uint32_t pitch = (uint32_t)a.K / 2;
  const __amdgpu_buffer_rsrc_t rw =
      make_rsrc(a.w + (size_t)e * a.N * pitch, (uint32_t)a.N * pitch);
  constexpr int SB = scale_bytes<FMT>(), SG = step_scales<FMT, GM>();
  int skip_s, skip_z;
  const __amdgpu_buffer_rsrc_t rs =
      dword_rsrc(static_cast<const uint8_t*>(a.scale) + (size_t)e * a.N * KG * SB,
                 (uint32_t)a.N * KG * SB, skip_s);
  const bool has_zero = FMT == W4_INT && a.zero;
  const __amdgpu_buffer_rsrc_t rz = dword_rsrc(has_zero ? a.zero + (size_t)e * a.N * KG : a.w,
                                               has_zero ? (uint32_t)a.N * KG : 0, skip_z);
  const float z0 = (HALF ? -8.f : kInt4Offset) + (has_zero ? 0.f : 8.f);  // an empty buffer's loads read 0
  const bool one_scale = GM == 1 && FMT == W4_INT && KG == 1;  // of the whole row

  for (int m0 = 0; m0 < count; m0 += tile) {
    const int nt = min(tile, count - m0);
    // steps of each wave in one part of K: what the LDS holds for nt tokens
    const int fit = (token_lds / (PR * nt * 2) - kPad) / kUnit;
    const bool whole = D > 2 || fit >= JP;  // many steps ahead only where K fits
    const int S = whole ? JP : fit / D * D;  // fit >= D: the launch sees to it
    const int xrow = S * kUnit + kPad, inv_s = 65536 / S + 1;  // seg * inv_s >> 16 = seg / S
    // the lane's row, and its second operand behind it; of three parts the first
    // two are rows n16 and n16 + 8, the third is the second operand of both
    const int lt = XE == ELEM_PARTS ? n16 & 7 : n16, lp = XE == ELEM_PARTS ? n16 >> 3 : 0;
    const uint16_t* xa = xs + (size_t)(lp * nt + (lt < nt ? lt : 0)) * xrow;
    const int part = (XE == ELEM_PARTS ? 2 - lp : 1) * nt * xrow;

    // Requests run D steps ahead of the products (the scales of a round of D
    // steps a round ahead of its weights), over the parts of K and the tiles in
    // order.  All are unconditional, so that the waits count them exactly: past
    // the last tile the rows lie outside the buffers (the loads return zeros and
    // touch no memory), past the last step the last one is read again.
    uint4 wq[D][NT];
    ScaleWindow<FMT, D, GM, RAG> sn[NT], sc[NT];  // the next round's scales, this one's
    ZeroWindow<D, GM, RAG> zn[NT], zc[NT];
    constexpr bool ZRAG = RAG || D * GM % 4 != 0;
    // the places of a tile's rows (an up row's follows from the gate's, a zero
    // point's from its scale's: registers are short)
    constexpr int NR = SWIGLU ? 1 : NT;
    int wrow[NR], srow[NR];
    auto weight_row = [&](int t0, int t) {
      return SWIGLU ? min(t0 * 16 + n16, out_n - 1) : min((t0 * NT + t) * 16 + n16, a.N - 1);
    };
    const int up_rows = SWIGLU ? out_n : 0;
    // a position in the walk: tile, part of K, round's first step in the part
    struct Pos {
      int tile, part, i;
    };
    Pos pw{tile0, 0, 0}, ps{tile0, 0, 0};
    auto next_round = [&](Pos& p) {
      p.i += D;
      if (p.i < S) return false;
      p.i = 0;
      p.part += S * kWaves;
      if (p.part < KS) return false;
      p.part = 0;
      ++p.tile;
      return true;
    };
    auto weight_rows = [&] {
#pragma unroll
      for (int t = 0; t < NR; ++t)
        wrow[t] = pw.tile < tile1 ? (int)((uint32_t)weight_row(pw.tile, t) * pitch + 16 * g) : kNone;
    };
    auto scale_rows = [&] {
#pragma unroll
      for (int t = 0; t < NR; ++t) {
        const int n = weight_row(ps.tile, t) * KG;
        srow[t] = ps.tile < tile1 ? n * SB + skip_s : kNone;
      }
    };
    auto weights_request = [&](int u) {
      const int step = min(pw.part + wave * S + pw.i + u, KS - 1);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        // where a row may end inside a step, the whole offset is the one that the
        // range check sees
        const int row = wrow[t % NR];
        const uint32_t at = (RAG && row != kNone ? row + step * 64 : row) + t * up_rows * pitch;
        wq[u][t] = buf_load16(rw, at, RAG ? 0 : (uint32_t)step * 64);
      }
    };
    auto scale_step = [&](const Pos& p) {
      const int step = p.part + wave * S + p.i;
      return one_scale ? 0 : step < KS ? step : 0;
    };
    int salign[NT], zalign[NT];  // the windows' bytes inside their first dword
    auto scales_request = [&] {
      const int c = scale_step(ps) * SG;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int row = srow[t % NR];
        const bool on = row != kNone;
        const int srow_t = on ? row + t * up_rows * KG * SB : kNone;
        const int so = RAG && on ? srow_t + c * SB : srow_t;
        const int zrow = on ? (srow_t - skip_s) / SB + skip_z : kNone;
        const int zo = ZRAG && on ? zrow + c : zrow;
        sn[t].load(rs, so, RAG ? 0 : c * SB);
        if constexpr (FMT == W4_INT) zn[t].load(rz, zo, ZRAG ? 0 : c);
        salign[t] = so;
        zalign[t] = zo;
      }
      if (next_round(ps)) scale_rows();
    };
    auto scales_take = [&] {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        sc[t] = sn[t];
        sc[t].align(salign[t]);
        if constexpr (FMT == W4_INT) {
          zc[t] = zn[t];
          zc[t].align(zalign[t]);
        }
      }
    };

    // tokens' elements in segments of 512, one a wave at a time, kAhead of them (a
    // few loads either way) requested together
    constexpr int kAhead = XE == ELEM_PARTS ? 1 : 2;
    X8<XE> xr[kAhead];
    auto seg_request = [&](X8<XE>& x, int seg, int k0) {
      const int m = seg * inv_s >> 16;
      const bool on = m < nt;  // else an empty buffer
      const uint32_t r = on ? route(m0 + m) : 0;
      const size_t row = a.x_per_route || a.top_k == 1 ? r : __umulhi(r, a.inv_top_k);
      const __amdgpu_buffer_rsrc_t rx =
          make_rsrc(static_cast<const uint16_t*>(a.x) + row * a.K * kRowParts,
                    on ? (uint32_t)a.K * kRowParts * 2 : 0);
      load_tokens<XE>(x, rx, k0 + (seg - m * S) * kUnit + lane * 8, a.K);
    };
    auto seg_store = [&](const X8<XE>& x, int seg) {
      const int m = seg * inv_s >> 16;
      if (m >= nt) return;
      store_tokens<FMT, XE>(x, xs + (size_t)m * xrow + (seg - m * S) * kUnit + lane * 8, nt * xrow);
    };
    auto stage = [&](int k0, bool begun) {
      const int segs = nt * S;
      for (int seg = wave; seg < segs; seg += kAhead * kWaves) {
        if (!begun) {
#pragma unroll
          for (int i = 0; i < kAhead; ++i) seg_request(xr[i], seg + i * kWaves, k0);
        }
        begun = false;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) seg_store(xr[i], seg + i * kWaves);
      }
    };

    f32x4 acc[NT];
    const Int4Bits<HALF> bits;

    // the tokens' loads go first: loads return in order, so they are waited for
    // while the weights are still on their way
#pragma unroll
    for (int i = 0; i < kAhead; ++i) seg_request(xr[i], wave + i * kWaves, 0);
    scale_rows();
    scales_request();
    weight_rows();
#pragma unroll
    for (int u = 0; u < D; ++u) weights_request(u);
    if (next_round(pw)) weight_rows();
    if (m0) __syncthreads();  // the earlier tokens are read
    stage(0, true);
    __syncthreads();

    for (int ti = tile0; ti < tile1; ++ti) {
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int k0 = 0; k0 < KS; k0 += S * kWaves) {  // a part of K
        if (!whole && (k0 || ti > tile0)) {
          __syncthreads();
          stage(k0 * 128, false);
          __syncthreads();
        }
        for (int i = 0; i < S; i += D) {
          scales_take();
          scales_request();
#pragma unroll
          for (int u = 0; u < D; ++u) {
            const int step = k0 + wave * S + i + u;
            if (step < KS)
              step_product<FMT, GM, RAG, P, NT, D, false, SE, HALF>(
                  acc, xa + (wave * S + i + u) * 128, part, nullptr, wq[u], sc, zc, u,
                  KG - step * SG, one_scale, z0, bits);
            weights_request(u);
          }
          if (next_round(pw)) weight_rows();
        }
      }
      if constexpr (XE == ELEM_PARTS)  // a token's two rows
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t v = __float_as_uint(acc[t][j]);
            const u32x2 h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
            acc[t][j] = __uint_as_float(h[0]) + __uint_as_float(h[1]);
          }
      // the waves' sums: the others' through LDS to the first, which writes
      if (wave) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
          if (4 * g < nt)
            *reinterpret_cast<f32x4*>(red + (((wave - 1) * NT + t) * kSumLanes + lane) * 4) = acc[t];
      }
      __syncthreads();
      if (wave == 0 && 4 * g < nt) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int v = 0; v < kWaves - 1; ++v)
            acc[t] += *reinterpret_cast<const f32x4*>(red + ((v * NT + t) * kSumLanes + lane) * 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int m = 4 * g + j;
          if (m >= nt) break;
          const int r = a.ids ? list[m0 + m] : first + m0 + m;
          const size_t at = (size_t)r * out_n + ti * kCols + n16;
          if constexpr (SWIGLU) {
            const float v = swiglu(acc[0][j], acc[NT - 1][j]);
            const int n = ti * 16 + n16;
            if (n >= out_n) continue;
            if (a.oelem == ELEM_PARTS) {
              uint16_t* row = static_cast<uint16_t*>(a.out) + (size_t)r * out_n * 3 + place_of<FMT>(n);
              uint16_t p[3];
              split_parts(v, p);
#pragma unroll
              for (int i = 0; i < 3; ++i) row[(size_t)i * out_n] = p[i];
            } else {
              store_out(a.out, at, v, a.oelem);
            }
          } else {
#pragma unroll
            for (int t = 0; t < NT; ++t)
              if (ti * kCols + 16 * t + n16 < out_n) store_out(a.out, at + 16 * t, acc[t][j], a.oelem);
          }
        }
      }
      if (ti + 1 < tile1) __syncthreads();
    }
  }
}

// The second product and the weighted sum of a token at once: a workgroup has
// 16 output columns of a token, and each wave one of the token's routes at a
// time, over the whole of K.  Nothing goes through memory between the product
// and the sum, and there is one launch less; an expert that two tokens chose is
// read twice.  x (R, 3, K) in three parts: the product's first rows are those of
// the token (the halved third one twice), so that one instruction does for all of
// them.  Grid: x the columns, y the token.
constexpr int kTokenWaves = 8;   // routes at once
constexpr int kTokenPart = 2048; // K elements of a route in LDS at a time
// elements from a part's row to the next: 80 bytes past the row, so that the three
// parts' 16 bytes of the four lane groups (64 or 16 bytes apart) lie in different banks
constexpr int kTokenRow = kTokenPart + 40;
template <int FMT, int GM>
constexpr int token_lds() {
  return 3 * kTokenRow * 2 + (FMT == W4_INT ? kTokenPart / 128 * GM * 4 : 0);
}

template <int FMT, int SE, int GM, bool RAG>
__global__ void __launch_bounds__(kTokenWaves * 64, 2)
k_w4_token(W4Args a, const float* __restrict__ weights) {
  constexpr int D = 8, SB = scale_bytes<FMT>(), SG = step_scales<FMT, GM>();
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 63, wave = wave_id(), waves = blockDim.x / 64;
  const int n16 = lane & 15, g = lane >> 4;
  const int t = blockIdx.y, n = min((int)blockIdx.x * 16 + n16, a.N - 1);
  uint16_t* xs = reinterpret_cast<uint16_t*>(smem + (size_t)wave * token_lds<FMT, GM>());
  const uint16_t* xa = xs + min(n16, 2) * kTokenRow;
  float* sums = reinterpret_cast<float*>(xs + 3 * kTokenRow);  // of the scale groups
  const int KS = (a.K + 127) / 128, KG = a.K / a.group;
  const uint32_t pitch = (uint32_t)a.K / 2;
  const bool has_zero = FMT == W4_INT && a.zero;
  const float z0 = kInt4Offset + (has_zero ? 0.f : 8.f);
  const bool one_scale = GM == 1 && FMT == W4_INT && KG == 1;
  const Int4Bits<false> bits;
  float sum = 0.f;

  for (int q = wave; q < a.top_k; q += waves) {
    const int r = t * a.top_k + q;
    const int e = a.ids[r];
    if ((unsigned)e >= (unsigned)a.E) continue;
    const __amdgpu_buffer_rsrc_t rx =
        make_rsrc(static_cast<const uint16_t*>(a.x) + (size_t)r * a.K * 3, (uint32_t)a.K * 6);
    const __amdgpu_buffer_rsrc_t rw =
        make_rsrc(a.w + (size_t)e * a.N * pitch, (uint32_t)a.N * pitch);
    int skip_s, skip_z;
    const __amdgpu_buffer_rsrc_t rs =
        dword_rsrc(static_cast<const uint8_t*>(a.scale) + (size_t)e * a.N * KG * SB,
                   (uint32_t)a.N * KG * SB, skip_s);
    const __amdgpu_buffer_rsrc_t rz = dword_rsrc(has_zero ? a.zero + (size_t)e * a.N * KG : a.w,
                                                 has_zero ? (uint32_t)a.N * KG : 0, skip_z);
    const int wrow = (int)((uint32_t)n * pitch + 16 * g);
    const int srow = n * KG * SB + skip_s, zrow = n * KG + skip_z;

    uint4 wq[D][1];
    ScaleWindow<FMT, D, GM, RAG> sn[1], sc[1];
    ZeroWindow<D, GM, RAG> zn[1], zc[1];
    int salign = 0, zalign = 0;
    auto weights_request = [&](int u, int step) {  // past the end the last one again
      step = min(step, KS - 1);
      wq[u][0] = buf_load16(rw, (uint32_t)(RAG ? wrow + step * 64 : wrow),
                            RAG ? 0 : (uint32_t)step * 64);
    };
    auto scales_request = [&](int step) {
      const int c = (one_scale || step >= KS ? 0 : step) * SG;
      salign = RAG ? srow + c * SB : srow;
      zalign = RAG ? zrow + c : zrow;
      sn[0].load(rs, salign, RAG ? 0 : c * SB);
      if constexpr (FMT == W4_INT) zn[0].load(rz, zalign, RAG ? 0 : c);
    };
    f32x4 acc[1] = {{0.f, 0.f, 0.f, 0.f}};
    for (int k0 = 0; k0 < a.K; k0 += kTokenPart) {
      X8<ELEM_PARTS> xr[kTokenPart / 512];
#pragma unroll
      for (int i = 0; i < kTokenPart / 512; ++i)
        load_tokens<ELEM_PARTS>(xr[i], rx, k0 + i * 512 + lane * 8, a.K);
      if (k0 == 0) {
        scales_request(0);
#pragma unroll
        for (int u = 0; u < D; ++u) weights_request(u, u);
      }
#pragma unroll
      for (int i = 0; i < kTokenPart / 512; ++i)
      {
        float v = store_tokens<FMT, ELEM_PARTS>(xr[i], xs + i * 512 + lane * 8, kTokenRow);
        if constexpr (FMT == W4_INT) {
          v = group_sum<GM>(v);
          if (lane % (16 / GM) == 0) sums[(i * 512 + lane * 8) / (128 / GM)] = v;
        }
      }
      wave_lds_fence();  // the wave's own LDS
      const int end = min(KS, (k0 + kTokenPart) / 128);
      for (int s0 = k0 / 128; s0 < end; s0 += D) {
        sc[0] = sn[0];
        sc[0].align(salign);
        if constexpr (FMT == W4_INT) {
          zc[0] = zn[0];
          zc[0].align(zalign);
        }
        scales_request(s0 + D);
#pragma unroll
        for (int u = 0; u < D; ++u) {
          if (s0 + u < KS)
            step_product<FMT, GM, RAG, 1, 1, D, true, SE, false>(
                acc, xa + (s0 + u) * 128 - k0, 0, sums + ((s0 + u) - k0 / 128) * GM, wq[u], sc,
                zc, u, KG - (s0 + u) * SG, one_scale, z0, bits);
          weights_request(u, s0 + u + D);
        }
      }
      wave_lds_fence();
    }
    sum += weights[r] * (FMT == W4_MX ? (acc[0][0] + acc[0][1]) + (acc[0][2] + acc[0][3]) : acc[0][0]);
  }
  float* red = reinterpret_cast<float*>(smem);
  __syncthreads();  // the tokens are read
  if (g == 0) red[wave * 16 + n16] = sum;
  __syncthreads();
  const int c = blockIdx.x * 16 + threadIdx.x;
  if (threadIdx.x < 16 && c < a.N) {
    float v = 0.f;
    for (int w = 0; w < waves; ++w) v += red[w * 16 + threadIdx.x];
    store_out(a.out, (size_t)t * a.N + c, v, a.oelem);
  }
}

constexpr int kCombineThreads = 256;

// out[t] = the sum of w[r] y[r]; eight routes' ids, weights and rows are
// requested before any is added.
__global__ void __launch_bounds__(kCombineThreads)
k_w4_combine(const float* __restrict__ y, const int32_t* __restrict__ ids,
             const float* __restrict__ w, void* __restrict__ out, int oelem, int top_k, int K,
             int E) {
  constexpr int kBatch = 8;
  const int t = blockIdx.y, c = (blockIdx.x * kCombineThreads + threadIdx.x) * 4;
  if (c >= K) return;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < top_k; j0 += kBatch) {
    int id[kBatch];
    float wr[kBatch];
    f32x4 v[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int r = t * top_k + min(j0 + u, top_k - 1);
      id[u] = ids[r];
      wr[u] = w[r];
      v[u] = *reinterpret_cast<const f32x4*>(y + (size_t)r * K + c);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (j0 + u < top_k && (unsigned)id[u] < (unsigned)E) s += wr[u] * v[u];
  }
  const size_t at = (size_t)t * K + c;
#pragma unroll
  for (int i = 0; i < 4; ++i) store_out(out, at + i, s[i], oelem);
}

// Lets Kernel have `bytes` of dynamic LDS past the default limit of 64 KiB: once
// on each device.
template <auto* Kernel>
hipError_t allow_lds(int bytes) {
  static std::atomic<uint64_t> raised{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (dev <= 63 && (raised.load(std::memory_order_relaxed) & bit)) return hipSuccess;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(Kernel),
                          hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) raised.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Output tiles, the grid's y and the bytes of a workgroup's list of routes.
template <int XE>
int out_tiles(const W4Args& a) {
  const int cols = XE == ELEM_PARTS ? 32 : 16;
  return ((a.swiglu ? a.N / 2 : a.N) + cols - 1) / cols;
}
int list_bytes(const W4Args& a) { return a.ids ? (a.R * 2 + 15) / 16 * 16 : 0; }
int grid_y(const W4Args& a, int tile) {
  return !a.ids ? (a.R + tile - 1) / tile : a.R <= a.E ? a.R : a.E + 1;
}

template <int FMT, int XE, int SE, int GM, bool RAG, int NT, bool SWIGLU, int D>
hipError_t launch_one(const W4Args& a, int tile, int token_lds, hipStream_t stream) {
  const int tiles = out_tiles<XE>(a), y = grid_y(a, tile);
  // Several tiles a workgroup once there are some times more tiles than the 768 to
  // 1,024 workgroups that the GPU holds at once.  FFNs of K = 4096, I = 2048, int4
  // with zeros, by tiles of each product:
  //   1,152 (16 tokens, 8 experts, top-2)   48 us with one, 53 with two, 79 with four
  //   4,224 (16 tokens, 32 experts, top-4)  118, 112, 124
  //   8,320 (32 tokens, 64 experts, top-4)  223, 203, 216
  //   24,576 (32 tokens, 256 experts, top-6)  482, 413, 409
  // and K = 2048, I = 1024: 12,288 (32 tokens, 256 experts, top-6) 156, 127, 123.
  const int64_t all = (int64_t)tiles * y;
  const int run = all < 4096 ? 1 : all < 12288 ? 2 : 4;
  const int lds = token_lds + sum_lds<XE, NT>() + list_bytes(a);
  constexpr auto kernel = k_w4<FMT, XE, SE, GM, RAG, NT, SWIGLU, D>;
  if (lds > 65536) {
    const hipError_t e = allow_lds<kernel>(kTokenLdsMost + kSumLds + kW4MaxRoutes * 2);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, dim3((tiles + run - 1) / run, y), dim3(kThreads), lds, stream, a, tile,
                     run, token_lds);
  return hipGetLastError();
}

template <int FMT, int XE, int SE, int GM, bool RAG, bool DEEP>
hipError_t launch_shape(const W4Args& a, int tile, int token_lds, hipStream_t stream) {
  constexpr int D = DEEP ? 4 : 2;
  if constexpr (XE == ELEM_PARTS) {
    return launch_one<FMT, XE, SE, GM, RAG, 2, false, D>(a, tile, token_lds, stream);
  } else {
    if (a.swiglu) return launch_one<FMT, XE, SE, GM, RAG, 2, true, D>(a, tile, token_lds, stream);
    return launch_one<FMT, XE, SE, GM, RAG, 1, false, D>(a, tile, token_lds, stream);
  }
}

template <int FMT, int XE, int SE, int GM, bool RAG>
hipError_t launch_walk(const W4Args& a, hipStream_t stream) {
  // Tokens of one pass over the weights: 16, or 8 of more parts, so that two
  // steps of them fit the LDS.  Where the experts have few routes on average,
  // passes of fewer tokens leave room for more steps ahead, and an expert with
  // more routes takes another pass.  At most a route an expert (T = 32, 256
  // experts, top-6): 369 us with passes of 4, 392 with 8.  At most two (FFN of 16
  // tokens in int4, 64 experts, top-6): K = 4096, I = 2048 197 us with half passes,
  // 201 with whole ones; K = 2048, I = 1024 58 and 62; K = 1024, I = 768, whose
  // tokens fit the LDS either way, 41 and 40.
  const int tokens = a.R / a.top_k;
  int tile = kTile / parts<FMT, XE>();
  if (a.ids && a.R <= a.E) tile = 4;
  else if (a.ids && a.R <= 2 * (int64_t)a.E) tile /= 2;
  if (tokens < tile) tile = tokens;
  // Four steps ahead, where the tokens' K fits the LDS whole, or two.  A round of
  // four that a wave has one or two steps of loads the last one again for the
  // others: two is better there (40 routes of 64 experts, groups of 128, first
  // product: K = 1024 17.5 us against 20.2, 2048 38.1 against 35.4).  Narrow groups
  // are short of vector instructions before they are short of loads in flight
  // (groups of 32, 2048: 43.4 against 49.0; 4096: 83.3 against 81.2), and so are
  // those of 64 in the second product, which holds the tokens in three parts (FFN
  // of 8 tokens, 256 experts, top-6, K = 1024, I = 2048: 54.1 us with two steps,
  // 54.6 with four; I = 1920 52.9 and 56.4; e2m1 49.2 and 49.2, 32 tokens 121.5
  // and 120.1).  Its ragged int4 rows of 128 have registers for two only, of three
  // waves a SIMD (I = 1920: 51.5 us against 52.5 with four, which spill).
  const int steps = (a.K + kUnit - 1) / kUnit, last = steps % 4;
  const int rounded = (steps + 3) / 4 * 4, row = lds_rows<FMT, XE>() * tile * 2;
  // More LDS for the tokens, so that K fits whole, where all workgroups still
  // find a place at once (8 tokens of 4096 x 4096 in groups of 128: 7.7 us against
  // 8.5, 16 tokens 10.3 against 11.3; 32 tokens of 4096 x 8192, which no longer
  // do, 41.4 against 19.2).
  const int64_t whole = row * ((int64_t)rounded * kUnit + kPad);
  const int64_t groups = (int64_t)out_tiles<XE>(a) * grid_y(a, tile);
  int token_lds = least_token_lds<XE>();
  if (whole > token_lds && whole <= kTokenLdsMost &&
      groups <= kCUs * (kLds / (whole + kSumLds + list_bytes(a) + 64)))
    token_lds = (int)(whole + 15) / 16 * 16;
  const int held = (token_lds / row - kPad) / kUnit;
  if constexpr (XE != ELEM_PARTS || (GM == 1 && !(RAG && FMT == W4_INT))) {
    if (held >= rounded && (last == 0 || last == 3) && (GM < 4 || steps > 6))
      return launch_shape<FMT, XE, SE, GM, RAG, true>(a, tile, token_lds, stream);
  }
  return launch_shape<FMT, XE, SE, GM, RAG, false>(a, tile, token_lds, stream);
}

template <int XE, int SE>
hipError_t launch_format(int format, const W4Args& a, hipStream_t stream) {
  const bool ragged = a.K % 512 || a.group == a.K;
  if (format == W4_MX)
    return ragged ? launch_walk<W4_MX, XE, ELEM_BF16, 1, true>(a, stream)
                  : launch_walk<W4_MX, XE, ELEM_BF16, 1, false>(a, stream);
  if (a.group == 32)
    return ragged ? launch_walk<W4_INT, XE, SE, 4, true>(a, stream)
                  : launch_walk<W4_INT, XE, SE, 4, false>(a, stream);
  if (a.group == 64)
    return ragged ? launch_walk<W4_INT, XE, SE, 2, true>(a, stream)
                  : launch_walk<W4_INT, XE, SE, 2, false>(a, stream);
  return ragged ? launch_walk<W4_INT, XE, SE, 1, true>(a, stream)
                : launch_walk<W4_INT, XE, SE, 1, false>(a, stream);
}

}  // namespace

hipError_t launch_w4(int format, const W4Args& args, hipStream_t stream) {
  if (args.R == 0) return hipSuccess;
  W4Args a = args;
  a.inv_top_k = (uint32_t)(((uint64_t(1) << 32) + a.top_k - 1) / a.top_k);
  if (a.xelem == ELEM_F16) return launch_format<ELEM_F16, ELEM_F16>(format, a, stream);
  if (a.xelem == ELEM_BF16) return launch_format<ELEM_BF16, ELEM_BF16>(format, a, stream);
  if (a.scale_elem == ELEM_F16) return launch_format<ELEM_PARTS, ELEM_F16>(format, a, stream);
  return launch_format<ELEM_PARTS, ELEM_BF16>(format, a, stream);
}

namespace {

template <int FMT, int SE, int GM, bool RAG>
hipError_t launch_token(const W4Args& a, const float* weights, int T, hipStream_t stream) {
  constexpr auto kernel = k_w4_token<FMT, SE, GM, RAG>;
  // eight waves take a little over the default limit
  const hipError_t e = allow_lds<kernel>(kTokenWaves * token_lds<FMT, GM>());
  if (e != hipSuccess) return e;
  const int waves = a.top_k < kTokenWaves ? a.top_k : kTokenWaves;
  constexpr int lds = token_lds<FMT, GM>();
  hipLaunchKernelGGL(kernel, dim3((a.N + 15) / 16, T), dim3(waves * 64), waves * lds, stream, a,
                     weights);
  return hipGetLastError();
}

template <int FMT, int SE, int GM>
hipError_t launch_token(const W4Args& a, const float* weights, int T, hipStream_t stream) {
  return a.K % 512 || a.group == a.K
             ? launch_token<FMT, SE, GM, true>(a, weights, T, stream)
             : launch_token<FMT, SE, GM, false>(a, weights, T, stream);
}

template <int SE>
hipError_t launch_token_int4(const W4Args& a, const float* weights, int T, hipStream_t stream) {
  if (a.group == 32) return launch_token<W4_INT, SE, 4>(a, weights, T, stream);
  if (a.group == 64) return launch_token<W4_INT, SE, 2>(a, weights, T, stream);
  return launch_token<W4_INT, SE, 1>(a, weights, T, stream);
}

}  // namespace

hipError_t launch_w4_down(int format, const W4Args& a, const float* weights, float* y, int T,
                          hipStream_t stream) {
  // A route per wave reads and converts an expert's weights for every token that
  // chose it, so this is for few tokens whose routes seldom share one.  FFNs of K
  // = 4096, I = 2048, against the grouped products:
  //   256 experts, top-6, e2m1: two tokens 40.0 us against 44.0, four 75 and 75
  //   64 experts, top-6, four tokens: int4 76 against 79, e2m1 72 and 72
  //   8 experts, top-4, four tokens: int4 35.6 against 36.6, e2m1 34.0 and 35.3
  //   8 experts, top-6, four tokens: int4 48.8 against 40.7, e2m1 46.2 and 39.1
  //   8 experts, top-8, three tokens: int4 43.0 against 39.4, e2m1 41.4 and 36.8
  if (T <= kW4TokenMax && a.R <= 2 * (int64_t)a.E) {
    if (format == W4_MX) return launch_token<W4_MX, ELEM_BF16, 1>(a, weights, T, stream);
    return a.scale_elem == ELEM_F16 ? launch_token_int4<ELEM_F16>(a, weights, T, stream)
                                    : launch_token_int4<ELEM_BF16>(a, weights, T, stream);
  }
  W4Args down = a;
  down.out = y;
  down.oelem = ELEM_F32;
  const hipError_t e = launch_w4(format, down, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_w4_combine, dim3((a.N / 4 + kCombineThreads - 1) / kCombineThreads, T),
                     dim3(kCombineThreads), 0, stream, y, a.ids, weights, a.out, a.oelem, a.top_k,
                     a.N, a.E);
  return hipGetLastError();
}
