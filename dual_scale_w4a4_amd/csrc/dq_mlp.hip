// dq_mlp.hip -- products with packed MXFP4 weights and what follows them in a decoder layer's
// MLP, on gfx950's MX-scaled matrix cores:
//
//   epilogue  Y[t][i] = residual[t][i] + act(a_i s[t][i] + bias_i)
//   gated     H[t][i] = act(ag_i g[t][i]) * (au_i u[t][i]), stored or quantized
//
// with s, g, u the sums over k of activation times weight values. The activations are MXFP4
// or MXFP8 as the quantizers write them, the weights MXFP4 in the packed layout of
// dq_gemm_pack_weights: for each block of 32 rows, 256-k stage and k step i (0..3) a 1 KiB
// block in which lane L holds row L % 32, k chunk 4 (L / 32) + i of the stage (chunks of 32 k).
//
// One V_MFMA_SCALE_F32_32X32X64 step takes the weights as operand A and 32 tokens as operand B;
// lane half h = lane / 32. FP4: a lane holds the 32 k values of its half's chunk (16 bytes). FP8: a
// lane holds k values 16 h .. + 15 of both halves' chunks (16 bytes of each), while its scale
// byte stays that of its own half's chunk. Result v of a lane is D[(v / 4) * 8 + 4 h + v % 4]
// [lane % 32]. (Layouts checked exactly on gfx950 against the definition.)
//
// In its 8-bit mode the instruction truncates the products of each run of 8 k at 2^-13 of the
// power of two of the largest (a float64 emulation of that agrees with bf16 results in 99.96% of
// the elements, exact sums in 99.3%, at K 512); FP4 products are added exactly and accumulated in
// fp32.
#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "../../include/dq_mlp.h"
#include "dq_outq.h"

namespace dqm {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
// 4 channels of an output or residual, which are aligned to their element only
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef bf16x4 bf16x4_any __attribute__((aligned(2)));

constexpr int kStage = 256;           // k values per packed stage
constexpr int kPackStepB = 1024;      // packed codes of (row block, stage, step)
constexpr int kPackStageB = 4096;     // packed codes of (row block, stage)
constexpr int kPackScaleB = 256;      // packed scales of (row block, stage)
constexpr uint32_t kBufRsrcWord3 = 0x00020000u;  // raw buffer, 32-bit data format
constexpr uint32_t kOob = 0x80000000u;           // an offset past every buffer: reads zero
// cache policy of buffer stores: nontemporal, since outputs are written once and not read here (ordinary
// stores 1% slower: 14336 -> 4096, 2048 tokens 60.1 against 59.4 us)
constexpr int kNt = 2;

constexpr int64_t kMaxOut = 1 << 22;  // 127 rows of fp32 outputs span less than 2^31 bytes

enum Out : int { kOutF32 = 0, kOutBf16 = 1, kOutFp4 = 2, kOutFp8 = 3 };

struct MlpArgs {
  const uint8_t* xc;     // tokens x K/2 (FP4) or tokens x K (FP8)
  const uint8_t* xs;     // tokens x K/32
  const uint8_t* wc[2];  // packed codes: [0] the product's or the gate's, [1] the up weights'
  const uint8_t* ws[2];  // packed scales
  const float* a[2];     // out, or null
  const float* bias;     // out, or null (single product)
  const void* res;       // tokens x out of y's type, or null (single product)
  void* y;               // tokens x out
  const float* b;        // out, or null (quantized)
  uint8_t* codes;        // quantized
  uint8_t* scales;
  int tokens, out, K, act;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes,
                                           (int)kBufRsrcWord3);
}

// ---------------------------------------------------------------------------- activations

__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
}

// (1 + erf(z / sqrt 2)) / 2 to a few fp32 roundings of itself on both sides of zero: a sum of 1 and
// erf cancels for negative z (up to 1% off at z = -4.5, zero or one step below -5.6), and a
// group of negative channels is quantized by its own largest. For w = |z| the smaller half is
// exp(-w^2 / 2) times exp(w^2 / 2) erfc(w / sqrt 2) / 2, which is smooth and between 1/2 and 0: a
// polynomial in 1 / (1 + 0.23 w), fitted to the least largest relative error over w <= 14 (3.2e-8;
// beyond, the exponential is zero). The exponent's roundings leave 0.75 w^2 2^-23. No branches:
// 14336 -> 4096 with 2048 tokens 61 us, where the sum with erff took 66 and erfcf 69 (no activation
// 59); gated 4096 -> 14336 118, 118 and 135 (112).
__device__ __forceinline__ float normal_below(float z) {
  const float w = fabsf(z), t = __builtin_amdgcn_rcpf(fmaf(w, 0.23f, 1.0f));
  float g = -0.0790351118f;
  g = fmaf(g, t, 0.293058358f);
  g = fmaf(g, t, -0.283361436f);
  g = fmaf(g, t, 0.307211192f);
  g = fmaf(g, t, -0.0367220469f);
  g = fmaf(g, t, 0.121069719f);
  g = fmaf(g, t, 0.0853795898f);
  g = fmaf(g, t, 0.0924304118f);
  g = fmaf(g, t, -3.07274420e-05f);
  const float q = g * __builtin_amdgcn_exp2f(w * w * -0.721347520f);
  return z < 0.0f ? q : 1.0f - q;
}

template <int ACT>
__device__ __forceinline__ float activation(float z) {
  if (ACT == DQ_ACTIVATION_RELU) return z < 0.0f ? 0.0f : z;  // a NaN stays one
  if (ACT == DQ_ACTIVATION_SILU) return z * sigmoid(z);
  if (ACT == DQ_ACTIVATION_GELU) return z * normal_below(z);
  if (ACT == DQ_ACTIVATION_GELU_TANH)  // (1 + tanh u) / 2 = sigmoid(2 u)
    return z * sigmoid(1.5957691216057308f * (z + 0.044715f * z * z * z));
  return z;
}

// f(integral_constant<ACT>) for the call's activation (a uniform branch)
template <class F>
__device__ __forceinline__ void with_activation(int act, F f) {
  switch (act) {
    case DQ_ACTIVATION_RELU: f(std::integral_constant<int, DQ_ACTIVATION_RELU>{}); break;
    case DQ_ACTIVATION_SILU: f(std::integral_constant<int, DQ_ACTIVATION_SILU>{}); break;
    case DQ_ACTIVATION_GELU: f(std::integral_constant<int, DQ_ACTIVATION_GELU>{}); break;
    case DQ_ACTIVATION_GELU_TANH: f(std::integral_constant<int, DQ_ACTIVATION_GELU_TANH>{}); break;
    default: f(std::integral_constant<int, DQ_ACTIVATION_NONE>{}); break;
  }
}

// ------------------------------------------------------------------------------- epilogue

// out floats of p at channels ich .. ich + 3 (0 or 1 where p is null or the channel is past
// the end)
__device__ __forceinline__ f32x4 load_channels(const float* p, int ich, int out, float none) {
  f32x4 v = {none, none, none, none};
  if (p) {
    if (ich + 3 < out) {
      v = *reinterpret_cast<const f32x4*>(p + ich);
    } else {
#pragma unroll
      for (int e = 0; e < 4; e++) v[e] = ich + e < out ? p[ich + e] : none;
    }
  }
  return v;
}

// The epilogue's value of 4 channels from the raw sums s0 (and s1)
template <bool GATED>
__device__ __forceinline__ f32x4 combine(int act, const f32x4& a0, const f32x4& a1,
                                         const f32x4& bias, const f32x4& s0, const f32x4& s1) {
  f32x4 y;
  with_activation(act, [&](auto k) {
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const float z = GATED ? s0[e] * a0[e] : s0[e] * a0[e] + bias[e];
      y[e] = activation<decltype(k)::value>(z);
      if (GATED) y[e] *= s1[e] * a1[e];
    }
  });
  return y;
}

// Store channels ich .. ich + 3 of token t, those that exist, after adding the residual.
template <int OUT>
__device__ __forceinline__ void store_row(const MlpArgs& p, int64_t t, int ich, f32x4 y) {
  const int64_t off = t * p.out + ich;
  typedef typename std::conditional<OUT == kOutF32, float, __bf16>::type T;
  typedef typename std::conditional<OUT == kOutF32, f32x4_any, bf16x4_any>::type T4;
  T* yp = static_cast<T*>(p.y) + off;
  const T* rp = static_cast<const T*>(p.res) + off;
  if (ich + 3 < p.out) {
    if (p.res) {
      const T4 r = *reinterpret_cast<const T4*>(rp);
#pragma unroll
      for (int e = 0; e < 4; e++) y[e] = (float)r[e] + y[e];
    }
    *reinterpret_cast<T4*>(yp) = T4{(T)y[0], (T)y[1], (T)y[2], (T)y[3]};
  } else {
#pragma unroll
    for (int e = 0; e < 3; e++)
      if (ich + e < p.out) yp[e] = (T)(p.res ? (float)rp[e] + y[e] : y[e]);
  }
}

// Quantize channels ich .. ich + 3 of token t and store codes and scale: the 8 lanes of an
// aligned group of 8 hold the 32 channels of one scale group of one token, and all are here.
template <int OUT>
__device__ __forceinline__ void store_quantized(const MlpArgs& p, int64_t t, int ich,
                                                const f32x4& b, const f32x4& y) {
  const int64_t off = t * p.out + ich;
  float x[4];
  uint32_t mb = 0u;
#pragma unroll
  for (int e = 0; e < 4; e++) {
    x[e] = y[e] * b[e];
    mb = max(mb, dq::f2u(x[e]) & 0x7FFFFFFFu);
  }
  mb = dq::group_max_bits<8>(mb);
  const bool bad = mb >= 0x7F800000u;  // a NaN or an infinity in the group
  if (bad) {
    mb = 0u;
#pragma unroll
    for (int e = 0; e < 4; e++) x[e] = 0.0f;
  }
  const uint32_t sc = dq::mx_scale_code<OUT == kOutFp8 ? 8 : 2>(mb);
  if (OUT == kOutFp8)
    *reinterpret_cast<uint32_t*>(p.codes + off) = dq::fp8_pack4(x, dq::u2f((254u - sc) << 23));
  else
    *reinterpret_cast<uint16_t*>(p.codes + (off >> 1)) =
        (uint16_t)dq::fp4_pack<4>(x, dq::mx_group(sc));
  if ((threadIdx.x & 7) == 0) p.scales[off >> 5] = bad ? 0xFFu : (uint8_t)sc;
}

// ------------------------------------------------------------------- operands
// k runs in stages of 128 bytes of a token row: 256 k in four steps (FP4), 128 k in two (FP8:
// half a packed stage, steps 2 hs and 2 hs + 1 of it, hs = stage % 2; of each token row the bytes
// of k chunks 2 hs, 2 hs + 1, 4 + 2 hs and 5 + 2 hs). In LDS a row's eight 16-byte pieces are
// XOR-swizzled so that neither the loads to LDS (whole rows) nor the reads (one piece of 32 rows
// and both lane halves) conflict.

typedef __attribute__((address_space(3))) void* lds_ptr_t;

// s_waitcnt operand: at most n vector-memory operations outstanding, the other counters free
constexpr int vmcnt_imm(int n) { return (n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14); }

constexpr int kRowB = 128;         // bytes of a token row in a stage
constexpr int kScaleRowB = 16;     // token scale bytes per row and period (512 k)
constexpr int steps(bool act8) { return act8 ? 2 : 4; }

// 16 bytes per lane from memory to LDS: lane l's at dst + 16 l
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t rs, uint8_t* dst, uint32_t voff,
                                         int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)dst, 16, (int)voff, soff, 0, 0);
}

// The 16-byte piece(s) of one token row that step ks takes: xt = the row's swizzle term with the
// lane half folded in (FP4: piece 4 h + ks; FP8: pieces 2 ks + h and 4 + 2 ks + h).
template <bool ACT8>
__device__ __forceinline__ u32x4 read_x(const uint8_t* row, int ks, int part, int xt) {
  return *reinterpret_cast<const u32x4*>(row + (((ACT8 ? 2 * ks + 4 * part : ks) ^ xt) * 16));
}

// order LDS accesses of one wave (its LDS instructions execute in order; this keeps the compiler
// from moving them)
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <bool ACT8>
__device__ __forceinline__ v16f mfma(const u32x4& a, const u32x4* b, v16f c, uint32_t sa,
                                     uint32_t sb, int step) {
  const v8i A = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const u32x4 b0 = b[0], b1 = ACT8 ? b[1] : u32x4{0u, 0u, 0u, 0u};
  const v8i B = {(int)b0[0], (int)b0[1], (int)b0[2], (int)b0[3],
                 (int)b1[0], (int)b1[1], (int)b1[2], (int)b1[3]};
  constexpr int F = ACT8 ? 0 : 4;  // operand B: E4M3 or E2M1
  switch (step) {  // the scale byte is chosen by an immediate
    case 0: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, 4, F, 0, (int)sa, 0, (int)sb);
    case 1: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, 4, F, 1, (int)sa, 1, (int)sb);
    case 2: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, 4, F, 2, (int)sa, 2, (int)sb);
    default: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, 4, F, 3, (int)sa, 3, (int)sb);
  }
}

// ------------------------------------------------------------------- split-k kernel
// A workgroup owns M row blocks of 32 (the product's M neighbouring ones; gated: the gate's and
// the up weights' block of the same 32 channels) and 32 NB tokens; its W waves share k between
// them in periods of 512, wave w taking periods w, w + W, .., and their partial sums are joined
// in LDS in wave order. Every wave runs by itself: its weights go from memory straight to
// registers, its tokens through a ring of two LDS stages of its own, both loaded two of its
// stages ahead, and the token scales (16 bytes of a row for a whole period, instead of 4 of
// every row and stage: 14336 -> 4096 at 256 tokens 20 -> 17 us) through LDS as well. Token
// fragments are read kAhead blocks before their products. Bound by the weights' memory traffic:
// gated 4096 -> 14336 with 32 tokens 12.3 us for 63 MB (5.1 TB/s, a copy's rate), 14336 -> 4096 with
// one token 8.0 us for 31 MB (3.9 TB/s: about 2 us of it launch, ramp and join).

// LDS row of one token's 32 partial sums, padded so that 8 rows cover distinct banks
constexpr int kPartRow = 36;
constexpr int kPartBlock = 32 * kPartRow;  // floats of one 32 x 32 block

// Token fragments are read kAhead blocks of 32 tokens before their products, in a ring of four.
constexpr int kAhead = 3;

// One stage's weights of a wave.
template <bool ACT8, int M>
struct Frags {
  u32x4 a[M][steps(ACT8)];
  uint32_t sa[M];
};

template <bool ACT8, bool GATED, int M, int NB, int OUT, int W>
__global__ __launch_bounds__(W * 64) void k_mlp_split(MlpArgs p) {
  static_assert(!GATED || M == 2, "gate and up");
  constexpr int NK = steps(ACT8);
  constexpr int PER = ACT8 ? 4 : 2;       // stages of a period
  constexpr int NS = (NB + 1) / 2;        // scale loads of a period, 64 rows each
  constexpr int kRing = NB * 32 * kRowB;  // one stage of a wave's tokens
  constexpr int kXs = NS * 1024;          // one period of a wave's token scales
  constexpr int kWave = 2 * kRing + 2 * kXs;
  constexpr int kPart = W * M * kPartBlock * 4;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[W * kWave > kPart ? W * kWave : kPart];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rl = lane & 31, h = lane >> 5;
  const int nrb = (p.out + 31) / 32;
  const int ntr = GATED ? nrb : (nrb + M - 1) / M;   // row tiles
  const int rb0 = (blockIdx.x % ntr) * (GATED ? 1 : M);
  const int t0 = (blockIdx.x / ntr) * (32 * NB);
  const int rows = min(p.tokens - t0, 32 * NB);
  const int ldb = ACT8 ? p.K : p.K / 2, nkb = p.K / 32, npk = p.K / kStage;
  const int nper = p.K / 512;

  __amdgpu_buffer_rsrc_t rw[M], rs[M];
#pragma unroll
  for (int m = 0; m < M; m++) {
    const int rb = GATED ? rb0 : rb0 + m;
    const bool in = rb < nrb;  // a block past the last weight row reads nothing
    const int64_t at = in ? rb : 0;
    rw[m] = rsrc(p.wc[GATED ? m : 0] + at * npk * kPackStageB, in ? (uint32_t)npk * kPackStageB : 0u);
    rs[m] = rsrc(p.ws[GATED ? m : 0] + at * npk * kPackScaleB, in ? (uint32_t)npk * kPackScaleB : 0u);
  }
  const __amdgpu_buffer_rsrc_t rx = rsrc(p.xc + (int64_t)t0 * ldb, (uint32_t)rows * (uint32_t)ldb);
  const __amdgpu_buffer_rsrc_t rxs = rsrc(p.xs + (int64_t)t0 * nkb, (uint32_t)rows * (uint32_t)nkb);
  uint32_t vx[4 * NB], vs[NS];
#pragma unroll
  for (int j = 0; j < 4 * NB; j++) {
    // lane l writes piece position l % 8 of row r, which holds the row's piece (l % 8) ^ term
    const int r = 8 * j + (lane >> 3);
    const int pc = (lane & 7) ^ (r & 7) ^ ((r >> 3) & 1);
    vx[j] = r < rows ? (uint32_t)r * (uint32_t)ldb + (uint32_t)pc * 16u + (ACT8 && pc >= 4 ? 64u : 0u)
                     : kOob;
  }
#pragma unroll
  for (int j = 0; j < NS; j++) {
    const int r = 64 * j + lane;
    vs[j] = r < rows ? (uint32_t)r * (uint32_t)nkb : kOob;
  }
  uint8_t* ring = lds + wave * kWave;
  uint8_t* xsb = ring + 2 * kRing;
  const int xt = (rl & 7) ^ ((rl >> 3) & 1) ^ (ACT8 ? h : 4 * h);

  v16f acc[M][NB];
#pragma unroll
  for (int m = 0; m < M; m++)
#pragma unroll
    for (int n = 0; n < NB; n++) acc[m][n] = v16f{};

  // the loads of stage J of period q: kLoads, and before them on a period's first the scales.
  // Past the last period they read nothing, so that every stage issues the same number and the
  // loop body stays one basic block.
  constexpr int kLoads = 4 * NB + M * (NK + 1);
  static_assert(kLoads + NS < 64, "the wait counts to 63");
  const __amdgpu_buffer_rsrc_t rnone = rsrc(p.xc, 0u);
  auto load = [&](auto jc, int q, int par, Frags<ACT8, M>& f) {
    constexpr int J = decltype(jc)::value;
    const int s = q * PER + J;
    const bool on = q < nper;
    if (J == 0)
#pragma unroll
      for (int j = 0; j < NS; j++)
        load_lds(on ? rxs : rnone, xsb + par * kXs + j * 1024, vs[j], q * 16);
#pragma unroll
    for (int j = 0; j < 4 * NB; j++)
      load_lds(on ? rx : rnone, ring + (J & 1) * kRing + j * 1024, vx[j],
               ACT8 ? (s >> 1) * 256 + (s & 1) * 64 : s * kRowB);
#pragma unroll
    for (int m = 0; m < M; m++) {
#pragma unroll
      for (int i = 0; i < NK; i++)
        f.a[m][i] = __builtin_amdgcn_raw_buffer_load_b128(on ? rw[m] : rnone, (uint32_t)lane * 16u,
                                                          (uint32_t)((s * NK + i) * kPackStepB), 0);
      f.sa[m] = __builtin_amdgcn_raw_buffer_load_b32(on ? rs[m] : rnone, (uint32_t)lane * 4u,
                                                     (uint32_t)((ACT8 ? s >> 1 : s) * kPackScaleB), 0);
    }
  };
  // the products of stage J of a period whose scales are in xsb + par * kXs
  auto products = [&](auto jc, int par, const Frags<ACT8, M>& f) {
    constexpr int J = decltype(jc)::value, HS = ACT8 ? J & 1 : 0, F = NK * NB;
    const uint8_t* xb = ring + (J & 1) * kRing + rl * kRowB;
    const uint8_t* xp = xsb + par * kXs + rl * kScaleRowB + 4 * h + (ACT8 ? J >> 1 : J) * 8;
    u32x4 b[4][ACT8 ? 2 : 1];
    uint32_t sx[NB];
    auto read = [&](int k) {
#pragma unroll
      for (int e = 0; e < (ACT8 ? 2 : 1); e++)
        b[k % 4][e] = read_x<ACT8>(xb + (k % NB) * 32 * kRowB, k / NB, e, xt);
    };
#pragma unroll
    for (int n = 0; n < NB; n++) sx[n] = *reinterpret_cast<const uint32_t*>(xp + n * 32 * kScaleRowB);
#pragma unroll
    for (int k = 0; k < (F < kAhead ? F : kAhead); k++) read(k);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < F; k++) {
      if (k + kAhead < F) read(k + kAhead);
#pragma unroll
      for (int m = 0; m < M; m++)
        acc[m][k % NB] = mfma<ACT8>(f.a[m][k / NB], b[k % 4], acc[m][k % NB], f.sa[m], sx[k % NB],
                                    ACT8 ? 2 * HS + k / NB : k / NB);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  Frags<ACT8, M> f0, f1;
  // A stage's loads are done before it is read (only the next stage's are newer), and its reads
  // are done before its buffer is loaded again with the stage after the next: no other wave
  // touches the ring.
  auto stage = [&](auto jc, int q, int par) {
    constexpr int J = decltype(jc)::value;
    Frags<ACT8, M>& f = (J & 1) ? f1 : f0;
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(kLoads + (J + 1 < PER ? 0 : NS)));
    wave_lds_order();
    products(jc, par, f);
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    wave_lds_order();
    if constexpr (J + 2 < PER)
      load(std::integral_constant<int, J + 2>{}, q, par, f);
    else
      load(std::integral_constant<int, J + 2 - PER>{}, q + W, par ^ 1, f);
    __builtin_amdgcn_sched_barrier(0);
  };
  load(std::integral_constant<int, 0>{}, wave, 0, f0);
  __builtin_amdgcn_sched_barrier(0);
  load(std::integral_constant<int, 1>{}, wave, 0, f1);
  for (int q = wave, par = 0; q < nper; q += W, par ^= 1) {
    stage(std::integral_constant<int, 0>{}, q, par);
    stage(std::integral_constant<int, 1>{}, q, par);
    if constexpr (PER == 4) {
      stage(std::integral_constant<int, 2>{}, q, par);
      stage(std::integral_constant<int, 3>{}, q, par);
    }
  }
  // the last loads read nothing but still write zeros into LDS: drain them before the join
  // reuses that memory
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));

  // the factors of the 4 channels whose sums this thread finishes
  constexpr int MS = GATED ? 1 : M;                         // blocks of results
  constexpr int NX = (256 * MS + W * 64 - 1) / (W * 64);    // 4-channel pieces per thread and n
  const int ch = (threadIdx.x & 7) * 4;
  f32x4 a0[NX], a1[NX], cc[NX];
#pragma unroll
  for (int x = 0; x < NX; x++) {
    const int ich = (rb0 + (threadIdx.x + x * W * 64) / 256) * 32 + ch;
    a0[x] = load_channels(p.a[0], ich, p.out, 1.0f);
    a1[x] = load_channels(GATED ? p.a[1] : nullptr, ich, p.out, 1.0f);
    cc[x] = load_channels(GATED ? p.b : p.bias, ich, p.out, GATED ? 1.0f : 0.0f);
  }
  // join: block (m, n) of every wave as rows of tokens, then each thread adds the W partial sums
  // of 4 channels of one token in wave order
  float* part = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int n = 0; n < NB; n++) {
    __syncthreads();  // every wave is done with its ring, or with the block before
#pragma unroll
    for (int m = 0; m < M; m++)
#pragma unroll
      for (int g = 0; g < 4; g++)
        *reinterpret_cast<f32x4*>(part + (wave * M + m) * kPartBlock + rl * kPartRow + g * 8 + h * 4) =
            f32x4{acc[m][n][g * 4], acc[m][n][g * 4 + 1], acc[m][n][g * 4 + 2], acc[m][n][g * 4 + 3]};
    __syncthreads();
#pragma unroll
    for (int x = 0; x < NX; x++) {
      const int id = threadIdx.x + x * W * 64, mr = id / 256, tr = (id >> 3) & 31;
      const int t = t0 + n * 32 + tr, ich = (rb0 + mr) * 32 + ch;
      if (mr >= MS || t >= p.tokens) continue;  // the same for the 8 lanes of a group of channels
      f32x4 s[2] = {f32x4{}, f32x4{}};
#pragma unroll
      for (int k = 0; k < (GATED ? 2 : 1); k++)
#pragma unroll
        for (int w = 0; w < W; w++)
          s[k] += *reinterpret_cast<const f32x4*>(part + (w * M + (GATED ? k : mr)) * kPartBlock +
                                                  tr * kPartRow + ch);
      const f32x4 y = combine<GATED>(p.act, a0[x], a1[x], cc[x], s[0], s[1]);
      if constexpr (OUT >= kOutFp4) store_quantized<OUT>(p, t, ich, cc[x], y);
      else store_row<OUT>(p, t, ich, y);
    }
  }
}

// --------------------------------------------------------------------- tile kernel
// Four waves, each with two 32-row weight blocks m (single product: blocks 2 w, 2 w + 1 of the
// tile's 256 rows; gated: the gate's and the up weights' block of the tile's channels 32 w ..)
// times all the tile's 32 NB tokens. Weight fragments go from memory straight into registers,
// each entering the CU once; the tokens go through LDS.
//
// Loads run two stages ahead: the fragments of two stages are a ring of registers, each reloaded
// right after the last product that reads it, and the tokens use a ring of four LDS buffers.
//
// Two workgroups fit a CU (one of 256 x 256: gated 4096 -> 14336 with 8192 tokens 470 us against
// 450). That product runs at 4.1 - 4.35 PFLOP/s (441 - 469 us by the box) where a stream of the
// instruction on random register operands reaches 6.3 - 6.4 at the clock that the chip's power
// allows: the matrix cores are 62% busy, the rest waits for operands (copies without the weight
// or the token loads take 388 and 367 us of 446, without both and the LDS reads 335). 14336 ->
// 4096 with MXFP8 activations and 2048 tokens runs at 2.65 - 2.8 (86 - 91 us) of 4.1: 256 tiles,
// one wave per SIMD.

constexpr int kGroupM = 4;         // weight tiles per tile group (L2 reuse)

template <int NB>
struct TileLds {
  uint8_t x[4][NB * 32 * kRowB];   // [stage % 4]: token stages
  uint8_t xs[2][256 * kScaleRowB]; // [period parity]: token scales
};

template <bool ACT8, int NB>
struct TileCtx {
  __amdgpu_buffer_rsrc_t rw[2], rs[2], rx, rxs, rnone;
  int wave, nst;
  uint32_t vw[2], vs[2];  // this lane's offsets in the wave's weight blocks' codes and scales
  uint32_t vx[NB];        // token-stage offsets of this lane's rows, or kOob
  uint32_t vxs;           // token-scale offset of this lane's row, or kOob
};

// Token-stage load j of this wave: LDS rows 8 (NB wave + j) .. + 7, lane l writing row
// l / 8 of them at piece position l % 8.
template <bool ACT8, int NB>
__device__ __forceinline__ void load_x(const TileCtx<ACT8, NB>& c, uint8_t* xb, int j, int s,
                                       bool on) {
  const int o = ACT8 ? (s >> 1) * 256 + (s & 1) * 64 : s * kRowB;
  load_lds(on ? c.rx : c.rnone, xb + (c.wave * NB + j) * 1024, c.vx[j], o);
}

template <bool ACT8, int NB>
__device__ __forceinline__ void load_xs(const TileCtx<ACT8, NB>& c, uint8_t* xs, int q, bool on) {
  load_lds(on ? c.rxs : c.rnone, xs + c.wave * 1024, c.vxs, q * 16);
}

template <bool ACT8, int NB>
__device__ __forceinline__ u32x4 load_w(const TileCtx<ACT8, NB>& c, int m, int s, int ks, bool on) {
  return __builtin_amdgcn_raw_buffer_load_b128(
      on ? c.rw[m] : c.rnone, c.vw[m], (uint32_t)((s * steps(ACT8) + ks) * kPackStepB), 0);
}

template <bool ACT8, int NB>
__device__ __forceinline__ uint32_t load_ws(const TileCtx<ACT8, NB>& c, int m, int s, bool on) {
  return __builtin_amdgcn_raw_buffer_load_b32(on ? c.rs[m] : c.rnone, c.vs[m],
                                              (uint32_t)((ACT8 ? s >> 1 : s) * kPackScaleB), 0);
}

// Step KS of a stage (HS: FP8's half of the packed stage): 2 NB products in the order (n, m), and
// between them the token fragments kAhead blocks on, from LDS (past the stage's last those of
// the next stage, with its token scales); the reload of the step's weight fragments with stage
// s + 2's after their last products; and in step 0, before any of those, stage s + 2's token
// loads (XS: first the next period's token scales). Loads past the last stage read nothing (they
// still write zeros to LDS, into buffers no longer read), so every stage issues the same number.
//
// The stage's one barrier stands before the block kAhead from its end, the first at which stage
// s + 1's tokens are read. There those tokens' loads, the first of the loads issued in stage
// s - 1, are complete in this wave (the weight loads after them and this stage's loads may be in
// flight: a fixed count; the weights' own waits are at their uses), and after it in every
// wave. It also stands between the last reads of a token buffer, whose products every wave has
// issued a stage before, and the loads that fill the buffer again: with four buffers stage
// s + 1 loads into the one that stage s - 1 read.
template <bool ACT8, int NB, int KS, int HS, bool XS>
__device__ __forceinline__ void tile_step(v16f (&acc)[2][NB], u32x4 (&fa)[2][steps(ACT8)],
                                          u32x4 (&fb)[4][ACT8 ? 2 : 1], uint32_t (&sw)[2],
                                          const uint32_t (&sx)[NB], uint32_t (&sn)[NB],
                                          const uint8_t* lx, const uint8_t* lxn,
                                          const uint8_t* xsn, int xt, const TileCtx<ACT8, NB>& c,
                                          uint8_t* xb, uint8_t* xsb, int s, int q, bool xs_on) {
  constexpr int NK = steps(ACT8), F = NK * NB, kBar = F - kAhead;
  static_assert(F % 4 == 0 && kBar > 0, "the ring of fragments");
  const int s2 = s + 2;
  const bool on = s2 < c.nst;
#pragma unroll
  for (int n = 0; n < NB; n++) {
    const int i = KS * NB + n;            // this block of the stage
    const int f = (i + kAhead) % F;       // the block read now, of the next stage once it wraps
    const bool next = i + kAhead >= F;
    if (i == kBar) {
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(2 * NK + 2 + (XS ? 1 : 0) + (kBar < NB ? kBar : NB) +
                                           2 * (kBar / NB)));
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      __builtin_amdgcn_s_barrier();
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < NB; k++)
        sn[k] = *reinterpret_cast<const uint32_t*>(xsn + k * 32 * kScaleRowB);
    }
#pragma unroll
    for (int m = 0; m < 2; m++) {
      acc[m][n] = mfma<ACT8>(fa[m][KS], fb[i % 4], acc[m][n], sw[m], sx[n], ACT8 ? 2 * HS + KS : KS);
      if (XS && KS == 0 && n == 0 && m == 0) load_xs(c, xsb, q, xs_on);
      if (KS == 0 && m == 0) load_x(c, xb, n, s2, on);
      if (ACT8 || m == 0)
        fb[f % 4][ACT8 ? m : 0] = read_x<ACT8>((next ? lxn : lx) + (f % NB) * 32 * kRowB, f / NB, m, xt);
      if (n == NB - 1) {
        fa[m][KS] = load_w(c, m, s2, KS, on);
        if (KS == NK - 1) sw[m] = load_ws(c, m, s2, on);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// The epilogue, 32 tokens (one n) at a time. Result v of block (m, n) is channel
// 32 rb + 8 (v / 4) + 4 h + v % 4 of the block's 32 and token 32 n + lane % 32.
//   gated: the gate's and the up product of a channel lie in the same lane, so scales, activation
//     and product are applied there, on registers. Quantized outputs then need one exchange
//     between the lane halves (a token's 32 channels lie in lanes l and l + 32) and are stored
//     from there.
//   bf16 and fp32 outputs go through LDS, so that the stores cover whole rows of the wave's
//     channels instead of 8 or 16 bytes of 32 rows. The single product applies its factors
//     there, where a lane has the same 4 channels in every row, and loads its residual one
//     chunk ahead. Where the channels or the arrays do not fit 4-channel accesses they are made
//     all the same, at addresses aligned to the element only (out 9001, 700 tokens, K 2560: 15.8
//     us in bf16, 19.9 in fp32; out 9004 15.2 and 19.5; one channel per lane instead 18.2 and
//     21.6), and the last 1 .. 3 channels element by element.
template <bool GATED, int OUT>
__device__ __forceinline__ void quantize_chunk(const MlpArgs& p, f32x4 (&y)[4], int t, int rb,
                                               int h, bool in) {
  uint32_t mb = 0u;
#pragma unroll
  for (int g = 0; g < 4; g++)
#pragma unroll
    for (int e = 0; e < 4; e++) mb = max(mb, dq::f2u(y[g][e]) & 0x7FFFFFFFu);
  mb = max(mb, (uint32_t)__shfl_xor((int)mb, 32, 64));
  const bool bad = mb >= 0x7F800000u;  // a NaN or an infinity in the group
  if (bad) {
    mb = 0u;
#pragma unroll
    for (int g = 0; g < 4; g++) y[g] = f32x4{};
  }
  const uint32_t sc = dq::mx_scale_code<OUT == kOutFp8 ? 8 : 2>(mb);
  uint32_t c[4];  // the codes of channels 8 g + 4 h .. + 3
  if (OUT == kOutFp8) {
    const float rd = dq::u2f((254u - sc) << 23);
#pragma unroll
    for (int g = 0; g < 4; g++) c[g] = dq::fp8_pack4(reinterpret_cast<const float*>(&y[g]), rd);
  } else {
    const dq::GroupQ gq = dq::mx_group(sc);
#pragma unroll
    for (int g = 0; g < 4; g++) c[g] = dq::fp4_pack<4>(reinterpret_cast<const float*>(&y[g]), gq);
  }
  // after the swaps lane half 0 holds groups 0, 1 of both halves and lane half 1 groups 2, 3
  const auto s0 = __builtin_amdgcn_permlane32_swap(c[0], c[2], false, false);
  const auto s1 = __builtin_amdgcn_permlane32_swap(c[1], c[3], false, false);
  if (!in) return;
  const int64_t off = (int64_t)t * p.out + rb * 32 + 16 * h;
  if (OUT == kOutFp8) {
    *reinterpret_cast<u32x4*>(p.codes + off) =
        u32x4{(uint32_t)s0[0], (uint32_t)s0[1], (uint32_t)s1[0], (uint32_t)s1[1]};
  } else {
    const uint64_t lo = (uint32_t)s0[0] | ((uint32_t)s0[1] << 16);
    const uint64_t hi = (uint32_t)s1[0] | ((uint32_t)s1[1] << 16);
    *reinterpret_cast<uint64_t*>(p.codes + (off >> 1)) = lo | (hi << 32);
  }
  if (h == 0) p.scales[off >> 5] = bad ? 0xFFu : (uint8_t)sc;
}

template <bool GATED>
constexpr int kWaveStaging = 2 * 32 * (128 * (GATED ? 1 : 2) + 16);  // LDS bytes of a wave

template <bool GATED, int NB, int OUT>
__device__ __forceinline__ void tile_store(const MlpArgs& p, const v16f (&acc)[2][NB], int rb0,
                                           int t0, int rows, uint8_t* region) {
  constexpr int ME = GATED ? 1 : 2;       // row blocks of results
  constexpr int LPR = 8 * ME;             // lanes per token row in the read-back
  constexpr int NR = 32 * LPR / 64;       // row accesses of a chunk per lane
  constexpr int kRow = 128 * ME + 16;     // bytes of a staged token row, padded
  const int lane = threadIdx.x & 63, rl = lane & 31, h = lane >> 5;
  const int cl = lane % LPR, rr = lane / LPR;
  const int ich = rb0 * 32 + cl * 4;      // the 4 channels this lane stores
  f32x4 a0[4], a1[4], cb[4];              // gated: factors of the 16 channels of this lane's results
  f32x4 as = {}, bias = {};               // single: of the 4 channels it stores
  if (GATED) {
#pragma unroll
    for (int g = 0; g < 4; g++) {
      const int ch = rb0 * 32 + 8 * g + 4 * h;
      a0[g] = load_channels(p.a[0], ch, p.out, 1.0f);
      a1[g] = load_channels(p.a[1], ch, p.out, 1.0f);
      if (OUT >= kOutFp4) cb[g] = load_channels(p.b, ch, p.out, 1.0f);
    }
  } else {
    as = load_channels(p.a[0], ich, p.out, 1.0f);
    bias = load_channels(p.bias, ich, p.out, 0.0f);
  }
  // rows through buffer accesses relative to the wave's first channel of the tile's first token;
  // rows past the last token lie past the buffer's end, and pieces that the channels do not fill
  // take an offset past it (offsets below 2^31 by kMaxOut, plus kOob below 2^32): such loads read
  // zeros, such stores write nothing
  constexpr int kEs = OUT == kOutF32 ? 4 : 2;
  const int pitch = p.out * kEs;
  const int64_t corner = ((int64_t)t0 * p.out + rb0 * 32) * kEs;
  // (readfirstlane: the compiler takes the clamp for a per-lane value, and each access for a loop
  // over descriptors)
  const uint32_t span = __builtin_amdgcn_readfirstlane(
      (uint32_t)(rows - 1) * (uint32_t)pitch + (uint32_t)min(32 * ME, max(p.out - rb0 * 32, 0)) * kEs);
  const __amdgpu_buffer_rsrc_t ry = rsrc(static_cast<char*>(p.y) + corner, span);
  const bool has_res = !GATED && p.res;
  const __amdgpu_buffer_rsrc_t rr4 = rsrc(static_cast<const char*>(has_res ? p.res : p.y) + corner, span);
  const uint32_t vrow = ich + 3 < p.out ? (uint32_t)rr * (uint32_t)pitch + (uint32_t)(cl * 4 * kEs) : kOob;
  // whether the channels end in this wave's with a piece of 1 .. 3
  const bool ragged = (p.out & 3) && p.out > rb0 * 32 && p.out < (rb0 + ME) * 32;
  typedef typename std::conditional<OUT == kOutF32, u32x4, u32x2>::type raw4;
  typedef typename std::conditional<OUT == kOutF32, float, __bf16>::type T;
  raw4 res[NR];
  auto fetch = [&](int n) {
    if (has_res) {
#pragma unroll
      for (int r = 0; r < NR; r++) {
        const uint32_t vo = vrow + (uint32_t)(n * 32 + r * (64 / LPR)) * (uint32_t)pitch;
        if constexpr (OUT == kOutF32) res[r] = __builtin_amdgcn_raw_buffer_load_b128(rr4, vo, 0, 0);
        else res[r] = __builtin_amdgcn_raw_buffer_load_b64(rr4, vo, 0, 0);
      }
    }
  };
  if constexpr (OUT < kOutFp4) fetch(0);
#pragma unroll
  for (int n = 0; n < NB; n++) {
    __builtin_amdgcn_sched_barrier(0);  // one chunk's registers at a time
    f32x4 y[ME][4];
    if (GATED) {
      with_activation(p.act, [&](auto k) {
#pragma unroll
        for (int g = 0; g < 4; g++)
#pragma unroll
          for (int e = 0; e < 4; e++)
            y[0][g][e] = activation<decltype(k)::value>(acc[0][n][4 * g + e] * a0[g][e]) *
                         (acc[1][n][4 * g + e] * a1[g][e]);
      });
    } else {
#pragma unroll
      for (int m = 0; m < ME; m++)
#pragma unroll
        for (int g = 0; g < 4; g++)
          y[m][g] = f32x4{acc[m][n][4 * g], acc[m][n][4 * g + 1], acc[m][n][4 * g + 2],
                          acc[m][n][4 * g + 3]};
    }
    if constexpr (OUT >= kOutFp4) {
#pragma unroll
      for (int g = 0; g < 4; g++) y[0][g] *= cb[g];
      const int t = t0 + n * 32 + rl;
      quantize_chunk<GATED, OUT>(p, y[0], t, rb0, h, t < p.tokens && rb0 * 32 < p.out);
    } else {
      uint8_t* reg = region + (n & 1) * (32 * kRow);  // two chunks, taken in turn
#pragma unroll
      for (int m = 0; m < ME; m++)
#pragma unroll
        for (int g = 0; g < 4; g++)
          *reinterpret_cast<f32x4*>(reg + rl * kRow + (m * 32 + g * 8 + h * 4) * 4) = y[m][g];
      wave_lds_order();
      if (ragged && rl < rows - n * 32) {  // a row per lane of each half, channel by channel
        for (int ch = (p.out & ~3) + h; ch < p.out; ch += 2) {
          float v = *reinterpret_cast<const float*>(reg + rl * kRow + (ch - rb0 * 32) * 4);
          if (!GATED) {
            v = v * (p.a[0] ? p.a[0][ch] : 1.0f) + (p.bias ? p.bias[ch] : 0.0f);
            with_activation(p.act, [&](auto k) { v = activation<decltype(k)::value>(v); });
          }
          const int64_t off = (int64_t)(t0 + n * 32 + rl) * p.out + ch;
          if (p.res) v = (float)static_cast<const T*>(p.res)[off] + v;
          static_cast<T*>(p.y)[off] = (T)v;
        }
      }
      f32x4 v[NR];
#pragma unroll
      for (int r = 0; r < NR; r++)
        v[r] = *reinterpret_cast<const f32x4*>(reg + (r * (64 / LPR) + rr) * kRow + cl * 16);
      if (!GATED)
        with_activation(p.act, [&](auto k) {
#pragma unroll
          for (int r = 0; r < NR; r++)
#pragma unroll
            for (int e = 0; e < 4; e++)
              v[r][e] = activation<decltype(k)::value>(v[r][e] * as[e] + bias[e]);
        });
      if (has_res) {
#pragma unroll
        for (int r = 0; r < NR; r++) {
          if constexpr (OUT == kOutF32) {
            v[r] = __builtin_bit_cast(f32x4, res[r]) + v[r];
          } else {
            const bf16x4 x = __builtin_bit_cast(bf16x4, res[r]);
#pragma unroll
            for (int e = 0; e < 4; e++) v[r][e] = (float)x[e] + v[r][e];
          }
        }
        if (n + 1 < NB) fetch(n + 1);
      }
#pragma unroll
      for (int r = 0; r < NR; r++) {
        const uint32_t vo = vrow + (uint32_t)(n * 32 + r * (64 / LPR)) * (uint32_t)pitch;
        if constexpr (OUT == kOutF32) {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v[r]), ry, vo, 0, kNt);
        } else {
          const bf16x4 o = {(__bf16)v[r][0], (__bf16)v[r][1], (__bf16)v[r][2], (__bf16)v[r][3]};
          __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, o), ry, vo, 0, kNt);
        }
      }
      wave_lds_order();
    }
  }
}

// Workgroups are dealt round-robin to the eight XCDs, so consecutive ids are spread: each XCD
// gets a contiguous range of tiles, ordered in groups of kGroupM weight tiles by every token
// tile, so that the workgroups running together on one XCD share weights and tokens in its L2.
__device__ __forceinline__ void tile_origin(int nti, int ntt, int& ti, int& tt) {
  const int ntiles = nti * ntt, bid = blockIdx.x;
  const int full = (ntiles / 8) * 8;
  const int L = bid < full ? (bid % 8) * (ntiles / 8) + bid / 8 : bid;
  const int gsz = kGroupM * ntt;
  const int first = (L / gsz) * kGroupM;
  const int gm = min(nti - first, kGroupM);
  ti = first + (L % gsz) % gm;
  tt = (L % gsz) / gm;
}

template <bool ACT8, bool GATED, int NB, int OUT>
__global__ __launch_bounds__(256, 2) void k_mlp_tile(MlpArgs p, int nti, int ntt) {
  // the epilogue stages two 32-token chunks of every wave's channels in the same memory
  constexpr int kStaging = OUT >= kOutFp4 ? 0 : 4 * kWaveStaging<GATED>;
  constexpr int kRings = (int)sizeof(TileLds<NB>);
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kRings > kStaging ? kRings : kStaging];
  constexpr int NK = steps(ACT8);
  constexpr int PER = ACT8 ? 4 : 2;  // stages per period (512 k)
  int ti, tt;
  tile_origin(nti, ntt, ti, tt);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  TileLds<NB>& L = *reinterpret_cast<TileLds<NB>*>(lds);
  const int rl = lane & 31, h = lane >> 5;
  const int t0 = tt * 32 * NB;
  const int rows = min(p.tokens - t0, 32 * NB);
  const int ldb = ACT8 ? p.K : p.K / 2, nkb = p.K / 32, npk = p.K / kStage;
  const int nrb = (p.out + 31) / 32;
  const int rb0 = ti * (GATED ? 4 : 8) + wave * (GATED ? 1 : 2);  // this wave's first row block
  const int periods = p.K / 512;

  TileCtx<ACT8, NB> c;
  c.wave = wave;
  c.nst = PER * periods;
#pragma unroll
  for (int m = 0; m < 2; m++) {
    // a block past the last weight row reads nothing: a descriptor without records
    const int rb = GATED ? rb0 : rb0 + m;
    const bool in = rb < nrb;
    const int64_t at = in ? (int64_t)rb * npk : 0;
    c.rw[m] = rsrc(p.wc[GATED ? m : 0] + at * kPackStageB, in ? (uint32_t)npk * kPackStageB : 0u);
    c.rs[m] = rsrc(p.ws[GATED ? m : 0] + at * kPackScaleB, in ? (uint32_t)npk * kPackScaleB : 0u);
    c.vw[m] = (uint32_t)lane * 16u;
    c.vs[m] = (uint32_t)lane * 4u;
  }
  c.rx = rsrc(p.xc + (int64_t)t0 * ldb, (uint32_t)rows * (uint32_t)ldb);
  c.rxs = rsrc(p.xs + (int64_t)t0 * nkb, (uint32_t)rows * (uint32_t)nkb);
  c.rnone = rsrc(p.xc, 0u);
#pragma unroll
  for (int j = 0; j < NB; j++) {
    // lane l writes piece position l % 8 of row r, which holds the row's piece (l % 8) ^ term
    const int r = 8 * (wave * NB + j) + (lane >> 3);
    const int pc = (lane & 7) ^ (r & 7) ^ ((r >> 3) & 1);
    const uint32_t o = (uint32_t)pc * 16u + (ACT8 && pc >= 4 ? 64u : 0u);
    c.vx[j] = r < rows ? (uint32_t)r * (uint32_t)ldb + o : kOob;
  }
  {
    const int r = wave * 64 + lane;
    c.vxs = r < rows ? (uint32_t)r * (uint32_t)nkb : kOob;
  }

  v16f acc[2][NB];
#pragma unroll
  for (int m = 0; m < 2; m++)
#pragma unroll
    for (int n = 0; n < NB; n++) acc[m][n] = v16f{};

  const int xt = (rl & 7) ^ ((rl >> 3) & 1) ^ (ACT8 ? h : 4 * h);
  const int xrow = rl * kRowB;
  const int xsrow = rl * kScaleRowB + 4 * h;

  u32x4 fa[2][2][NK];              // [stage parity][m][step]: weight fragments
  uint32_t sw[2][2];               // [stage parity][m]: their scale dwords
  u32x4 fb[4][ACT8 ? 2 : 1];       // ring of token fragments
  uint32_t sx[2][NB];              // [stage parity]: token scale dwords

  // stages 0 and 1 and the first period's token scales, in the order that the loop's wait
  // counts on; only stage 0 has to land before the loop
#pragma unroll
  for (int st = 0; st < 2; st++) {
    if (st == 0) load_xs(c, L.xs[0], 0, true);
#pragma unroll
    for (int j = 0; j < NB; j++) load_x(c, L.x[st], j, st, true);
#pragma unroll
    for (int m = 0; m < 2; m++) {
#pragma unroll
      for (int i = 0; i < NK; i++) fa[st][m][i] = load_w(c, m, st, i, true);
      sw[st][m] = load_ws(c, m, st, true);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(2 * NK + 2 + NB));  // stage 1's loads may be in flight
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
#pragma unroll
  for (int n = 0; n < NB; n++)
    sx[0][n] = *reinterpret_cast<const uint32_t*>(L.xs[0] + xsrow + n * 32 * kScaleRowB);
#pragma unroll
  for (int n = 0; n < kAhead; n++)
#pragma unroll
    for (int e = 0; e < (ACT8 ? 2 : 1); e++)
      fb[n][e] = read_x<ACT8>(L.x[0] + xrow + (n % NB) * 32 * kRowB, n / NB, e, xt);

  // stage s of period position J: fragments fa[J % 2], token buffer s % 4, while stage s + 2 loads
  // into the registers it frees and buffer (s + 2) % 4
  auto stage = [&](auto jc, int s, int q, bool more) {
    constexpr int J = decltype(jc)::value, P = J & 1;
    constexpr bool XS = J == 0;
    const uint8_t* lx = L.x[s & 3] + xrow;
    const uint8_t* lxn = L.x[(s + 1) & 3] + xrow;
    uint8_t* xb = L.x[(s + 2) & 3];
    // stage s + 1's token scales: its period, and the half (256 k) of it
    const uint8_t* xsn = L.xs[((s + 1) / PER) & 1] + xsrow + (((J + 1) % PER) / (PER / 2)) * 8;
    uint8_t* xsb = L.xs[(q + 1) & 1];
    auto step = [&](auto kc) {
      constexpr int KS = decltype(kc)::value;
      tile_step<ACT8, NB, KS, P, XS>(acc, fa[P], fb, sw[P], sx[P], sx[P ^ 1], lx, lxn, xsn, xt, c,
                                     xb, xsb, s, q + 1, more);
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    if constexpr (NK == 4) {
      step(std::integral_constant<int, 2>{});
      step(std::integral_constant<int, 3>{});
    }
  };
  for (int q = 0; q < periods; q++) {
    const bool more = q + 1 < periods;
    stage(std::integral_constant<int, 0>{}, PER * q, q, more);
    stage(std::integral_constant<int, 1>{}, PER * q + 1, q, more);
    if constexpr (PER == 4) {
      stage(std::integral_constant<int, 2>{}, PER * q + 2, q, more);
      stage(std::integral_constant<int, 3>{}, PER * q + 3, q, more);
    }
  }
  // the last stages' loads read nothing but still write zeros into LDS: drain them before the
  // epilogue reuses that memory
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
  __syncthreads();  // every wave is done with the main loop's LDS
  uint8_t* region = lds + (OUT >= kOutFp4 ? 0 : wave * kWaveStaging<GATED>);
  tile_store<GATED, NB, OUT>(p, acc, rb0, t0, rows, region);
}

// ---------------------------------------------------------------------------------- host

template <bool ACT8, bool GATED, int OUT, int NB>
hipError_t launch_tile(const MlpArgs& p, hipStream_t s) {
  const int nti = (p.out + (GATED ? 127 : 255)) / (GATED ? 128 : 256);
  const int ntt = (p.tokens + 32 * NB - 1) / (32 * NB);
  hipLaunchKernelGGL((k_mlp_tile<ACT8, GATED, NB, OUT>), dim3((unsigned)(nti * ntt)), dim3(256), 0,
                     s, p, nti, ntt);
  return hipGetLastError();
}

template <bool ACT8, bool GATED, int OUT, int M, int NB>
hipError_t launch_split(const MlpArgs& p, hipStream_t s) {
  constexpr int W = 4;
  const int rows = GATED ? 32 : 32 * M;
  const int64_t nrt = (p.out + rows - 1) / rows, ntt = (p.tokens + 32 * NB - 1) / (32 * NB);
  hipLaunchKernelGGL((k_mlp_split<ACT8, GATED, M, NB, OUT, W>), dim3((unsigned)(nrt * ntt)),
                     dim3(W * 64), 0, s, p);
  return hipGetLastError();
}

// Which kernel, by the number of 32 x 32 blocks of results (row blocks times 32-token blocks).
// With few the split kernel brings the whole chip to bear on k, in the smallest tile (M row
// blocks by NB token blocks) that still fits it in about one round; with more the tile kernel
// reads each operand fewer times, in tiles of 64 tokens as long as those do not fill the chip
// twice over (one a CU), else of 128. A single block of tokens always splits: 8192 -> 28672 at 32
// tokens 29 / 36 us in 64 x 32. Measured, us (MXFP4 / MXFP8 activations, bf16 out), both sides of
// each border:
//   single -> 4096, tokens      64         96         128        160        256        288
//   (blocks)                    256        384        512        640        1024       1152
//   K 512    split 32 x 32      3.8 / 3.9  4.3 / 4.3  4.4 / 4.4  4.9 / 5.0  5.6 / 5.8  6.5 / 6.9
//            split 64 x 32      4.7 / 4.8  4.7 / 4.8  4.7 / 4.9  5.5 / 5.5  5.7 / 5.6  6.6 / 6.3
//            split 64 x 64      6.2 / 6.8  6.2 / 6.8  6.3 / 6.9  6.3 / 6.9  6.5 / 7.0  6.8 / 7.2
//            tile of 64 tokens  5.8 / 5.8  5.8 / 5.8  5.8 / 5.8  5.8 / 5.9  5.9 / 5.9  5.9 / 6.0
//   K 4096   split 32 x 32      5.2 / 7.4  6.8 / 10   7.2 / 11   8.8 / 14   11  / 19   12  / 22
//            split 64 x 32      6.4 / 7.7  6.7 / 7.9  6.8 / 8.3  9.0 / 11   9.5 / 12   12  / 15
//            split 64 x 64      8.3 / 10   8.4 / 10   8.6 / 11   8.6 / 10   8.9 / 12   11  / 15
//            tile of 64 tokens  10  / 13   12  / 14   12  / 15   12  / 14   12  / 15   12  / 14
//   K 14336  split 32 x 32      9.7 / 16   15  / 24   16  / 27   21  / 37   28  / 50   33  / 60
//            split 64 x 32      12  / 18   13  / 18   13  / 19   21  / 30   22  / 33   30  / 45
//            split 64 x 64      17  / 27   16  / 22   17  / 26   17  / 24   18  / 29   26  / 40
//            tile of 64 tokens  30  / 42   29  / 40   31  / 42   29  / 40   30  / 42   29  / 40
//   single -> 4096, tokens (tiles of 64)  512 (128)           1024 (256)          1056 (272)
//   tile of 64, K 512 / 4096 / 14336      6.1  13  31         6.4  17  38         8.0  22  59
//   tile of 128                           8.1  17  40         8.3  18  43         8.3  19  44
//   split 64 x 64                         8.0  13  30         14   23  54         16   26  60
//   gated, blocks (tiles of 64)  2048 -> 5632: 704 (88), 880 (132)   4096 -> 14336: 448, 896 (112)
//     split                      9.3 / 10, 11 / 12                   13 / 14, 21 / 24
//     tile of 64                 8.9 / 10, 9.0 / 10                  -, 14 / 17
//     .. (tiles of 64)           2048 -> 5632: 220, 264              4096 -> 14336: 224, 336
//     tile of 64                 11 / 11, 14 / 17                    15 / 18, 25 / 29
//     tile of 128                12 / 14, 12 / 15                    18 / 23, 22 / 25
// The borders are K 4096's. Elsewhere another kernel is up to a quarter faster near them: for K
// up to 1024 the smaller split tiles between 257 and 1024 blocks (160 tokens, K 512: 4.9 against
// 6.3), at K 14336 the 64 x 64 split tile just past 1024 (288 tokens, MXFP4: 26 against 29), for
// the gated product 32 x 64 split tiles at K 8192 -> 2816 with 128 tokens (11 against 13), which
// are not built for it; nor are 64 x 128 ones for the single product (14336 -> 4096, 512 tokens:
// 28 / 48 against 31 / 43).
template <bool ACT8, bool GATED, int OUT>
hipError_t launch_t(const MlpArgs& p, hipStream_t s) {
  const int64_t nrb = (p.out + 31) / 32, ntb = (p.tokens + 31) / 32, blocks = nrb * ntb;
  if constexpr (GATED) {
    if (blocks <= 704 || ntb == 1) return launch_split<ACT8, true, OUT, 2, 1>(p, s);
  } else {
    if (blocks <= 256) return launch_split<ACT8, false, OUT, 1, 1>(p, s);
    if (blocks <= 512 || ntb == 1) return launch_split<ACT8, false, OUT, 2, 1>(p, s);
    if (blocks <= 1024) return launch_split<ACT8, false, OUT, 2, 2>(p, s);
  }
  constexpr int kRows = GATED ? 4 : 8;
  const int64_t tiles64 = ((nrb + kRows - 1) / kRows) * ((ntb + 1) / 2);
  if (tiles64 <= 256) return launch_tile<ACT8, GATED, OUT, 2>(p, s);
  return launch_tile<ACT8, GATED, OUT, 4>(p, s);
}

// Bytes of n elements of an output
size_t out_bytes(int o, int64_t n) {
  return o == kOutFp4 ? (size_t)n / 2 : (size_t)n * (o == kOutF32 ? 4 : o == kOutBf16 ? 2 : 1);
}

// Launches over chunks of tokens so that no grid passes 2^31 threads (one launch for all but
// millions of tokens); the arrays' offsets are 64-bit here and relative to a tile in the kernels.
template <bool GATED, int OUT>
hipError_t launch_o(const MlpArgs& whole, bool act8, hipStream_t s) {
  const int64_t nrb = (whole.out + 31) / 32;
  const int64_t chunk = std::max<int64_t>(256, ((int64_t)1 << 21) / nrb * 32 / 256 * 256);
  for (int64_t t = 0; t < whole.tokens; t += chunk) {
    MlpArgs p = whole;
    p.tokens = (int)std::min<int64_t>(chunk, whole.tokens - t);
    p.xc += t * (act8 ? p.K : p.K / 2);
    p.xs += t * (p.K / 32);
    const size_t off = out_bytes(OUT, t * p.out);
    if (p.res) p.res = static_cast<const char*>(p.res) + off;
    if (OUT >= kOutFp4) {
      p.codes += off;
      p.scales += t * (p.out / 32);
    } else {
      p.y = static_cast<char*>(p.y) + off;
    }
    hipError_t e = hipErrorInvalidValue;
    if (!act8) e = launch_t<false, GATED, OUT>(p, s);
    else if constexpr (OUT != kOutF32) e = launch_t<true, GATED, OUT>(p, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// The checks that the products share. Sizes first: they bound the rest.
dq_status check_product(const void* xc, const void* xs, dq_format act_fmt, int64_t tokens,
                        int64_t K, const void* wc, const void* ws, const void* a, int64_t out,
                        dq_activation act) {
  if (act_fmt != DQ_FMT_MXFP4 && act_fmt != DQ_FMT_MXFP8) return DQ_ERR_UNSUPPORTED;
  if ((int)act < 0 || (int)act > DQ_ACTIVATION_GELU_TANH) return DQ_ERR_UNSUPPORTED;
  if (!xc || !xs || !wc || !ws) return DQ_ERR_ARG;
  if (tokens < 1 || out < 1 || K < 512 || K % 512 != 0 || K > (1 << 22)) return DQ_ERR_ARG;
  if (tokens > INT32_MAX - 256 || out > kMaxOut) return DQ_ERR_ARG;
  if (((uintptr_t)xc | (uintptr_t)xs | (uintptr_t)wc | (uintptr_t)a) & 15u) return DQ_ERR_ARG;
  if ((uintptr_t)ws & 3u) return DQ_ERR_ARG;
  return DQ_OK;
}

// The bytes of a product's operands
size_t act_bytes(dq_format fmt, int64_t tokens, int64_t K) {
  return (size_t)tokens * (size_t)(fmt == DQ_FMT_MXFP8 ? K : K / 2);
}
size_t packed_bytes(int64_t out, int64_t K) { return (size_t)((out + 31) / 32) * 16 * (size_t)K; }

}  // namespace dqm

extern "C" {

dq_status dq_gemm_mx_epilogue(const uint8_t* act_codes, const uint8_t* act_scales,
                              dq_format act_fmt, int64_t tokens, int64_t K,
                              const uint8_t* packed_codes, const uint8_t* packed_scales,
                              const float* a, const float* bias, dq_activation activation,
                              const void* residual, int64_t out, dq_dtype yt, void* Y,
                              hipStream_t stream) {
  using namespace dqm;
  const dq_status st = check_product(act_codes, act_scales, act_fmt, tokens, K, packed_codes,
                                     packed_scales, a, out, activation);
  if (st != DQ_OK) return st;
  if ((yt != DQ_F32 && yt != DQ_BF16) || (yt == DQ_F32 && act_fmt == DQ_FMT_MXFP8))
    return DQ_ERR_UNSUPPORTED;
  const size_t esz = yt == DQ_BF16 ? 2 : 4;
  if (!Y || ((uintptr_t)bias & 15u) || (((uintptr_t)Y | (uintptr_t)residual) & (esz - 1)))
    return DQ_ERR_ARG;
  const size_t bytes = (size_t)tokens * (size_t)out * esz;
  const size_t wb = packed_bytes(out, K), vb = (size_t)out * 4;
  if (dq::any_overlap({{Y, bytes}},
                      {{residual == Y ? nullptr : residual, bytes},
                       {act_codes, act_bytes(act_fmt, tokens, K)},
                       {act_scales, (size_t)(tokens * (K / 32))},
                       {packed_codes, wb},
                       {packed_scales, wb / 16},
                       {a, vb},
                       {bias, vb}}))
    return DQ_ERR_ARG;
  MlpArgs p{};
  p.xc = act_codes;
  p.xs = act_scales;
  p.wc[0] = packed_codes;
  p.ws[0] = packed_scales;
  p.a[0] = a;
  p.bias = bias;
  p.res = residual;
  p.y = Y;
  p.tokens = (int)tokens;
  p.out = (int)out;
  p.K = (int)K;
  p.act = activation;
  const bool act8 = act_fmt == DQ_FMT_MXFP8;
  const hipError_t e = yt == DQ_BF16 ? launch_o<false, kOutBf16>(p, act8, stream)
                                     : launch_o<false, kOutF32>(p, false, stream);
  return e == hipSuccess ? DQ_OK : DQ_ERR_HIP;
}

dq_status dq_gated_mx(const uint8_t* act_codes, const uint8_t* act_scales, dq_format act_fmt,
                      int64_t tokens, int64_t K, const uint8_t* gate_codes,
                      const uint8_t* gate_scales, const float* a_gate, const uint8_t* up_codes,
                      const uint8_t* up_scales, const float* a_up, dq_activation activation,
                      int64_t inner, dq_dtype yt, void* H, hipStream_t stream) {
  using namespace dqm;
  dq_status st = check_product(act_codes, act_scales, act_fmt, tokens, K, gate_codes, gate_scales,
                               a_gate, inner, activation);
  if (st == DQ_OK)
    st = check_product(act_codes, act_scales, act_fmt, tokens, K, up_codes, up_scales, a_up, inner,
                       activation);
  if (st != DQ_OK) return st;
  if ((yt != DQ_F32 && yt != DQ_BF16) || (yt == DQ_F32 && act_fmt == DQ_FMT_MXFP8))
    return DQ_ERR_UNSUPPORTED;
  const size_t esz = yt == DQ_BF16 ? 2 : 4;
  if (!H || ((uintptr_t)H & (esz - 1))) return DQ_ERR_ARG;
  const size_t wb = packed_bytes(inner, K), vb = (size_t)inner * 4;
  if (dq::any_overlap({{H, (size_t)tokens * (size_t)inner * esz}},
                      {{act_codes, act_bytes(act_fmt, tokens, K)},
                       {act_scales, (size_t)(tokens * (K / 32))},
                       {gate_codes, wb},
                       {gate_scales, wb / 16},
                       {up_codes, wb},
                       {up_scales, wb / 16},
                       {a_gate, vb},
                       {a_up, vb}}))
    return DQ_ERR_ARG;
  MlpArgs p{};
  p.xc = act_codes;
  p.xs = act_scales;
  p.wc[0] = gate_codes;
  p.wc[1] = up_codes;
  p.ws[0] = gate_scales;
  p.ws[1] = up_scales;
  p.a[0] = a_gate;
  p.a[1] = a_up;
  p.y = H;
  p.tokens = (int)tokens;
  p.out = (int)inner;
  p.K = (int)K;
  p.act = activation;
  const bool act8 = act_fmt == DQ_FMT_MXFP8;
  const hipError_t e = yt == DQ_BF16 ? launch_o<true, kOutBf16>(p, act8, stream)
                                     : launch_o<true, kOutF32>(p, false, stream);
  return e == hipSuccess ? DQ_OK : DQ_ERR_HIP;
}

dq_status dq_gated_mx_quantized(const uint8_t* act_codes, const uint8_t* act_scales,
                                dq_format act_fmt, int64_t tokens, int64_t K,
                                const uint8_t* gate_codes, const uint8_t* gate_scales,
                                const float* a_gate, const uint8_t* up_codes,
                                const uint8_t* up_scales, const float* a_up,
                                dq_activation activation, int64_t inner, const float* b,
                                dq_format fmt, uint8_t* codes, uint8_t* scales,
                                hipStream_t stream) {
  using namespace dqm;
  dq_status st = check_product(act_codes, act_scales, act_fmt, tokens, K, gate_codes, gate_scales,
                               a_gate, inner, activation);
  if (st == DQ_OK)
    st = check_product(act_codes, act_scales, act_fmt, tokens, K, up_codes, up_scales, a_up, inner,
                       activation);
  if (st != DQ_OK) return st;
  if (fmt != DQ_FMT_MXFP4 && fmt != DQ_FMT_MXFP8) return DQ_ERR_UNSUPPORTED;
  if (!codes || !scales || inner % 32 != 0) return DQ_ERR_ARG;
  if (((uintptr_t)codes | (uintptr_t)b) & 15u) return DQ_ERR_ARG;
  const size_t wb = packed_bytes(inner, K), vb = (size_t)inner * 4;
  if (dq::any_overlap({{codes, act_bytes(fmt, tokens, inner)},
                       {scales, (size_t)(tokens * (inner / 32))}},
                      {{act_codes, act_bytes(act_fmt, tokens, K)},
                       {act_scales, (size_t)(tokens * (K / 32))},
                       {gate_codes, wb},
                       {gate_scales, wb / 16},
                       {up_codes, wb},
                       {up_scales, wb / 16},
                       {a_gate, vb},
                       {a_up, vb},
                       {b, vb}}))
    return DQ_ERR_ARG;
  MlpArgs p{};
  p.xc = act_codes;
  p.xs = act_scales;
  p.wc[0] = gate_codes;
  p.wc[1] = up_codes;
  p.ws[0] = gate_scales;
  p.ws[1] = up_scales;
  p.a[0] = a_gate;
  p.a[1] = a_up;
  p.b = b;
  p.codes = codes;
  p.scales = scales;
  p.tokens = (int)tokens;
  p.out = (int)inner;
  p.K = (int)K;
  p.act = activation;
  const bool act8 = act_fmt == DQ_FMT_MXFP8;
  const hipError_t e = fmt == DQ_FMT_MXFP8 ? launch_o<true, kOutFp8>(p, act8, stream)
                                           : launch_o<true, kOutFp4>(p, act8, stream);
  return e == hipSuccess ? DQ_OK : DQ_ERR_HIP;
}

}  // extern "C"
