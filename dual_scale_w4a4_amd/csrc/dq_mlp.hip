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
// In its 8-bit mode the instruction aligns the products of each lane's run of 16 k to 2^-13 of
// the largest; FP4 products are added exactly and accumulated in fp32.
#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/dq_mlp.h"
#include "dq_outq.h"

namespace dqm {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

constexpr int kStage = 256;           // k values per packed stage
constexpr int kPackStepB = 1024;      // packed codes of (row block, stage, step)
constexpr int kPackStageB = 4096;     // packed codes of (row block, stage)
constexpr int kPackScaleB = 256;      // packed scales of (row block, stage)
constexpr uint32_t kBufRsrcWord3 = 0x00020000u;  // raw buffer, 32-bit data format
constexpr uint32_t kOob = 0x80000000u;           // an offset past every buffer: reads zero

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
  bool vec;              // whole 4-channel accesses: out % 4 == 0 and aligned arrays
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes,
                                           (int)kBufRsrcWord3);
}

// ---------------------------------------------------------------------------- activations

__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
}

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case DQ_ACTIVATION_RELU: return z < 0.0f ? 0.0f : z;  // a NaN stays one
    case DQ_ACTIVATION_SILU: return z * sigmoid(z);
    case DQ_ACTIVATION_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    case DQ_ACTIVATION_GELU_TANH:  // (1 + tanh u) / 2 = sigmoid(2 u)
      return z * sigmoid(1.5957691216057308f * (z + 0.044715f * z * z * z));
    default: return z;
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

// The factors of 4 channels, kept for every token a lane finishes.
struct Chan {
  f32x4 a0, a1, c;  // row scales; bias (single), column scales (quantized)
};

template <bool GATED, int OUT>
__device__ __forceinline__ Chan load_chan(const MlpArgs& p, int ich) {
  Chan c;
  c.a0 = load_channels(p.a[0], ich, p.out, 1.0f);
  if (GATED) c.a1 = load_channels(p.a[1], ich, p.out, 1.0f);
  if (!GATED) c.c = load_channels(p.bias, ich, p.out, 0.0f);
  if (OUT >= kOutFp4) c.c = load_channels(p.b, ich, p.out, 1.0f);
  return c;
}

// Finish channels ich .. ich + 3 of token t from the raw sums s0 (and s1) and store them. For a
// quantized output the 8 lanes of an aligned group of 8 hold the 32 channels of one scale
// group of one token, and all are here with the same t.
template <bool GATED, int OUT>
__device__ __forceinline__ void finish(const MlpArgs& p, int64_t t, int ich, const Chan& c,
                                       f32x4 s0, f32x4 s1) {
  f32x4 y;
#pragma unroll
  for (int e = 0; e < 4; e++) {
    const float z = s0[e] * c.a0[e];
    if (GATED)
      y[e] = activate(z, p.act) * (s1[e] * c.a1[e]);
    else
      y[e] = activate(z + c.c[e], p.act);
  }
  const int64_t off = t * p.out + ich;
  if (OUT >= kOutFp4) {
    float x[4];
    uint32_t mb = 0u;
#pragma unroll
    for (int e = 0; e < 4; e++) {
      x[e] = y[e] * c.c[e];
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
    if (ich < p.out) {
      if (OUT == kOutFp8) {
        *reinterpret_cast<uint32_t*>(p.codes + off) =
            dq::fp8_pack4(x, dq::u2f((254u - sc) << 23));
      } else {
        *reinterpret_cast<uint16_t*>(p.codes + (off >> 1)) =
            (uint16_t)dq::fp4_pack<4>(x, dq::mx_group(sc));
      }
      if ((threadIdx.x & 7) == 0) p.scales[off >> 5] = bad ? 0xFFu : (uint8_t)sc;
    }
    return;
  }
  const bool vec = p.vec && ich < p.out;  // then all 4 channels exist
  if (OUT == kOutBf16) {
    __bf16* yp = static_cast<__bf16*>(p.y) + off;
    if (!GATED && p.res) {
      const __bf16* rp = static_cast<const __bf16*>(p.res) + off;
      if (vec) {
        const bf16x4 r = *reinterpret_cast<const bf16x4*>(rp);
#pragma unroll
        for (int e = 0; e < 4; e++) y[e] = (float)r[e] + y[e];
      } else {
#pragma unroll
        for (int e = 0; e < 4; e++)
          if (ich + e < p.out) y[e] = (float)rp[e] + y[e];
      }
    }
    const bf16x4 hv = {(__bf16)y[0], (__bf16)y[1], (__bf16)y[2], (__bf16)y[3]};
    if (vec) {
      *reinterpret_cast<bf16x4*>(yp) = hv;
    } else {
#pragma unroll
      for (int e = 0; e < 4; e++)
        if (ich + e < p.out) yp[e] = hv[e];
    }
  } else {
    float* yp = static_cast<float*>(p.y) + off;
    if (!GATED && p.res) {
      const float* rp = static_cast<const float*>(p.res) + off;
      if (vec) {
        y = *reinterpret_cast<const f32x4*>(rp) + y;
      } else {
#pragma unroll
        for (int e = 0; e < 4; e++)
          if (ich + e < p.out) y[e] = rp[e] + y[e];
      }
    }
    if (vec) {
      *reinterpret_cast<f32x4*>(yp) = y;
    } else {
#pragma unroll
      for (int e = 0; e < 4; e++)
        if (ich + e < p.out) yp[e] = y[e];
    }
  }
}

// ------------------------------------------------------------------- split-k kernel
// A workgroup owns MB row blocks (the product's, or the gate's and the up weights' block of the
// same 32 channels) and NB blocks of 32 tokens; its W waves share the stages of k between
// them (wave w takes stages w, w + W, ..), every operand going from memory straight to
// registers, and their partial sums are joined in LDS in wave order.

// One stage's operands of a wave.
template <bool ACT8, int MB, int NB>
struct Frags {
  u32x4 a[MB][4];
  uint32_t sa[MB];
  u32x4 b[NB][ACT8 ? 8 : 4];
  uint32_t sb[NB];
};

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

// LDS row of one token's 32 partial sums, padded so that 8 rows cover distinct banks
constexpr int kPartRow = 36;
constexpr int kPartBlock = 32 * kPartRow;  // floats of one 32 x 32 block

template <bool ACT8, bool GATED, int NB, int OUT, int W>
__global__ __launch_bounds__(W * 64) void k_mlp_split(MlpArgs p) {
  constexpr int MB = GATED ? 2 : 1;
  __shared__ __attribute__((aligned(16))) float part[W * MB * kPartBlock];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rl = lane & 31, h = lane >> 5;
  const int nrb = (p.out + 31) / 32;
  const int rb = blockIdx.x % nrb;                // row block
  const int t0 = (blockIdx.x / nrb) * (32 * NB);
  const int ldb = ACT8 ? p.K : p.K / 2, nkb = p.K / 32, nst = p.K / kStage;
  const int rows = min(p.tokens - t0, 32 * NB);

  __amdgpu_buffer_rsrc_t rw[MB], rs[MB];
#pragma unroll
  for (int m = 0; m < MB; m++) {
    rw[m] = rsrc(p.wc[m] + (int64_t)rb * nst * kPackStageB, (uint32_t)nst * kPackStageB);
    rs[m] = rsrc(p.ws[m] + (int64_t)rb * nst * kPackScaleB, (uint32_t)nst * kPackScaleB);
  }
  const __amdgpu_buffer_rsrc_t rx = rsrc(p.xc + (int64_t)t0 * ldb, (uint32_t)rows * (uint32_t)ldb);
  const __amdgpu_buffer_rsrc_t rxs = rsrc(p.xs + (int64_t)t0 * nkb, (uint32_t)rows * (uint32_t)nkb);
  uint32_t vx[NB], vs[NB];
#pragma unroll
  for (int n = 0; n < NB; n++) {
    const int r = n * 32 + rl;
    vx[n] = r < rows ? (uint32_t)r * (uint32_t)ldb + (ACT8 ? 16u : 64u) * (uint32_t)h : kOob;
    vs[n] = r < rows ? (uint32_t)r * (uint32_t)nkb + 4u * (uint32_t)h : kOob;
  }

  v16f acc[MB][NB];
#pragma unroll
  for (int m = 0; m < MB; m++)
#pragma unroll
    for (int n = 0; n < NB; n++) acc[m][n] = v16f{};

  for (int s = wave; s < nst; s += W) {
    Frags<ACT8, MB, NB> f;
#pragma unroll
    for (int m = 0; m < MB; m++) {
#pragma unroll
      for (int i = 0; i < 4; i++)
        f.a[m][i] = __builtin_amdgcn_raw_buffer_load_b128(
            rw[m], (uint32_t)lane * 16u, (uint32_t)(s * kPackStageB + i * kPackStepB), 0);
      f.sa[m] = __builtin_amdgcn_raw_buffer_load_b32(rs[m], (uint32_t)lane * 4u,
                                                     (uint32_t)(s * kPackScaleB), 0);
    }
#pragma unroll
    for (int n = 0; n < NB; n++) {
#pragma unroll
      for (int i = 0; i < (ACT8 ? 8 : 4); i++) {
        // FP4: the lane's four chunks; FP8: 16 bytes of chunk i / 2 of either half
        const uint32_t o = ACT8 ? (uint32_t)(s * 256 + (i / 2) * 32 + (i % 2) * 128)
                                : (uint32_t)(s * 128 + i * 16);
        f.b[n][i] = __builtin_amdgcn_raw_buffer_load_b128(rx, vx[n], o, 0);
      }
      f.sb[n] = __builtin_amdgcn_raw_buffer_load_b32(rxs, vs[n], (uint32_t)(s * 8), 0);
    }
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int m = 0; m < MB; m++)
#pragma unroll
        for (int n = 0; n < NB; n++)
          acc[m][n] = mfma<ACT8>(f.a[m][i], &f.b[n][ACT8 ? 2 * i : i], acc[m][n], f.sa[m], f.sb[n], i);
  }

  // join: block (m, n) of every wave as rows of tokens, then thread x adds the W partial sums
  // of 4 channels of one token in wave order
#pragma unroll
  for (int n = 0; n < NB; n++) {
    if (n > 0) __syncthreads();
#pragma unroll
    for (int m = 0; m < MB; m++)
#pragma unroll
      for (int g = 0; g < 4; g++)
        *reinterpret_cast<f32x4*>(part + (wave * MB + m) * kPartBlock + rl * kPartRow + g * 8 + h * 4) =
            f32x4{acc[m][n][g * 4], acc[m][n][g * 4 + 1], acc[m][n][g * 4 + 2], acc[m][n][g * 4 + 3]};
    __syncthreads();
    for (int x = threadIdx.x; x < 256; x += W * 64) {
      const int tr = x >> 3, ch = (x & 7) * 4;
      f32x4 s[2] = {f32x4{}, f32x4{}};
#pragma unroll
      for (int m = 0; m < MB; m++)
#pragma unroll
        for (int w = 0; w < W; w++)
          s[m] += *reinterpret_cast<const f32x4*>(part + (w * MB + m) * kPartBlock + tr * kPartRow + ch);
      const int t = t0 + n * 32 + tr, ich = rb * 32 + ch;
      if (t < p.tokens)
        finish<GATED, OUT>(p, t, ich, load_chan<GATED, OUT>(p, ich), s[0], s[1]);
    }
  }
}

// ---------------------------------------------------------------------------------- host

template <bool ACT8, bool GATED, int OUT>
hipError_t launch_t(const MlpArgs& p, hipStream_t s) {
  constexpr int NB = 1, W = 8;
  const int64_t nrb = (p.out + 31) / 32, ntt = (p.tokens + 32 * NB - 1) / (32 * NB);
  hipLaunchKernelGGL((k_mlp_split<ACT8, GATED, NB, OUT, W>), dim3((unsigned)(nrb * ntt)),
                     dim3(W * 64), 0, s, p);
  return hipGetLastError();
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

bool overlap(const void* p, size_t pb, const void* q, size_t qb) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return a < b + qb && b < a + pb;
}

// The checks that the products share. Sizes first: they bound the rest.
dq_status check_product(const void* xc, const void* xs, dq_format act_fmt, int64_t tokens,
                        int64_t K, const void* wc, const void* ws, const void* a, int64_t out,
                        dq_activation act) {
  if (act_fmt != DQ_FMT_MXFP4 && act_fmt != DQ_FMT_MXFP8) return DQ_ERR_UNSUPPORTED;
  if ((int)act < 0 || (int)act > DQ_ACTIVATION_GELU_TANH) return DQ_ERR_UNSUPPORTED;
  if (!xc || !xs || !wc || !ws) return DQ_ERR_ARG;
  if (tokens < 1 || out < 1 || K < 512 || K % 512 != 0 || K > (1 << 22)) return DQ_ERR_ARG;
  if (tokens > INT32_MAX - 256 || out > INT32_MAX - 256) return DQ_ERR_ARG;
  if (((uintptr_t)xc | (uintptr_t)xs | (uintptr_t)wc | (uintptr_t)a) & 15u) return DQ_ERR_ARG;
  if ((uintptr_t)ws & 3u) return DQ_ERR_ARG;
  return DQ_OK;
}

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
  if (residual && residual != Y && overlap(residual, bytes, Y, bytes)) return DQ_ERR_ARG;
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
  p.vec = out % 4 == 0 && (((uintptr_t)Y | (uintptr_t)residual) & (4 * esz - 1)) == 0;
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
  p.vec = inner % 4 == 0 && ((uintptr_t)H & (4 * esz - 1)) == 0;
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
