// dq_norm.hip -- residual addition, root-mean-square norm, column scales and the group
// quantizer in one kernel: what stands between a decoder layer's residual stream and its
// quantized products.
//
//   h = round_xt(X + R) (stored), r = fl32(1 / sqrt(mean h^2 + eps)),
//   x = fl32(fl32(fl32(h r) w) b), then Q in groups of G channels.
//
// The codes have to be those of the definition bit for bit (a code next to a border moves
// with the last bit of x), so every step of x is one fp32 rounding, and the sum of squares and
// the root are taken in fp64: their error (below 2^-45) moves fl32(r) only where 1 / sqrt lies
// that close to a midpoint of two fp32 values.
//
// A workgroup owns one row. Lane l of chunk c holds the 16 consecutive channels
// 4096 c + 16 l ..; the first sweep forms and stores h and its squares, the second reads h
// back and quantizes.
#include <float.h>
#include <math.h>

#include "../../include/dq_mlp.h"
#include "dq_outq.h"

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

namespace dq {

constexpr int kNormEpl = 16;  // consecutive channels per lane

struct NormArgs {
  const void* X;
  const void* R;      // or null
  void* h;            // R + X, or null
  const void* w;      // channels, or null
  const float* b;     // channels, or null
  int64_t m, n;
  double eps;
  float g;            // NVFP4
  uint8_t* codes;
  void* scales;
  int* status;
  bool wbf;           // w is bf16
};

// 16 values of a bf16 or fp32 array
template <bool BF>
__device__ __forceinline__ void load16(const void* p, int64_t off, float (&v)[kNormEpl]) {
  if (BF) {
    const u32x4* s = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + off);
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const u32x4 u = s[k];
#pragma unroll
      for (int e = 0; e < 4; e++) {
        v[8 * k + 2 * e] = u2f(u[e] << 16);
        v[8 * k + 2 * e + 1] = u2f(u[e] & 0xFFFF0000u);
      }
    }
  } else {
    const u32x4* s = reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + off);
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const u32x4 u = s[k];
#pragma unroll
      for (int e = 0; e < 4; e++) v[4 * k + e] = u2f(u[e]);
    }
  }
}

// nearest bf16 (ties to even) of any fp32 value, as fp32
__device__ __forceinline__ float to_bf16(float x) { return (float)(__bf16)x; }

template <bool BF>
__device__ __forceinline__ void store16(void* p, int64_t off, const float (&v)[kNormEpl]) {
  if (BF) {
    u32x4* d = reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + off);
#pragma unroll
    for (int k = 0; k < 2; k++) {
      u32x4 u;
#pragma unroll
      for (int e = 0; e < 4; e++)
        u[e] = (f2u(v[8 * k + 2 * e]) >> 16) | (f2u(v[8 * k + 2 * e + 1]) & 0xFFFF0000u);
      d[k] = u;
    }
  } else {
    u32x4* d = reinterpret_cast<u32x4*>(static_cast<float*>(p) + off);
#pragma unroll
    for (int k = 0; k < 4; k++)
      d[k] = u32x4{f2u(v[4 * k]), f2u(v[4 * k + 1]), f2u(v[4 * k + 2]), f2u(v[4 * k + 3])};
  }
}

// Codes and scale of one lane's 16 values (all finite; the group of G values lies in G / 16
// neighbouring lanes) at element offset off of the outputs. `act`: whether the lane's
// channels exist (the group's lanes agree; all lanes of the wave take part in the maxima).
template <int FMT, int G>
__device__ __forceinline__ void quantize16(const float (&x)[kNormEpl], float mx, bool act,
                                           const NormArgs& p, int64_t off, float sixg) {
  constexpr int LPG = G / kNormEpl;
  const uint32_t gmb = LPG > 1 ? group_max_bits<LPG>(f2u(mx)) : f2u(mx);
  uint32_t scode;
  if (FMT == kMxFp8) {
    scode = mx_scale_code<8>(gmb);
    const float rd = u2f((254u - scode) << 23);
    const u32x4 c = {fp8_pack4(x, rd), fp8_pack4(x + 4, rd), fp8_pack4(x + 8, rd),
                     fp8_pack4(x + 12, rd)};
    if (act) *reinterpret_cast<u32x4*>(p.codes + off) = c;
  } else {
    u32x2 c;
    if (FMT == kMxFp4) {
      scode = mx_scale_code<2>(gmb);
      const GroupQ gq = mx_group(scode);
      c = u32x2{fp4_pack<8>(x, gq), fp4_pack<8>(x + 8, gq)};
    } else {
      // the exact rules of dq_device.h: the power-of-two quotient for MXINT4, the snapped
      // double quotient for INT4 and NVFP4
      const GroupQ gq = group_scale<FMT == kMxFp8 ? kMxInt4 : FMT>(u2f(gmb), p.g, sixg);
      constexpr int F = FMT == kMxFp8 ? kMxInt4 : FMT;
      const double r = F == kMxInt4 ? 0.0 : recip64(gq.d);
      scode = gq.scode;
#pragma unroll
      for (int k = 0; k < 2; k++) {
        uint32_t pk = 0u;
#pragma unroll
        for (int e = 0; e < 8; e++) {
          double q = code64<F>(x[8 * k + e], r, gq);
          if (F == kInt4Bf16) q = int4_clamp(q);
          pk |= nibble_of<F>((float)q) << (4 * e);
        }
        c[k] = pk;
      }
    }
    if (act) *reinterpret_cast<u32x2*>(p.codes + (off >> 1)) = c;
  }
  if (act && (LPG == 1 || (threadIdx.x % LPG) == 0)) {
    const int64_t si = off / G;  // rows hold whole groups
    if (FMT == kInt4Bf16)
      static_cast<uint16_t*>(p.scales)[si] = (uint16_t)scode;
    else
      static_cast<uint8_t*>(p.scales)[si] = (uint8_t)scode;
  }
}

template <int FMT, int G, bool BF>
__global__ __launch_bounds__(kBlock) void k_norm(NormArgs p) {
  __shared__ double red[kWaves];
  const int64_t row = (int64_t)blockIdx.x * p.n;
  int flags = 0;
  double sum = 0.0;
  for (int64_t c = threadIdx.x * kNormEpl; c < p.n; c += kBlock * kNormEpl) {
    float h[kNormEpl];
    load16<BF>(p.X, row + c, h);
    if (p.R) {
      float r[kNormEpl];
      load16<BF>(p.R, row + c, r);
      float in = 0.0f, out = 0.0f;
#pragma unroll
      for (int k = 0; k < kNormEpl; k++) {
        in = fmaf(h[k], 0.0f, fmaf(r[k], 0.0f, in));  // NaN once an input is not finite
        h[k] += r[k];
        if (BF) h[k] = to_bf16(h[k]);
        out = fmaf(h[k], 0.0f, out);
      }
      if (in != 0.0f) flags |= kStNonFinite;
      else if (out != 0.0f) flags |= kStRange;
      store16<BF>(p.h, row + c, h);
    } else {
      float in = 0.0f;
#pragma unroll
      for (int k = 0; k < kNormEpl; k++) in = fmaf(h[k], 0.0f, in);
      if (in != 0.0f) flags |= kStNonFinite;
    }
#pragma unroll
    for (int k = 0; k < kNormEpl; k++) sum = fma((double)h[k], (double)h[k], sum);
  }
  sum = block_sum4(sum, red);
  const float rstd = (float)(1.0 / sqrt(sum / (double)p.n + p.eps));
  const float sixg = 6.0f * p.g;
  const void* src = p.R ? p.h : p.X;
  // every lane of a wave runs the same trips (the group maxima exchange lanes); lanes past the
  // row's end read its start and store nothing
  for (int64_t c0 = 0; c0 < p.n; c0 += kBlock * kNormEpl) {
    const int64_t c = c0 + threadIdx.x * kNormEpl;
    const bool act = c < p.n;
    const int64_t lc = act ? c : 0;
    float x[kNormEpl], w[kNormEpl];
    load16<BF>(src, row + lc, x);
#pragma unroll
    for (int k = 0; k < kNormEpl; k++) x[k] *= rstd;
    if (p.w) {
      if (p.wbf) load16<true>(p.w, lc, w);
      else load16<false>(p.w, lc, w);
#pragma unroll
      for (int k = 0; k < kNormEpl; k++) x[k] *= w[k];
    }
    if (p.b) {
      load16<false>(p.b, lc, w);
#pragma unroll
      for (int k = 0; k < kNormEpl; k++) x[k] *= w[k];
    }
    float mx = 0.0f, chk = 0.0f;
#pragma unroll
    for (int k = 0; k < kNormEpl; k++) {
      mx = fmaxf(mx, fabsf(x[k]));
      chk = fmaf(x[k], 0.0f, chk);
    }
    if (chk != 0.0f) {  // not finite: a bad h in the row (reported above) or an overflow
      if (fabs(sum) <= DBL_MAX) flags |= kStRange;
      mx = 0.0f;
#pragma unroll
      for (int k = 0; k < kNormEpl; k++) x[k] = 0.0f;
    }
    quantize16<FMT, G>(x, mx, act, p, row + lc, sixg);
  }
  if (flags) atomicOr(p.status, flags);
}

template <int FMT, int G>
static hipError_t norm_launch(bool bf16, const NormArgs& p, hipStream_t s) {
  const dim3 grid((unsigned)p.m);
  if (bf16)
    hipLaunchKernelGGL((k_norm<FMT, G, true>), grid, dim3(kBlock), 0, s, p);
  else
    hipLaunchKernelGGL((k_norm<FMT, G, false>), grid, dim3(kBlock), 0, s, p);
  return hipGetLastError();
}

template <int FMT>
static hipError_t norm_group(int G, bool bf16, const NormArgs& p, hipStream_t s) {
  switch (G) {
    case 16: return norm_launch<FMT, 16>(bf16, p, s);
    case 32: return norm_launch<FMT, 32>(bf16, p, s);
    case 64: return norm_launch<FMT, 64>(bf16, p, s);
    default: return hipErrorInvalidValue;
  }
}

// Launches over chunks of rows so that no grid passes 2^31 threads.
static hipError_t launch_norm(int fmt, int G, bool bf16, const NormArgs& whole, hipStream_t s) {
  constexpr int64_t kRows = 1 << 22;
  for (int64_t t = 0; t < whole.m; t += kRows) {
    NormArgs p = whole;
    p.m = whole.m - t < kRows ? whole.m - t : kRows;
    const int64_t off = t * p.n, in = off * (bf16 ? 2 : 4);
    p.X = static_cast<const char*>(p.X) + in;
    if (p.R) {
      p.R = static_cast<const char*>(p.R) + in;
      p.h = static_cast<char*>(p.h) + in;
    }
    p.codes += fmt == kMxFp8 ? off : off / 2;
    p.scales = static_cast<char*>(p.scales) + off / G * (fmt == kInt4Bf16 ? 2 : 1);
    hipError_t e;
    switch (fmt) {
      case kInt4Bf16: e = norm_group<kInt4Bf16>(G, bf16, p, s); break;
      case kMxInt4: e = norm_group<kMxInt4>(G, bf16, p, s); break;
      case kMxFp4: e = norm_group<kMxFp4>(G, bf16, p, s); break;
      case kNvFp4: e = norm_group<kNvFp4>(G, bf16, p, s); break;
      default: e = norm_group<kMxFp8>(G, bf16, p, s); break;
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// whether [p, p + bytes) and [q, q + bytes) overlap without being the same array
static bool clash(const void* p, const void* q, size_t bytes) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return a != b && a < b + bytes && b < a + bytes;
}

// The host-side checks of both forms, and the kernel's arguments but for the status word.
static dq_status norm_args(const void* X, dq_dtype xt, const void* residual, void* residual_out,
                           int64_t tokens, int64_t cols, const void* weight, dq_dtype wt,
                           double eps, const float* b, dq_format fmt, int group, float g,
                           uint8_t* codes, void* inner_scales, NormArgs* p) {
  if ((int)fmt < 0 || (int)fmt > kMxFp8 || (xt != DQ_F32 && xt != DQ_BF16)) return DQ_ERR_UNSUPPORTED;
  if (weight && wt != DQ_F32 && wt != DQ_BF16) return DQ_ERR_UNSUPPORTED;
  if (!X || !codes || !inner_scales) return DQ_ERR_ARG;
  if ((residual == nullptr) != (residual_out == nullptr)) return DQ_ERR_ARG;
  if (tokens < 1 || cols < 1 || (group != 16 && group != 32 && group != 64) || cols % group != 0)
    return DQ_ERR_ARG;
  if (tokens > INT32_MAX || cols > ((int64_t)1 << 40) / tokens) return DQ_ERR_ARG;
  if (!(eps > 0.0) || eps > DBL_MAX) return DQ_ERR_ARG;
  if (fmt == DQ_FMT_NVFP4 && (!(g > 0.0f) || g > FLT_MAX)) return DQ_ERR_ARG;
  if (((uintptr_t)X | (uintptr_t)residual | (uintptr_t)residual_out | (uintptr_t)weight |
       (uintptr_t)b) & 15u)
    return DQ_ERR_ARG;
  if ((uintptr_t)codes & (fmt == DQ_FMT_MXFP8 ? 15u : 7u)) return DQ_ERR_ARG;
  if (fmt == DQ_FMT_INT4_BF16 && ((uintptr_t)inner_scales & 1u)) return DQ_ERR_ARG;
  const size_t bytes = (size_t)tokens * (size_t)cols * (xt == DQ_BF16 ? 2 : 4);
  if (residual && (clash(residual_out, residual, bytes) || clash(residual_out, X, bytes)))
    return DQ_ERR_ARG;
  p->X = X;
  p->R = residual;
  p->h = residual_out;
  p->w = weight;
  p->b = b;
  p->m = tokens;
  p->n = cols;
  p->eps = eps;
  p->g = fmt == DQ_FMT_NVFP4 ? g : 1.0f;
  p->codes = codes;
  p->scales = inner_scales;
  p->wbf = wt == DQ_BF16;
  return DQ_OK;
}

}  // namespace dq

extern "C" {

dq_status dq_norm_quantize_act_async(const void* X, dq_dtype xt, const void* residual,
                                     void* residual_out, int64_t tokens, int64_t cols,
                                     const void* weight, dq_dtype wt, double eps, const float* b,
                                     dq_format fmt, int group, float g, uint8_t* codes,
                                     void* inner_scales, int* status, hipStream_t stream) {
  using namespace dq;
  NormArgs p{};
  const dq_status st = norm_args(X, xt, residual, residual_out, tokens, cols, weight, wt, eps, b,
                                 fmt, group, g, codes, inner_scales, &p);
  if (st != DQ_OK) return st;
  if (!status || ((uintptr_t)status & 3u)) return DQ_ERR_ARG;
  p.status = status;
  return launch_norm(fmt, group, xt == DQ_BF16, p, stream) == hipSuccess ? DQ_OK : DQ_ERR_HIP;
}

dq_status dq_norm_quantize_act(const void* X, dq_dtype xt, const void* residual,
                               void* residual_out, int64_t tokens, int64_t cols,
                               const void* weight, dq_dtype wt, double eps, const float* b,
                               dq_format fmt, int group, float g, uint8_t* codes,
                               void* inner_scales, void* workspace, size_t workspace_bytes,
                               hipStream_t stream) {
  using namespace dq;
  NormArgs p{};
  dq_status st = norm_args(X, xt, residual, residual_out, tokens, cols, weight, wt, eps, b, fmt,
                           group, g, codes, inner_scales, &p);
  if (st != DQ_OK) return st;
  if (workspace && workspace_bytes < DQ_NORM_WORKSPACE_BYTES) return DQ_ERR_WORKSPACE;
  if ((uintptr_t)workspace & 255u) return DQ_ERR_ARG;
  void* ws = workspace;
  if (!ws && hipMallocAsync(&ws, DQ_NORM_WORKSPACE_BYTES, stream) != hipSuccess) return DQ_ERR_HIP;
  p.status = static_cast<int*>(ws);
  int host = 0;
  if (launch_clear(p.status, 1, stream) != hipSuccess ||
      launch_norm(fmt, group, xt == DQ_BF16, p, stream) != hipSuccess ||
      hipMemcpyAsync(&host, p.status, sizeof host, hipMemcpyDeviceToHost, stream) != hipSuccess ||
      hipStreamSynchronize(stream) != hipSuccess)
    st = DQ_ERR_HIP;
  if (!workspace) (void)hipFreeAsync(ws, stream);
  if (st != DQ_OK) return st;
  if (host & kStNonFinite) return DQ_ERR_NONFINITE;
  return (host & kStRange) ? DQ_ERR_RANGE : DQ_OK;
}

}  // extern "C"
