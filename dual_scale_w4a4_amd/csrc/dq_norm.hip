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
// k_norm: a workgroup has a thread per 16 channels (up to 16384) and takes row after row, w and b
// staying in registers; the next row's loads are in flight while a row is summed (one barrier)
// and quantized, so each array is read and written once. Bound by memory: 8192 x 4096 bf16 with
// residual to MXFP8 takes 44.7 us for 236 MB, 5.3 TB/s (a copy of 1 GiB runs at 5.1; two sweeps a
// row without the pipeline took 58 us); one row 3.0 us. k_norm_wide, for wider rows, sweeps the row
// twice (h is read back).
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

// 16 values of a bf16 or fp32 array as loaded, and unpacked to fp32
template <bool BF>
struct Raw16 {
  u32x4 v[BF ? 2 : 4];
  __device__ __forceinline__ void load(const void* p, int64_t off) {
    const u32x4* s = reinterpret_cast<const u32x4*>(static_cast<const char*>(p) + off * (BF ? 2 : 4));
#pragma unroll
    for (int k = 0; k < (BF ? 2 : 4); k++) v[k] = s[k];
  }
  __device__ __forceinline__ void unpack(float (&x)[kNormEpl]) const {
#pragma unroll
    for (int k = 0; k < (BF ? 2 : 4); k++)
#pragma unroll
      for (int e = 0; e < 4; e++) {
        if (BF) {
          x[8 * k + 2 * e] = u2f(v[k][e] << 16);
          x[8 * k + 2 * e + 1] = u2f(v[k][e] & 0xFFFF0000u);
        } else {
          x[4 * k + e] = u2f(v[k][e]);
        }
      }
  }
};

template <bool BF>
__device__ __forceinline__ void load16(const void* p, int64_t off, float (&v)[kNormEpl]) {
  Raw16<BF> r;
  r.load(p, off);
  r.unpack(v);
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

// The constants of a call's quantizer (NVFP4)
struct QuantConst {
  float g, sixg;
  double r6;
};

__device__ __forceinline__ QuantConst quant_const(float g) {
  const float sixg = 6.0f * g;
  return QuantConst{g, sixg, 1.0 / (double)sixg};
}

// Codes and scale of one lane's 16 values (the group of G values lies in G / 16 neighbouring
// lanes) at element offset off of the outputs. `act`: whether the lane's channels exist (the
// group's lanes agree; all lanes of the wave take part in the maxima). Returns whether a group
// that exists holds a NaN or an infinity; it is then written as a group of zeros.
template <int FMT, int G>
__device__ __forceinline__ bool quantize16(float (&x)[kNormEpl], bool act, const NormArgs& p,
                                           int64_t off, const QuantConst& q) {
  constexpr int LPG = G / kNormEpl;
  uint32_t gmb = 0u;  // the largest |x| as bits, above every finite value's for a NaN
#pragma unroll
  for (int k = 0; k < kNormEpl; k++) gmb = max(gmb, f2u(x[k]) & 0x7FFFFFFFu);
  if (LPG > 1) gmb = group_max_bits<LPG>(gmb);
  const bool bad = gmb >= 0x7F800000u;
  if (bad) {
    gmb = 0u;
#pragma unroll
    for (int k = 0; k < kNormEpl; k++) x[k] = 0.0f;
  }
  uint32_t scode;
  if (FMT == kMxFp8) {
    scode = mx_scale_code<8>(gmb);
    const float rd = u2f((254u - scode) << 23);
    const u32x4 c = {fp8_pack4(x, rd), fp8_pack4(x + 4, rd), fp8_pack4(x + 8, rd),
                     fp8_pack4(x + 12, rd)};
    if (act) __builtin_nontemporal_store(c, reinterpret_cast<u32x4*>(p.codes + off));
  } else {
    u32x2 c;
    if (FMT == kMxFp4) {
      scode = mx_scale_code<2>(gmb);
      const GroupQ gq = mx_group(scode);
      c = u32x2{fp4_pack<8>(x, gq), fp4_pack<8>(x + 8, gq)};
    } else {
      // the exact rules of dq_device.h: the power-of-two quotient for MXINT4, fp32 codes for
      // NVFP4 where every divisor of the wave allows them, else the snapped double quotient
      constexpr int F = FMT == kMxFp8 ? kMxInt4 : FMT;
      const GroupQ gq = F == kNvFp4 ? nv_group_scale(u2f(gmb), q.g, q.r6)
                                    : group_scale<F>(u2f(gmb), q.g, q.sixg);
      scode = gq.scode;
      if (F == kNvFp4 && __all(gq.d >= 0x1p-100f && gq.d <= 0x1p100f)) {
        c = u32x2{nv_pack8_fast<true>(x, gq.d, gq.rd), nv_pack8_fast<true>(x + 8, gq.d, gq.rd)};
      } else {
        const double r = F == kMxInt4 ? 0.0 : recip64(gq.d);
#pragma unroll
        for (int k = 0; k < 2; k++) {
          uint32_t pk = 0u;
#pragma unroll
          for (int e = 0; e < 8; e++) {
            double v = code64<F>(x[8 * k + e], r, gq);
            if (F == kInt4Bf16) v = int4_clamp(v);
            pk |= nibble_of<F>((float)v) << (4 * e);
          }
          c[k] = pk;
        }
      }
    }
    if (act) __builtin_nontemporal_store(c, reinterpret_cast<u32x2*>(p.codes + (off >> 1)));
  }
  if (act && (LPG == 1 || (threadIdx.x % LPG) == 0)) {
    const int64_t si = off / G;  // rows hold whole groups
    if (FMT == kInt4Bf16)
      static_cast<uint16_t*>(p.scales)[si] = (uint16_t)scode;
    else
      static_cast<uint8_t*>(p.scales)[si] = (uint8_t)scode;
  }
  return bad && act;
}

// h = X + R of 16 channels, rounded to the stream's type
template <bool BF>
__device__ __forceinline__ void add_residual(float (&h)[kNormEpl], const float (&r)[kNormEpl]) {
#pragma unroll
  for (int k = 0; k < kNormEpl; k++) {
    h[k] += r[k];
    if (BF) h[k] = to_bf16(h[k]);
  }
}

// this lane's sum of squares: not finite exactly where an h is not (finite squares fit fp64)
__device__ __forceinline__ double sum_squares(const float (&h)[kNormEpl]) {
  double sum = 0.0;
#pragma unroll
  for (int k = 0; k < kNormEpl; k++) sum = fma((double)h[k], (double)h[k], sum);
  return sum;
}

__device__ __forceinline__ bool any_nonfinite(const float (&v)[kNormEpl]) {
  bool bad = false;
#pragma unroll
  for (int k = 0; k < kNormEpl; k++) bad |= !(fabsf(v[k]) <= FLT_MAX);
  return bad;
}

// w and b of 16 channels (ones where there is none: a product with 1 is exact)
__device__ __forceinline__ void load_factors(const NormArgs& p, int64_t c, float (&w)[kNormEpl],
                                             float (&b)[kNormEpl]) {
#pragma unroll
  for (int k = 0; k < kNormEpl; k++) w[k] = b[k] = 1.0f;
  if (p.w) {
    if (p.wbf) load16<true>(p.w, c, w);
    else load16<false>(p.w, c, w);
  }
  if (p.b) load16<false>(p.b, c, b);
}

// sum of v over the workgroup's waves, in wave order, in every thread; red: a double per wave,
// not written again before the next barrier
__device__ __forceinline__ double block_sum(double v, double* red, int waves) {
  v = sum16_dpp(v);
  const double w = ((__shfl(v, 0, kWave) + __shfl(v, 16, kWave)) + __shfl(v, 32, kWave)) +
                   __shfl(v, 48, kWave);
  if (waves == 1) return w;
  if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x / kWave] = w;
  __syncthreads();
  double sum = red[0];
  for (int k = 1; k < waves; k++) sum += red[k];
  return sum;
}

constexpr int kNormThreads = 1024;  // k_norm: rows of up to kNormThreads * kNormEpl channels

template <int FMT, int G, bool BF>
__global__ __launch_bounds__(kNormThreads) void k_norm(NormArgs p) {
  __shared__ double red[2][kNormThreads / kWave];
  // Lanes past the row's end hold zeros: they load nothing, since where h replaces X or R another
  // wave may have stored already what they would read, and they store and report nothing.
  const int64_t c = threadIdx.x * kNormEpl;
  const bool act = c < p.n;
  const int waves = blockDim.x / kWave;
  const QuantConst q = quant_const(p.g);
  float w[kNormEpl], b[kNormEpl];
  Raw16<BF> xr = {}, rr = {};
  int64_t row = blockIdx.x;
  if (act) {
    xr.load(p.X, row * p.n + c);
    if (p.R) rr.load(p.R, row * p.n + c);
  }
  load_factors(p, act ? c : 0, w, b);
  int flags = 0;
  for (int par = 0; row < p.m; row += gridDim.x, par ^= 1) {
    const int64_t off = row * p.n + c;
    float h[kNormEpl];
    xr.unpack(h);
    if (p.R) {
      float r[kNormEpl];
      rr.unpack(r);
      add_residual<BF>(h, r);
      if (act) store16<BF>(p.h, off, h);
    }
    double sum = sum_squares(h);
    if (!(sum <= DBL_MAX)) {  // rare
      float v[kNormEpl];
      xr.unpack(v);
      bool in = any_nonfinite(v);
      if (p.R) {
        rr.unpack(v);
        in |= any_nonfinite(v);
      }
      flags |= in ? kStNonFinite : kStRange;
    }
    const int64_t next = row + gridDim.x;
    if (act && next < p.m) {
      xr.load(p.X, next * p.n + c);
      if (p.R) rr.load(p.R, next * p.n + c);
    }
    sum = block_sum(sum, red[par], waves);
    const float rstd = (float)(1.0 / sqrt(sum / (double)p.n + p.eps));
#pragma unroll
    for (int k = 0; k < kNormEpl; k++) h[k] = h[k] * rstd * w[k] * b[k];
    // an overflow of x, unless the row's h already was not finite (reported above)
    if (quantize16<FMT, G>(h, act, p, off, q) && sum <= DBL_MAX) flags |= kStRange;
  }
  if (flags) atomicOr(p.status, flags);
}

template <int FMT, int G, bool BF>
__global__ __launch_bounds__(kBlock) void k_norm_wide(NormArgs p) {
  __shared__ double red[kWaves];
  const int64_t row = (int64_t)blockIdx.x * p.n;
  int flags = 0;
  double sum = 0.0;
  for (int64_t c = threadIdx.x * kNormEpl; c < p.n; c += kBlock * kNormEpl) {
    float h[kNormEpl], r[kNormEpl];
    load16<BF>(p.X, row + c, h);
    bool in = any_nonfinite(h);
    if (p.R) {
      load16<BF>(p.R, row + c, r);
      in |= any_nonfinite(r);
      add_residual<BF>(h, r);
      store16<BF>(p.h, row + c, h);
    }
    const double s = sum_squares(h);
    if (!(s <= DBL_MAX)) flags |= in ? kStNonFinite : kStRange;
    sum += s;
  }
  sum = block_sum(sum, red, kWaves);
  const float rstd = (float)(1.0 / sqrt(sum / (double)p.n + p.eps));
  const QuantConst q = quant_const(p.g);
  const void* src = p.R ? p.h : p.X;
  // every lane of a wave runs the same trips (the group maxima exchange lanes); lanes past the
  // row's end read its start and store nothing
  for (int64_t c0 = 0; c0 < p.n; c0 += kBlock * kNormEpl) {
    const int64_t c = c0 + threadIdx.x * kNormEpl;
    const bool act = c < p.n;
    const int64_t lc = act ? c : 0;
    float x[kNormEpl], w[kNormEpl], b[kNormEpl];
    load16<BF>(src, row + lc, x);
    load_factors(p, lc, w, b);
#pragma unroll
    for (int k = 0; k < kNormEpl; k++) x[k] = x[k] * rstd * w[k] * b[k];
    if (quantize16<FMT, G>(x, act, p, row + lc, q) && sum <= DBL_MAX) flags |= kStRange;
  }
  if (flags) atomicOr(p.status, flags);
}

template <int FMT, int G>
static hipError_t norm_launch(bool bf16, const NormArgs& p, hipStream_t s) {
  if (p.n > kNormThreads * kNormEpl) {
    const dim3 grid((unsigned)p.m);
    if (bf16)
      hipLaunchKernelGGL((k_norm_wide<FMT, G, true>), grid, dim3(kBlock), 0, s, p);
    else
      hipLaunchKernelGGL((k_norm_wide<FMT, G, false>), grid, dim3(kBlock), 0, s, p);
    return hipGetLastError();
  }
  const int waves = (int)((p.n + kWave * kNormEpl - 1) / (kWave * kNormEpl));
  const int64_t most = 256 * (16 / waves);  // sixteen waves per CU
  const dim3 grid((unsigned)(p.m < most ? p.m : most));
  if (bf16)
    hipLaunchKernelGGL((k_norm<FMT, G, true>), grid, dim3(waves * kWave), 0, s, p);
  else
    hipLaunchKernelGGL((k_norm<FMT, G, false>), grid, dim3(waves * kWave), 0, s, p);
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

// The host-side checks of both forms, and the kernel's arguments. `word`: the status word, or the
// workspace that holds it (null: neither is the caller's); it is an output like the others.
static dq_status norm_args(const void* X, dq_dtype xt, const void* residual, void* residual_out,
                           int64_t tokens, int64_t cols, const void* weight, dq_dtype wt,
                           double eps, const float* b, dq_format fmt, int group, float g,
                           uint8_t* codes, void* inner_scales, const Span& word, NormArgs* p) {
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
  const size_t n = (size_t)tokens * (size_t)cols, vb = (size_t)cols * 4;
  if (any_overlap({{codes, fmt == DQ_FMT_MXFP8 ? n : n / 2},
                   {inner_scales, n / (size_t)group * (fmt == DQ_FMT_INT4_BF16 ? 2 : 1)},
                   {residual_out, bytes},
                   word},
                  {{X == residual_out ? nullptr : X, bytes},
                   {residual == residual_out ? nullptr : residual, bytes},
                   {weight, wt == DQ_BF16 ? vb / 2 : vb},
                   {b, vb}}))
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
  p->status = static_cast<int*>(const_cast<void*>(word.p));
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
                                 fmt, group, g, codes, inner_scales, {status, sizeof *status}, &p);
  if (st != DQ_OK) return st;
  if (!status || ((uintptr_t)status & 3u)) return DQ_ERR_ARG;
  return launch_norm(fmt, group, xt == DQ_BF16, p, stream) == hipSuccess ? DQ_OK : DQ_ERR_HIP;
}

dq_status dq_norm_quantize_act(const void* X, dq_dtype xt, const void* residual,
                               void* residual_out, int64_t tokens, int64_t cols,
                               const void* weight, dq_dtype wt, double eps, const float* b,
                               dq_format fmt, int group, float g, uint8_t* codes,
                               void* inner_scales, void* workspace, size_t workspace_bytes,
                               hipStream_t stream) {
  using namespace dq;
  if (workspace && workspace_bytes < DQ_NORM_WORKSPACE_BYTES) return DQ_ERR_WORKSPACE;
  NormArgs p{};
  dq_status st = norm_args(X, xt, residual, residual_out, tokens, cols, weight, wt, eps, b, fmt,
                           group, g, codes, inner_scales, {workspace, DQ_NORM_WORKSPACE_BYTES},
                           &p);
  if (st != DQ_OK) return st;
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
