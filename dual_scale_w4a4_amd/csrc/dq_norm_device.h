// dq_norm_device.h -- what the norm kernels share: rows of 16 channels per lane, their loads and
// stores, sums of squares over a workgroup, and the group quantizer on 16 values in registers.
#pragma once

#include <float.h>
#include <math.h>

#include "dq_outq.h"

namespace dq {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kNormEpl = 16;  // consecutive channels per lane

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
// lanes) at element offset off of the outputs p.codes and p.scales. `act`: whether the lane's channels exist (the
// group's lanes agree; all lanes of the wave take part in the maxima). Returns whether a group
// that exists holds a NaN or an infinity; it is then written as a group of zeros.
template <int FMT, int G, class P>
__device__ __forceinline__ bool quantize16(float (&x)[kNormEpl], bool act, const P& p,
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

}  // namespace dq
