// dq_outq.h -- quantized outputs of the MLP operators: the group quantizer's codes for values in
// registers, for the formats of dq_device.h and for MXFP8 (E4M3 elements, E8M0 scale).
#pragma once

#include "dq_device.h"

namespace dq {

// An array of a call, for the host's checks of what may overlap
struct Span {
  const void* p;  // null: not given
  size_t bytes;
};

inline bool overlap(const Span& s, const Span& t) {
  const uintptr_t a = (uintptr_t)s.p, b = (uintptr_t)t.p;
  return s.p && t.p && a < b + t.bytes && b < a + s.bytes;
}

// whether an output overlaps an input or another output
template <size_t O, size_t I>
bool any_overlap(const Span (&out)[O], const Span (&in)[I]) {
  for (size_t o = 0; o < O; o++) {
    for (size_t i = 0; i < I; i++)
      if (overlap(out[o], in[i])) return true;
    for (size_t k = 0; k < o; k++)
      if (overlap(out[o], out[k])) return true;
  }
  return false;
}

constexpr int kMxFp8 = 4;  // DQ_FMT_MXFP8

// The E8M0 divisor of an MXFP4 (EMAX 2) or MXFP8 (EMAX 8) group from the bits of its largest
// |x| (finite): biased exponent e + 127 of 2^e, e = clamp(floor(log2 max) - EMAX, -126, 126); a
// group of zeros takes 2^0. A subnormal maximum has exponent field 0 and clamps.
template <int EMAX>
DQ_HD uint32_t mx_scale_code(uint32_t max_bits) {
  const int e = (int)(max_bits >> 23) - EMAX;
  return max_bits == 0u ? 127u : (uint32_t)(e < 1 ? 1 : e);
}

// 4 E4M3 codes (one per byte) of x / d, rd = 1 / d a power of two (so x rd is exact wherever
// the code is not zero): clamped to the largest code first, since the conversion turns
// larger values into NaN; a zero is stored as 0x00 whatever its sign.
__device__ __forceinline__ uint32_t fp8_pack4(const float* x, float rd) {
  float v[4];
#pragma unroll
  for (int k = 0; k < 4; k++) v[k] = __builtin_amdgcn_fmed3f(x[k] * rd, -448.0f, 448.0f);
  int pk = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  pk = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], pk, true);
  const uint32_t u = (uint32_t)pk, mag = u & 0x7F7F7F7Fu;
  return mag | (u & (mag + 0x7F7F7F7Fu) & 0x80808080u);
}

// N (4 or 8) E2M1 codes of x / d as nibbles, first value lowest, d = 2^e. The hardware
// conversion divides by d and rounds to nearest even, saturating; it is used where it was
// checked on every input, d in [2^-100, 2^20], and the exact fp32 path elsewhere.
template <int N>
__device__ __forceinline__ uint32_t fp4_pack(const float* x, const GroupQ& gq) {
  uint32_t pk = 0u;
  if (gq.d >= 0x1p-100f && gq.d <= 0x1p20f) {
    pk = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, x[0], x[1], gq.d, 0);
    pk = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(pk, x[2], x[3], gq.d, 1);
    if (N == 8) {
      pk = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(pk, x[4 % N], x[5 % N], gq.d, 2);
      pk = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(pk, x[6 % N], x[7 % N], gq.d, 3);
    }
    const uint32_t mag = pk & 0x77777777u;  // keep the sign only where the magnitude is
    return mag | (pk & (mag + 0x77777777u) & 0x88888888u);  // nonzero (no -0 code)
  }
#pragma unroll
  for (int k = 0; k < N; k++) pk |= nibble_of<kMxFp4>(code_of<kMxFp4>(x[k], gq)) << (4 * k);
  return pk;
}

// The divisor of an MX group from its scale code, as the pack functions take it.
__device__ __forceinline__ GroupQ mx_group(uint32_t scode) {
  GroupQ r;
  r.scode = scode;
  r.d = u2f(scode << 23);
  r.rd = u2f((254u - scode) << 23);
  r.sc = 1.0f;
  r.ds = r.d;
  r.hds = 0.5f * r.d;
  return r;
}

}  // namespace dq
