// dq_mlp.hip -- the entry points of the MLP's products (include/dq_mlp.h); their kernels are in
// dq_mlp_kernels.h.
#include "dq_mlp_kernels.h"

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
  const hipError_t e = yt == DQ_BF16 ? launch_o<false, kOutBf16>(p, Plain{}, act8, stream)
                                     : launch_o<false, kOutF32>(p, Plain{}, false, stream);
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
  const hipError_t e = yt == DQ_BF16 ? launch_o<true, kOutBf16>(p, Plain{}, act8, stream)
                                     : launch_o<true, kOutF32>(p, Plain{}, false, stream);
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
  const hipError_t e = fmt == DQ_FMT_MXFP8 ? launch_o<true, kOutFp8>(p, Plain{}, act8, stream)
                                           : launch_o<true, kOutFp4>(p, Plain{}, act8, stream);
  return e == hipSuccess ? DQ_OK : DQ_ERR_HIP;
}

}  // extern "C"
