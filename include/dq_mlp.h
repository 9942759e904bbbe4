/*
 * dq_mlp.h -- C ABI of libdq.so's MLP operators: what lies between and around the W4A4 products
 * of dq.h in a decoder layer, as fused kernels on the same operands.
 *
 *   dq_norm_quantize_act      residual addition, root-mean-square norm, column scales, quantizer
 *   dq_gemm_mx_epilogue       the packed product with bias, activation and residual
 *   dq_gated_mx               both products of a gated MLP, the activation and their product
 *   dq_gated_mx_quantized     the same, quantized for the next product
 *
 * The MLP of a decoder layer is three launches: norm_quantize_act, gated_mx_quantized,
 * gemm_mx_epilogue with the residual.
 *
 * The conventions are dq.h's: dense row-major device arrays owned by the caller, host-side
 * argument checks before anything is enqueued, no state between calls, deterministic results
 * (no floating-point atomics; the order of every sum depends on the shape alone). An output
 * (a status word or a workspace too) overlaps neither an input nor another output (DQ_ERR_ARG)
 * but where a call says so. The calls allocate nothing and use no workspace unless they say so,
 * so they can be captured into a graph. `stream` belongs to the current device, where the arrays
 * are.
 */
#ifndef DQ_MLP_H
#define DQ_MLP_H

#include "dq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* MXFP8 activations, a format of these operators only: E4M3 elements (one byte each, zero
 * always 0x00) and one E8M0 scale per group, 2^clamp(floor(log2 max) - 8, -126, 126) (the
 * element format's largest exponent is 8), elements rounded to nearest, ties to even, and
 * saturated at 448. Codes: tokens x K bytes. */
#define DQ_FMT_MXFP8 ((dq_format)4)

/* Activations of the epilogues, computed in fp32 with the matrix results: none, max(z, 0),
 * z / (1 + exp(-z)), z (1 + erf(z / sqrt 2)) / 2, and the tanh form of the last. */
typedef enum {
  DQ_ACTIVATION_NONE = 0,
  DQ_ACTIVATION_RELU = 1,
  DQ_ACTIVATION_SILU = 2,
  DQ_ACTIVATION_GELU = 3,
  DQ_ACTIVATION_GELU_TANH = 4
} dq_activation;

/* The norm in front of a quantized product, with the addition of the residual stream:
 *     h  = X + residual, rounded to X's type and stored (what the stream holds is what is
 *          normalized, so the result is that of a separate addition); h = X without residual
 *     r  = fl32(1 / sqrt(mean_j h_tj^2 + eps)), the sum of squares and the root in fp64
 *     x  = fl32(fl32(fl32(h r) weight_j) b_j)
 * and then the group quantizer of dq_quantize_act on x, bit for bit.
 *  X:            tokens x cols, fp32 or bf16 (xt), 16-byte aligned.
 *  residual:     as X, or NULL.  residual_out: out, h, as X; both are given or neither is.
 *                residual_out may equal residual or X (updated in place).
 *  weight:       cols values of type wt (fp32 or bf16), 16-byte aligned, or NULL for ones.
 *  eps:          > 0, finite.
 *  b:            cols floats > 0, 16-byte aligned, or NULL for ones.
 *  fmt, group:   any format of dq.h or DQ_FMT_MXFP8; group 16, 32 or 64, cols % group == 0.
 *  g:            NVFP4's tensor scale, > 0 (a scale computed from the output would need the
 *                whole output first); ignored otherwise.
 *  codes:        out, packed as for dq_quantize_act (8-byte aligned), or for MXFP8 tokens x
 *                cols bytes (16-byte aligned).
 *  inner_scales: out, tokens x (cols / group) entries, as for dq_quantize_act.
 * The asynchronous form only enqueues; errors found on the device are OR-ed into *status
 * (device, caller-owned, 4-byte aligned): bit 1 a NaN / Inf in X or residual, bit 2 an overflow
 * of their sum or of x. A row with an error has unspecified codes and scales; other rows are
 * not affected. The blocking form returns them as DQ_ERR_NONFINITE / DQ_ERR_RANGE after
 * synchronizing `stream`; its workspace holds the status word: DQ_NORM_WORKSPACE_BYTES, 256-byte
 * aligned, or NULL to allocate it stream-ordered. */
#define DQ_NORM_WORKSPACE_BYTES 256u
dq_status dq_norm_quantize_act_async(const void* X, dq_dtype xt, const void* residual,
                                     void* residual_out, int64_t tokens, int64_t cols,
                                     const void* weight, dq_dtype wt, double eps, const float* b,
                                     dq_format fmt, int group, float g, uint8_t* codes,
                                     void* inner_scales, int* status, hipStream_t stream);
dq_status dq_norm_quantize_act(const void* X, dq_dtype xt, const void* residual,
                               void* residual_out, int64_t tokens, int64_t cols,
                               const void* weight, dq_dtype wt, double eps, const float* b,
                               dq_format fmt, int group, float g, uint8_t* codes,
                               void* inner_scales, void* workspace, size_t workspace_bytes,
                               hipStream_t stream);

/* The product with packed weights (dq_gemm_pack_weights), with its epilogue:
 *     Y[t][i] = residual[t][i] + act(a_i * sum_k x^[t][k] Qhat[i][k] + bias_i)
 * the sum in fp32 on the matrix cores, everything after it in fp32, one rounding to Y's type.
 *  act_codes, act_scales: the activations in act_fmt, MXFP4 (tokens x K/2 bytes) or MXFP8
 *                (tokens x K bytes), group 32, both 16-byte aligned; scales tokens x K/32.
 *  packed_codes, packed_scales: as for dq_gemm_mx_packed (out x K, K % 512 == 0, K <= 2^22).
 *  a, bias:      out floats, 16-byte aligned, or NULL (ones / zeros).
 *  residual:     tokens x out of Y's type, or NULL; may equal Y.
 *  Y:            out, tokens x out, fp32 or bf16 (yt), aligned to its element; likewise residual.
 * MXFP8 activations give bf16 only: in its 8-bit mode the matrix instruction truncates the
 * products of 8 neighbouring k at 2^-13 of the power of two of the largest, about 2^-15 of a long
 * sum, which changes the last bit of 1 or 2 bf16 results in a hundred and would show in fp32. An
 * E8M0 byte 0xFF makes the outputs it reaches NaN. tokens < 2^31 - 256, out <= 2^22.
 * Only enqueues. */
dq_status dq_gemm_mx_epilogue(const uint8_t* act_codes, const uint8_t* act_scales,
                              dq_format act_fmt, int64_t tokens, int64_t K,
                              const uint8_t* packed_codes, const uint8_t* packed_scales,
                              const float* a, const float* bias, dq_activation activation,
                              const void* residual, int64_t out, dq_dtype yt, void* Y,
                              hipStream_t stream);

/* The gated half of an MLP: both projections of the same activations, the activation function
 * and the product, in one kernel:
 *     H[t][i] = act(a_gate_i * sum_k x^[t][k] Qgate[i][k]) * (a_up_i * sum_k x^[t][k] Qup[i][k])
 * with gate and up weights inner x K, each packed by itself. Arguments as for
 * dq_gemm_mx_epilogue. */
dq_status dq_gated_mx(const uint8_t* act_codes, const uint8_t* act_scales, dq_format act_fmt,
                      int64_t tokens, int64_t K, const uint8_t* gate_codes,
                      const uint8_t* gate_scales, const float* a_gate, const uint8_t* up_codes,
                      const uint8_t* up_scales, const float* a_up, dq_activation activation,
                      int64_t inner, dq_dtype yt, void* H, hipStream_t stream);

/* The same, handed to the next product: x = fl32(H * b) (H in fp32, not rounded to bf16 first),
 * quantized in groups of 32 channels by the rule of dq_quantize_act (MXFP4) or of DQ_FMT_MXFP8.
 *  b:      inner floats > 0 (the next weights' column inverse scales), 16-byte aligned, or NULL.
 *  codes:  out, tokens x inner/2 (MXFP4) or tokens x inner (MXFP8) bytes, 16-byte aligned.
 *  scales: out, tokens x inner/32 E8M0 bytes.  inner % 32 == 0.
 * With MXFP8 activations the sums carry the truncation described above, so that a value next to
 * the border between two codes (or a group's largest next to a power of two) may fall on either
 * side; every code is the quantizer's of a sum within that error.
 * A group that holds a NaN or an infinity gets the scale 0xFF (E8M0's NaN) and zero codes, so
 * that the next product's outputs are NaN there; there is no device-side error to report. */
dq_status dq_gated_mx_quantized(const uint8_t* act_codes, const uint8_t* act_scales,
                                dq_format act_fmt, int64_t tokens, int64_t K,
                                const uint8_t* gate_codes, const uint8_t* gate_scales,
                                const float* a_gate, const uint8_t* up_codes,
                                const uint8_t* up_scales, const float* a_up,
                                dq_activation activation, int64_t inner, const float* b,
                                dq_format fmt, uint8_t* codes, uint8_t* scales,
                                hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* DQ_MLP_H */
