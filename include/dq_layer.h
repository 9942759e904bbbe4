/*
 * dq_layer.h -- C ABI of libdq.so's operators for decoder layers beyond the dense MLP of
 * dq_mlp.h: norms on both sides of a block, a projection that many requests share with a low-rank
 * adapter of each request beside it, and a layer of experts with its router.
 *
 *   dq_block_norm_quantize_act  norm after a block, its gate, the scaled residual, norm before the
 *                               next block, column scales, quantizer
 *   dq_gemm_mx_adapters         dq_gemm_mx_epilogue with each token's own low-rank adapter
 *   dq_moe_route                scores of the experts, the top k of them and their weights
 *   dq_moe_mx                   gated products, quantizer, down products and weighted sum of every
 *                               token's experts
 *
 * The conventions are dq_mlp.h's: dense row-major device arrays owned by the caller, host-side
 * argument checks before anything is enqueued, no state between calls, deterministic results (no
 * floating-point atomics), outputs that overlap nothing but where a call says so (DQ_ERR_ARG), no
 * allocation. The calls only enqueue (except dq_block_norm_quantize_act) and can be captured into
 * a graph. A workspace is scratch memory of one call at a time: calls (and replays of graphs) that
 * share one have to follow each other on the device. `stream` belongs to the current device, where
 * the arrays are.
 */
#ifndef DQ_LAYER_H
#define DQ_LAYER_H

#include "dq_mlp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What lies between a block (attention, MLP, experts) and the next one's quantized product:
 *     m  = X, or with post_norm fl32(fl32(X r1) post_weight_j), r1 = fl32(1 / sqrt(mean_j X_tj^2
 *          + post_eps))
 *     m  = fl32(fl32(m gate_j) token_gate_t)
 *     h  = fl32(fl32(residual_scale residual) + m), rounded to X's type and stored
 *     n  = fl32(fl32(h r2) weight_j),  r2 = fl32(1 / sqrt(mean_j h_tj^2 + eps))
 *     x  = fl32(n b_j)
 * (sums of squares and roots in fp64) and then the group quantizer of dq_quantize_act on x, bit
 * for bit.
 *  X:            the block's output, tokens x cols, fp32 or bf16 (xt), 16-byte aligned.
 *  post_norm:    0 or 1.  post_weight: cols values of type wt, or NULL for ones; NULL without
 *                post_norm.  post_eps: > 0, finite (ignored without post_norm).
 *  gate:         cols floats, or NULL for ones.  token_gate: tokens floats (4-byte aligned), or
 *                NULL for ones.
 *  residual:     as X, or NULL for zeros.  residual_scale: finite.
 *  residual_out: out, h, as X; may equal residual or X (updated in place).
 *  weight:       cols values of type wt (fp32 or bf16), or NULL for ones.  eps: > 0, finite.
 *  x_out:        out, n rounded to type xot (fp32 or bf16), tokens x cols, or NULL: what a router
 *                or an adapter reads.
 *  b, fmt, group, g, codes, inner_scales, status, workspace: as for dq_norm_quantize_act.
 * All arrays of cols or tokens x cols values 16-byte aligned. Status bits: 1 a NaN / Inf in X or
 * residual, 2 a value of h, n (as x_out holds it) or x that is not finite in a row whose X and
 * residual are. A row with an error has unspecified outputs; other rows are not affected. */
dq_status dq_block_norm_quantize_act_async(
    const void* X, dq_dtype xt, int post_norm, const void* post_weight, double post_eps,
    const float* gate, const float* token_gate, const void* residual, float residual_scale,
    void* residual_out, int64_t tokens, int64_t cols, const void* weight, dq_dtype wt, double eps,
    void* x_out, dq_dtype xot, const float* b, dq_format fmt, int group, float g, uint8_t* codes,
    void* inner_scales, int* status, hipStream_t stream);
dq_status dq_block_norm_quantize_act(
    const void* X, dq_dtype xt, int post_norm, const void* post_weight, double post_eps,
    const float* gate, const float* token_gate, const void* residual, float residual_scale,
    void* residual_out, int64_t tokens, int64_t cols, const void* weight, dq_dtype wt, double eps,
    void* x_out, dq_dtype xot, const float* b, dq_format fmt, int group, float g, uint8_t* codes,
    void* inner_scales, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* dq_gemm_mx_epilogue with a low-rank adapter of each token beside the shared weights:
 *     Y[t][i] = residual[t][i] + act(a_i * sum_k x^[t][k] Qhat[i][k] + bias_i
 *                                    + scale_r * sum_j u[t][j] B_r[i][j])
 *     u[t][j] = sum_k X[t][k] A_r[j][k],  r = adapter[t]
 * both sums in fp32 on the matrix cores, of exact products of bf16 values in u; for B u is split
 * into bf16 values that hold 16 bits of it, or all 24 where Y is fp32.
 *  X:            the activations before column scales and quantizer, tokens x K, bf16 (A is the
 *                adapter as trained: no column scale is in it).
 *  adapter:      tokens values (4-byte aligned); a token with one outside 0 .. adapters - 1 has no
 *                adapter. Tokens of one adapter need not be neighbours, but blocks of 32 tokens with
 *                few adapters are faster.
 *  A:            adapters x rank x K, bf16.  B: adapters x out x rank, bf16.  X, A, B 16-byte
 *                aligned.  1 <= adapters <= 2^20; rank a multiple of 8, 8 .. 256 (shorter adapters
 *                padded with zeros).
 *  scale:        adapters floats (4-byte aligned), or NULL for ones.
 *  workspace:    dq_adapter_workspace_bytes, 256-byte aligned.
 * A NaN or an infinity in an adapter reaches its own tokens only. The other arguments as for
 * dq_gemm_mx_epilogue. */
dq_status dq_adapter_workspace_bytes(int64_t tokens, int64_t K, int rank, size_t* bytes);
dq_status dq_gemm_mx_adapters(const uint8_t* act_codes, const uint8_t* act_scales, dq_format act_fmt,
                              int64_t tokens, int64_t K, const uint8_t* packed_codes,
                              const uint8_t* packed_scales, const float* a, const float* bias,
                              const void* X, const int32_t* adapter, int64_t adapters, int rank,
                              const void* A, const void* B, const float* scale,
                              dq_activation activation, const void* residual, int64_t out,
                              dq_dtype yt, void* Y, void* workspace, size_t workspace_bytes,
                              hipStream_t stream);

/* How a router turns a logit into a score: the softmax over all experts, or 1 / (1 + exp(-l)). */
typedef enum { DQ_SCORE_SOFTMAX = 0, DQ_SCORE_SIGMOID = 1 } dq_score;

/* The router of a layer of experts:
 *     l_te = fl32(sum_k X_tk W_ek)  (the sum in fp64, so that its order does not matter)
 *     s_te = the score of l_te, in fp64
 *     ids[t] = the top_k experts with the largest s_te + bias_e (fp64), largest first, ties to the
 *              lower index
 *     weights[t] = fl32(scale * s_te) of those, or with renormalize fl32(scale * s_te / their sum)
 *              (zeros where the sum is zero)
 *  X:            tokens x cols, fp32 or bf16 (xt).  W: experts x cols, fp32 or bf16 (wt). Both 16-byte
 *                aligned, cols a multiple of 8, at most 2^22.  1 <= experts <= 1024.
 *  bias:         experts floats (4-byte aligned), or NULL for zeros.
 *  top_k:        1 .. min(32, experts).  renormalize: 0 or 1.  scale: finite.
 *  ids, weights: out, tokens x top_k (4-byte aligned).
 *  workspace:    dq_moe_route_workspace_bytes, 256-byte aligned.
 * A NaN s_te + bias_e ranks as -infinity, so ids are always top_k different experts. */
dq_status dq_moe_route_workspace_bytes(int64_t tokens, int64_t experts, size_t* bytes);
dq_status dq_moe_route(const void* X, dq_dtype xt, int64_t tokens, int64_t cols, const void* W,
                       dq_dtype wt, int64_t experts, const float* bias, dq_score score, int top_k,
                       int renormalize, float scale, int32_t* ids, float* weights, void* workspace,
                       size_t workspace_bytes, hipStream_t stream);

/* A layer of experts: for each token its top_k experts' gated MLPs, summed with the token's weights:
 *     H  = act(a_gate_ei * sum_k x^ Qgate_e) * (a_up_ei * sum_k x^ Qup_e),  e = ids[t][s]
 *     q  = the quantizer's values of fl32(H * b_e) in groups of 32 channels (inner_fmt)
 *     Y[t][i] = residual[t][i] + sum_s weights[t][s] * (a_down_ei * sum_j q_j Qdown_e)
 * products as dq_gated_mx_quantized and dq_gemm_mx_epilogue compute them, except that MXFP8
 * activations are multiplied in two parts (codes of at least 4, and the others), which leaves the
 * gate's and up products whole: truncated sums would change codes near a border (up to 6 10^-3 of Y).
 * The down product of MXFP8 codes q is truncated as dq_gemm_mx_epilogue's (about 5 10^-5 of Y).
 * The sum over s in fp32 in ascending order, residual last, one rounding to Y's type.
 *  act_codes, act_scales, act_fmt, K: the activations, as for dq_gated_mx. Gate's, up and all experts'
 *                weights multiply the same x^, so they share one set of column scales b; only the
 *                down products' are each expert's own (b_inner).
 *  ids:          tokens x top_k experts (4-byte aligned), in any order; a value outside
 *                0 .. experts - 1 contributes nothing; an expert named twice counts twice.
 *  weights:      tokens x top_k floats (4-byte aligned).   1 <= top_k <= 32.
 *  gate, up, down codes and scales: one packed matrix each (dq_gemm_pack_weights), the experts'
 *                rows one expert after the other: (experts inner) x K, and (experts out) x inner.
 *                1 <= experts <= 1024; K and inner multiples of 512, out of 32; each at most 2^22.
 *  a_gate, a_up, a_down: experts x inner (x out) floats, 16-byte aligned, or NULL.
 *  b_inner:      experts x inner floats > 0, 16-byte aligned, or NULL.
 *  inner_fmt:    DQ_FMT_MXFP4 or DQ_FMT_MXFP8.
 *  residual:     tokens x out of Y's type, or NULL; may equal Y.
 *  Y:            out, tokens x out, fp32 or bf16 (yt), 16-byte aligned; likewise residual. fp32 where
 *                act_fmt and inner_fmt are MXFP4, for dq_gemm_mx_epilogue's reason.
 *  workspace:    dq_moe_workspace_bytes, 256-byte aligned.
 * A token's result can depend in its last bits on the batch it is in (which kernel, and so which
 * order of the fp32 sums over k, goes by the number of tokens). */
dq_status dq_moe_workspace_bytes(int64_t tokens, int64_t K, int64_t inner, int64_t out,
                                 int64_t experts, int top_k, size_t* bytes);
dq_status dq_moe_mx(const uint8_t* act_codes, const uint8_t* act_scales, dq_format act_fmt,
                    int64_t tokens, int64_t K, const int32_t* ids, const float* weights, int top_k,
                    int64_t experts, const uint8_t* gate_codes, const uint8_t* gate_scales,
                    const float* a_gate, const uint8_t* up_codes, const uint8_t* up_scales,
                    const float* a_up, dq_activation activation, int64_t inner,
                    const float* b_inner, dq_format inner_fmt, const uint8_t* down_codes,
                    const uint8_t* down_scales, const float* a_down, const void* residual,
                    int64_t out, dq_dtype yt, void* Y, void* workspace, size_t workspace_bytes,
                    hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* DQ_LAYER_H */
