// dq_route.hip -- the router of a layer of experts: each token's scores of the experts, its top_k of
// them and their weights.
//
// Which experts a token takes must not depend on the order of a sum, so a logit is the fp64 sum of
// the exact products rounded once to fp32, and scores and selection keys are fp64.
//
// Two launches. The logits: with few tokens a wave takes one expert and up to 8 tokens, k over its
// lanes; with more the fp64 matrix instruction takes tiles of 32 tokens by 32 experts a wave, k over
// the workgroup's waves. Then a wave per token selects.
#include <float.h>
#include <limits.h>

#include <algorithm>

#include "../../include/dq_layer.h"
#include "dq_outq.h"

namespace dqr {

using dq::u2f;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxExperts = 1024;

struct LogitArgs {
  const void* X;    // tokens x cols
  const void* W;    // experts x cols
  float* logits;    // tokens x experts
  int64_t tokens;
  int cols, experts;
};

// 8 consecutive values as fp32
template <bool BF>
__device__ __forceinline__ void load8(const void* p, int64_t off, float (&v)[8]) {
  if (BF) {
    const u32x4 u = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + off);
#pragma unroll
    for (int k = 0; k < 4; k++) {
      v[2 * k] = u2f(u[k] << 16);
      v[2 * k + 1] = u2f(u[k] & 0xFFFF0000u);
    }
  } else {
    const u32x4* s = reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + off);
#pragma unroll
    for (int k = 0; k < 8; k++) v[k] = u2f(s[k / 4][k % 4]);
  }
}

// Wave: one expert, T tokens; lane l takes 8 channels of every 512.
template <bool XB, bool WB, int T>
__global__ __launch_bounds__(256) void k_logits_few(LogitArgs p) {
  const int lane = threadIdx.x & 63;
  const int ne = (p.experts + 3) / 4;
  const int e = (blockIdx.x % ne) * 4 + (threadIdx.x >> 6);
  const int64_t t0 = (int64_t)(blockIdx.x / ne) * T;
  if (e >= p.experts) return;
  const int n = (int)min((int64_t)T, p.tokens - t0);
  double sum[T] = {};
  for (int c = lane * 8; c < p.cols; c += 512) {
    float w[8];
    load8<WB>(p.W, (int64_t)e * p.cols + c, w);
#pragma unroll
    for (int t = 0; t < T; t++) {
      float x[8];
      load8<XB>(p.X, (t0 + min(t, n - 1)) * p.cols + c, x);
#pragma unroll
      for (int k = 0; k < 8; k++) sum[t] = fma((double)x[k], (double)w[k], sum[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < T; t++) {
    const double s = dq::wave_sum(sum[t]);
    if (lane == 0 && t < n) p.logits[(t0 + t) * p.experts + e] = (float)s;
  }
}

// Workgroup of W waves: 32 tokens by 32 experts, wave w taking channels 32 w .. of every 32 W (one
// wave's partial sums joined in wave order). V_MFMA_F64_16X16X4: lane l holds row (column) l % 16,
// k l / 16; result v of lane l is D[4 v + l / 16][l % 16]. The order of k inside a sum is free, so
// lane quarter q takes channels 8 q .. 8 q + 7 of the 32, in 8 steps.
template <bool XB, bool WB, int W>
__global__ __launch_bounds__(W * 64) void k_logits_many(LogitArgs p) {
  __shared__ double part[W][4][4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int rl = lane & 15, q = lane >> 4;
  const int ne = (p.experts + 31) / 32;
  const int e0 = (blockIdx.x % ne) * 32;
  const int64_t t0 = (int64_t)(blockIdx.x / ne) * 32;
  // rows past the end read the last one; their results are not stored
  int64_t xo[2], wo[2];
#pragma unroll
  for (int m = 0; m < 2; m++) {
    xo[m] = min(t0 + 16 * m + rl, p.tokens - 1) * p.cols;
    wo[m] = (int64_t)min(e0 + 16 * m + rl, p.experts - 1) * p.cols;
  }
  f64x4 acc[2][2] = {};
  for (int c0 = wave * 32; c0 < p.cols; c0 += W * 32) {
    const int c = c0 + 8 * q;
    float x[2][8] = {}, w[2][8] = {};
    if (c < p.cols) {
#pragma unroll
      for (int m = 0; m < 2; m++) {
        load8<XB>(p.X, xo[m] + c, x[m]);
        load8<WB>(p.W, wo[m] + c, w[m]);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; k++)
#pragma unroll
      for (int m = 0; m < 2; m++)
#pragma unroll
        for (int n = 0; n < 2; n++)
          acc[m][n] = __builtin_amdgcn_mfma_f64_16x16x4f64((double)x[m][k], (double)w[n][k],
                                                           acc[m][n], 0, 0, 0);
  }
#pragma unroll
  for (int m = 0; m < 2; m++)
#pragma unroll
    for (int n = 0; n < 2; n++)
#pragma unroll
      for (int v = 0; v < 4; v++) part[wave][2 * m + n][v][lane] = acc[m][n][v];
  __syncthreads();
  for (int i = threadIdx.x; i < 1024; i += W * 64) {
    const int b = i >> 8, v = (i >> 6) & 3, l = i & 63;
    double s = 0.0;
    for (int w = 0; w < W; w++) s += part[w][b][v][l];
    const int64_t t = t0 + 16 * (b >> 1) + 4 * v + (l >> 4);
    const int e = e0 + 16 * (b & 1) + (l & 15);
    if (t < p.tokens && e < p.experts) p.logits[t * p.experts + e] = (float)s;
  }
}

struct SelectArgs {
  const float* logits;
  const float* bias;   // experts, or null
  int* ids;
  float* weights;
  int64_t tokens;
  int experts, top_k, renormalize;
  float scale;
};

// Wave: one token; lane l holds experts l, l + 64, ... N of them. The k-th largest key is found k
// times: the largest of each lane's, then of the wave's, ties to the lower index; a taken key becomes
// -inf. NaN keys rank as -inf, and -inf keys by index.
template <bool SIGMOID, int N>
__global__ __launch_bounds__(256) void k_select(SelectArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= p.tokens) return;
  double score[N], key[N];
  bool free_[N];
  double top = -INFINITY;
#pragma unroll
  for (int n = 0; n < N; n++) {
    const int e = n * 64 + lane;
    free_[n] = e < p.experts;
    score[n] = free_[n] ? (double)p.logits[t * p.experts + e] : -INFINITY;
    top = fmax(top, score[n]);
  }
  double total = 1.0;
  if (SIGMOID) {
#pragma unroll
    for (int n = 0; n < N; n++) score[n] = 1.0 / (1.0 + exp(-score[n]));
  } else {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) top = fmax(top, __shfl_xor(top, m, 64));
    double sum = 0.0;
#pragma unroll
    for (int n = 0; n < N; n++) {
      score[n] = free_[n] ? exp(score[n] - top) : 0.0;
      sum += score[n];
    }
    total = dq::wave_sum(sum);
#pragma unroll
    for (int n = 0; n < N; n++) score[n] = score[n] / total;
  }
#pragma unroll
  for (int n = 0; n < N; n++) {
    const int e = n * 64 + lane;
    key[n] = score[n] + (p.bias && free_[n] ? (double)p.bias[e] : 0.0);
    if (!(key[n] == key[n])) key[n] = -INFINITY;
  }
  double chosen = 0.0, mine = 0.0;  // the sum of the chosen scores; lane k: the k-th chosen
  int id = 0;
  for (int k = 0; k < p.top_k; k++) {
    double best = -INFINITY;
    int at = INT_MAX;
#pragma unroll
    for (int n = 0; n < N; n++)
      if (free_[n] && (at == INT_MAX || key[n] > best)) {
        best = key[n];
        at = n * 64 + lane;
      }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const double b = __shfl_xor(best, m, 64);
      const int a = __shfl_xor(at, m, 64);
      if (b > best || (b == best && a < at)) {
        best = b;
        at = a;
      }
    }
    double s = 0.0;
#pragma unroll
    for (int n = 0; n < N; n++)
      if (n * 64 + lane == at) {
        free_[n] = false;
        s = score[n];
      }
    s = __shfl(s, at & 63, 64);
    chosen += s;
    if (lane == k) {
      mine = s;
      id = at;
    }
  }
  if (lane < p.top_k) {
    double w = mine;
    if (p.renormalize) w = chosen == 0.0 ? 0.0 : mine / chosen;
    p.ids[t * p.top_k + lane] = id;
    p.weights[t * p.top_k + lane] = (float)(w * (double)p.scale);
  }
}

// ---------------------------------------------------------------------------------- host

constexpr int kMaxTopK = 32;

template <bool XB, bool WB>
hipError_t launch_logits(const LogitArgs& p, hipStream_t s) {
  if (p.tokens <= 64) {
    const int64_t ne = (p.experts + 3) / 4;
    if (p.tokens == 1)
      hipLaunchKernelGGL((k_logits_few<XB, WB, 1>), dim3((unsigned)ne), dim3(256), 0, s, p);
    else
      hipLaunchKernelGGL((k_logits_few<XB, WB, 4>), dim3((unsigned)(ne * ((p.tokens + 3) / 4))),
                         dim3(256), 0, s, p);
  } else {
    const int64_t n = (int64_t)((p.experts + 31) / 32) * ((p.tokens + 31) / 32);
    hipLaunchKernelGGL((k_logits_many<XB, WB, 4>), dim3((unsigned)n), dim3(256), 0, s, p);
  }
  return hipGetLastError();
}

template <bool SIGMOID>
hipError_t launch_select(const SelectArgs& p, hipStream_t s) {
  const dim3 grid((unsigned)((p.tokens + 3) / 4)), block(256);
  if (p.experts <= 64) hipLaunchKernelGGL((k_select<SIGMOID, 1>), grid, block, 0, s, p);
  else if (p.experts <= 128) hipLaunchKernelGGL((k_select<SIGMOID, 2>), grid, block, 0, s, p);
  else if (p.experts <= 256) hipLaunchKernelGGL((k_select<SIGMOID, 4>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((k_select<SIGMOID, 16>), grid, block, 0, s, p);
  return hipGetLastError();
}

}  // namespace dqr

extern "C" {

dq_status dq_moe_route_workspace_bytes(int64_t tokens, int64_t experts, size_t* bytes) {
  using namespace dqr;
  if (!bytes || tokens < 1 || tokens > INT32_MAX - 256 || experts < 1 || experts > kMaxExperts)
    return DQ_ERR_ARG;
  *bytes = ((size_t)tokens * (size_t)experts * 4 + 255) / 256 * 256;
  return DQ_OK;
}

dq_status dq_moe_route(const void* X, dq_dtype xt, int64_t tokens, int64_t cols, const void* W,
                       dq_dtype wt, int64_t experts, const float* bias, dq_score score, int top_k,
                       int renormalize, float scale, int32_t* ids, float* weights, void* workspace,
                       size_t workspace_bytes, hipStream_t stream) {
  using namespace dqr;
  if ((xt != DQ_F32 && xt != DQ_BF16) || (wt != DQ_F32 && wt != DQ_BF16)) return DQ_ERR_UNSUPPORTED;
  if (score != DQ_SCORE_SOFTMAX && score != DQ_SCORE_SIGMOID) return DQ_ERR_UNSUPPORTED;
  if (!X || !W || !ids || !weights || !workspace) return DQ_ERR_ARG;
  size_t need = 0;
  if (dq_moe_route_workspace_bytes(tokens, experts, &need) != DQ_OK) return DQ_ERR_ARG;
  if (cols < 8 || cols % 8 != 0 || cols > (1 << 22)) return DQ_ERR_ARG;
  if (top_k < 1 || top_k > kMaxTopK || top_k > experts) return DQ_ERR_ARG;
  if ((renormalize != 0 && renormalize != 1) || !(fabsf(scale) <= FLT_MAX)) return DQ_ERR_ARG;
  if (((uintptr_t)X | (uintptr_t)W) & 15u) return DQ_ERR_ARG;
  if (((uintptr_t)ids | (uintptr_t)weights | (uintptr_t)bias) & 3u) return DQ_ERR_ARG;
  if ((uintptr_t)workspace & 255u) return DQ_ERR_ARG;
  if (workspace_bytes < need) return DQ_ERR_WORKSPACE;
  const size_t n = (size_t)tokens * top_k * 4;
  if (dq::any_overlap({{ids, n}, {weights, n}, {workspace, need}},
                      {{X, (size_t)tokens * (size_t)cols * (xt == DQ_BF16 ? 2 : 4)},
                       {W, (size_t)experts * (size_t)cols * (wt == DQ_BF16 ? 2 : 4)},
                       {bias, (size_t)experts * 4}}))
    return DQ_ERR_ARG;
  // rounds of tokens so that no grid passes 2^31 threads
  const int64_t chunk = 1 << 22;
  for (int64_t t = 0; t < tokens; t += chunk) {
    LogitArgs l{};
    l.X = static_cast<const char*>(X) + t * cols * (xt == DQ_BF16 ? 2 : 4);
    l.W = W;
    l.logits = static_cast<float*>(workspace) + t * experts;
    l.tokens = std::min(chunk, tokens - t);
    l.cols = (int)cols;
    l.experts = (int)experts;
    hipError_t e;
    if (xt == DQ_BF16) e = wt == DQ_BF16 ? launch_logits<true, true>(l, stream)
                                         : launch_logits<true, false>(l, stream);
    else e = wt == DQ_BF16 ? launch_logits<false, true>(l, stream)
                           : launch_logits<false, false>(l, stream);
    if (e != hipSuccess) return DQ_ERR_HIP;
    SelectArgs s{};
    s.logits = l.logits;
    s.bias = bias;
    s.ids = ids + t * top_k;
    s.weights = weights + t * top_k;
    s.tokens = l.tokens;
    s.experts = l.experts;
    s.top_k = top_k;
    s.renormalize = renormalize;
    s.scale = scale;
    e = score == DQ_SCORE_SIGMOID ? launch_select<true>(s, stream) : launch_select<false>(s, stream);
    if (e != hipSuccess) return DQ_ERR_HIP;
  }
  return DQ_OK;
}

}  // extern "C"
