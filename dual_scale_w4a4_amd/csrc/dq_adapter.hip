// dq_adapter.hip -- the product with packed MXFP4 weights that many requests share, with each token's
// own low-rank adapter beside it:
//
//   Y[t][i] = residual[t][i] + act(a_i s[t][i] + bias_i + scale_r sum_j u[t][j] B_r[i][j])
//   u[t][j] = sum_k X[t][k] A_r[j][k],  r = adapter[t]
//
// Two launches: u (here), then the products of dq_mlp.hip, whose kernels add the adapters' part to
// their sums (adapter_block in dq_mlp_kernels.h).
#include "../../include/dq_layer.h"
#include "dq_mlp_kernels.h"

namespace dqm {

struct RankArgs {
  const uint16_t* X;     // tokens x K, bf16
  const int* adapter;    // tokens
  const uint16_t* A;     // adapters x rank x K, bf16
  float* u;              // slices x tokens x rank
  int64_t stride;        // from a slice of u to the next
  int tokens, K, adapters, rank;
  int slots, slices;     // workgroups that share a block of tokens: by adapters, by k
};

// A workgroup takes 32 tokens, 32 of the rank values and one slice of k, for the slot-th, slot +
// slots-th, .. of the distinct adapters of its tokens; its waves share the slice in periods of 64 k
// and join their sums in LDS in wave order. V_MFMA_F32_32X32X16_BF16 takes A's rows as operand A and the
// tokens as operand B; of each 64 k (a cache line of every row) lane half h takes chunks 2 i + h of
// 8, the i-th step's.
__global__ __launch_bounds__(256) void k_adapter_rank(RankArgs p) {
  __shared__ float part[4][kPartBlock];
  const int lane = threadIdx.x & 63, rl = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nr = (p.rank + 31) / 32;
  int b = blockIdx.x;
  const int slot = b % p.slots;
  b /= p.slots;
  const int slice = b % p.slices;
  b /= p.slices;
  const int r0 = (b % nr) * 32, t0 = (b / nr) * 32;
  const int t = t0 + rl;
  int id = t < p.tokens ? p.adapter[t] : -1;
  if ((unsigned)id >= (unsigned)p.adapters) id = -1;
  const int periods = p.K / 64, per = (periods + p.slices - 1) / p.slices;
  const int from = slice * per, to = min(from + per, periods);
  const uint16_t* x = p.X + (int64_t)min(t, p.tokens - 1) * p.K + 8 * h;
  uint32_t left = (uint32_t)__ballot(id >= 0);  // the halves agree
  for (int q = 0; left; q++) {
    const int r = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
    left &= ~(uint32_t)__ballot(id == r);
    if (q % p.slots != slot) continue;
    // rows past the rank read the last one; their results are not stored
    const uint16_t* a = p.A + ((int64_t)r * p.rank + min(r0 + rl, p.rank - 1)) * p.K + 8 * h;
    v16f acc = {};
    for (int c = from + wave; c < to; c += 4) {
      bf16x8 av[4], xv[4];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        av[i] = *reinterpret_cast<const bf16x8*>(a + c * 64 + 16 * i);
        xv[i] = *reinterpret_cast<const bf16x8*>(x + c * 64 + 16 * i);
      }
#pragma unroll
      for (int i = 0; i < 4; i++)
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(av[i], xv[i], acc, 0, 0, 0);
    }
    __syncthreads();  // the adapter before is stored
#pragma unroll
    for (int g = 0; g < 4; g++)
      *reinterpret_cast<f32x4*>(&part[wave][rl * kPartRow + g * 8 + h * 4]) =
          f32x4{acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]};
    __syncthreads();
    const int tr = threadIdx.x >> 3, j = (threadIdx.x & 7) * 4;
    const bool mine = t0 + tr < p.tokens && p.adapter[t0 + tr] == r;
    if (mine && r0 + j < p.rank) {
      f32x4 s = {};
#pragma unroll
      for (int w = 0; w < 4; w++) s += *reinterpret_cast<const f32x4*>(&part[w][tr * kPartRow + j]);
      *reinterpret_cast<f32x4*>(p.u + slice * p.stride + (int64_t)(t0 + tr) * p.rank + r0 + j) = s;
    }
  }
}

// ---------------------------------------------------------------------------------- host

constexpr int kMaxRank = 256, kMaxSlices = 8;

// How the rank values' kernel fills the chip: slots up to the distinct adapters that a block of 32
// tokens can have, then slices of k (at least 512 each).
void rank_shape(int64_t tokens, int64_t K, int rank, int* slots, int* slices) {
  const int64_t blocks = (tokens + 31) / 32 * ((rank + 31) / 32);
  *slots = (int)std::clamp<int64_t>(256 / blocks, 1, std::min<int64_t>(tokens, 32));
  *slices = (int)std::clamp<int64_t>(512 / (blocks * *slots), 1,
                                     std::min<int64_t>(K / 512, kMaxSlices));
}

}  // namespace dqm

extern "C" {

dq_status dq_adapter_workspace_bytes(int64_t tokens, int64_t K, int rank, size_t* bytes) {
  using namespace dqm;
  if (!bytes || tokens < 1 || tokens > INT32_MAX - 256 || K < 512 || K % 512 != 0 || K > (1 << 22) ||
      rank < 8 || rank % 8 != 0 || rank > kMaxRank)
    return DQ_ERR_ARG;
  int slots, slices;
  rank_shape(tokens, K, rank, &slots, &slices);
  *bytes = ((size_t)slices * (size_t)tokens * (size_t)rank * 4 + 255) / 256 * 256;
  return DQ_OK;
}

dq_status dq_gemm_mx_adapters(const uint8_t* act_codes, const uint8_t* act_scales, dq_format act_fmt,
                              int64_t tokens, int64_t K, const uint8_t* packed_codes,
                              const uint8_t* packed_scales, const float* a, const float* bias,
                              const void* X, const int32_t* adapter, int64_t adapters, int rank,
                              const void* A, const void* B, const float* scale,
                              dq_activation activation, const void* residual, int64_t out,
                              dq_dtype yt, void* Y, void* workspace, size_t workspace_bytes,
                              hipStream_t stream) {
  using namespace dqm;
  const dq_status st = check_product(act_codes, act_scales, act_fmt, tokens, K, packed_codes,
                                     packed_scales, a, out, activation);
  if (st != DQ_OK) return st;
  if ((yt != DQ_F32 && yt != DQ_BF16) || (yt == DQ_F32 && act_fmt == DQ_FMT_MXFP8))
    return DQ_ERR_UNSUPPORTED;
  const size_t esz = yt == DQ_BF16 ? 2 : 4;
  size_t need = 0;
  if (dq_adapter_workspace_bytes(tokens, K, rank, &need) != DQ_OK) return DQ_ERR_ARG;
  if (!Y || !X || !adapter || !A || !B || !workspace) return DQ_ERR_ARG;
  if (adapters < 1 || adapters > (1 << 20)) return DQ_ERR_ARG;
  if (((uintptr_t)bias | (uintptr_t)X | (uintptr_t)A | (uintptr_t)B) & 15u) return DQ_ERR_ARG;
  if (((uintptr_t)adapter | (uintptr_t)scale) & 3u) return DQ_ERR_ARG;
  if (((uintptr_t)Y | (uintptr_t)residual) & (esz - 1)) return DQ_ERR_ARG;
  if ((uintptr_t)workspace & 255u) return DQ_ERR_ARG;
  if (workspace_bytes < need) return DQ_ERR_WORKSPACE;
  const size_t bytes = (size_t)tokens * (size_t)out * esz;
  const size_t wb = packed_bytes(out, K), vb = (size_t)out * 4;
  const size_t ranks = (size_t)adapters * (size_t)rank;
  if (dq::any_overlap({{Y, bytes}, {workspace, need}},
                      {{residual == Y ? nullptr : residual, bytes},
                       {act_codes, act_bytes(act_fmt, tokens, K)},
                       {act_scales, (size_t)(tokens * (K / 32))},
                       {packed_codes, wb},
                       {packed_scales, wb / 16},
                       {a, vb},
                       {bias, vb},
                       {X, (size_t)tokens * (size_t)K * 2},
                       {adapter, (size_t)tokens * 4},
                       {A, ranks * (size_t)K * 2},
                       {B, ranks * (size_t)out * 2},
                       {scale, (size_t)adapters * 4}}))
    return DQ_ERR_ARG;
  RankArgs r{};
  r.X = static_cast<const uint16_t*>(X);
  r.adapter = adapter;
  r.A = static_cast<const uint16_t*>(A);
  r.u = static_cast<float*>(workspace);
  r.stride = tokens * rank;
  r.K = (int)K;
  r.adapters = (int)adapters;
  r.rank = rank;
  rank_shape(tokens, K, rank, &r.slots, &r.slices);
  // rounds of tokens so that no grid passes 2^31 threads
  const int64_t chunk = 1 << 20;
  for (int64_t t = 0; t < tokens; t += chunk) {
    RankArgs p = r;
    p.X += t * K;
    p.adapter += t;
    p.u += t * rank;
    p.tokens = (int)std::min(chunk, tokens - t);
    const int64_t blocks = (int64_t)((p.tokens + 31) / 32) * ((rank + 31) / 32) * p.slots * p.slices;
    hipLaunchKernelGGL(k_adapter_rank, dim3((unsigned)blocks), dim3(256), 0, stream, p);
    if (hipGetLastError() != hipSuccess) return DQ_ERR_HIP;
  }
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
  Adapters x{};
  x.u = r.u;
  x.adapter = adapter;
  x.B = static_cast<const uint16_t*>(B);
  x.scale = scale;
  x.adapters = r.adapters;
  x.rank = rank;
  x.slices = r.slices;
  x.stride = r.stride;
  const bool act8 = act_fmt == DQ_FMT_MXFP8;
  const hipError_t e = yt == DQ_BF16 ? launch_o<false, kOutBf16>(p, x, act8, stream)
                                     : launch_o<false, kOutF32>(p, x, false, stream);
  return e == hipSuccess ? DQ_OK : DQ_ERR_HIP;
}

}  // extern "C"
