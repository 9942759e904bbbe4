// dq_adapter.hip -- the product with packed MXFP4 weights that many requests share, with each token's
// own low-rank adapter beside it:
//
//   Y[t][i] = residual[t][i] + act(a_i s[t][i] + bias_i + scale_r sum_j u[t][j] B_r[i][j])
//   u[t][j] = sum_k X[t][k] A_r[j][k],  r = adapter[t]
//
// Two launches: u (here), then the products of dq_mlp.hip, whose kernels add the adapters' part to
// their sums (adapter_blocks and adapter_tile in dq_mlp_kernels.h). Measured by kernel, us, u + product
// (the product without adapters):
//   32 sequences, 28 of 40 adapters, rank 16, 14336 -> 4096, bf16       8 - 9 + 15   (9)
//   the same from MXFP8 activations                                     8 - 9 + 21   (14)
//   4096 tokens in runs, 6 adapters, rank 64, 4096 -> 14336, bf16       16 - 19 + 141 - 150   (114 - 147)
//   515 tokens in runs, 5 adapters, rank 24, 2560 -> 1733, fp32         8 - 9 + 12   (8 - 9)
// The first reads 13 MB of A next to 31 MB of weights. In the second u is 2 10^9 multiply-adds on 33 MB
// of X: 256 workgroups, of which those of the first slot, every other one and so on four of the eight
// XCDs, have work where a block of tokens has one adapter; each waits for its own loads (1.8 - 2.1
// TB/s). B's products are 1/64 of the main ones but at a quarter of their rate and with a third more
// operands.
#include "../../include/dq_layer.h"
#include "dq_mlp_kernels.h"

namespace dqm {

struct RankArgs {
  const uint16_t* X;     // tokens x K, bf16
  const int* adapter;    // tokens
  const uint16_t* A;     // adapters x rank x K, bf16
  const float* scale;    // adapters, or null (parts)
  uint16_t* parts;       // as struct Adapters has them, or null
  float* u;              // else slices x tokens x rank
  int64_t stride;        // from a slice of u to the next
  int tokens, K, adapters, rank;
  int slots, slices;     // workgroups that share a block of tokens: by adapters, by k
};

// A workgroup takes 32 tokens, 32 MR of the rank values and one slice of k, for the slot-th, slot +
// slots-th, .. of the distinct adapters of its tokens; its W waves share the slice in periods of 64 k
// (a cache line of every row) and join their sums in LDS in wave order.
//
// V_MFMA_F32_32X32X16_BF16 takes A's rows as operand A and the tokens as operand B; lane half h takes
// pieces 2 i + h of 8 values of each row's period, the i-th step's. Loaded straight into such
// registers every lane would touch a cache line of its own (32 sequences, rank 16, K
// 14336: 29 us); so rows go to a ring of two LDS stages of the wave's own, eight lanes to a line, their
// pieces XOR-swizzled as the products' tokens are. Rows past the rank, and tokens of other adapters,
// read zeros through an offset past the buffer.
template <int MR, int NP, int W>
__global__ __launch_bounds__(W * 64) void k_adapter_rank(RankArgs p) {
  constexpr int kTile = 32 * kRowB;                 // 32 rows of one period
  constexpr int kRing = 2 * (1 + MR) * kTile;       // a wave's two stages
  constexpr int kJoin = W * MR * kPartBlock * 4;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[W * kRing > kJoin ? W * kRing : kJoin];
  const int lane = threadIdx.x & 63, rl = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nr = (p.rank + 32 * MR - 1) / (32 * MR);
  int b = blockIdx.x;
  const int slot = b % p.slots;
  b /= p.slots;
  const int slice = b % p.slices;
  b /= p.slices;
  const int r0 = (b % nr) * 32 * MR, t0 = (b / nr) * 32;
  auto adapter = [&](int t) {
    const int id = t < p.tokens ? p.adapter[t] : -1;
    return (unsigned)id < (unsigned)p.adapters ? id : -1;
  };
  const int id = adapter(t0 + rl);
  int idr[4];  // of the rows that this lane loads: 8 j + lane / 8
  uint32_t vo[4];
  const uint32_t pitch = (uint32_t)p.K * 2u;
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const int r = 8 * j + (lane >> 3);
    idr[j] = adapter(t0 + r);
    vo[j] = (uint32_t)r * pitch + (uint32_t)(((lane & 7) ^ (r & 7) ^ ((r >> 3) & 1)) * 16);
  }
  const int periods = p.K / 64, per = (periods + p.slices - 1) / p.slices;
  const int from = min(slice * per, periods), to = min(from + per, periods);
  const __amdgpu_buffer_rsrc_t rx =
      rsrc(p.X + (int64_t)t0 * p.K, (uint32_t)min(p.tokens - t0, 32) * pitch);
  const __amdgpu_buffer_rsrc_t rnone = rsrc(p.X, 0u);
  uint8_t* ring = lds + wave * kRing;
  const int xt = (rl & 7) ^ ((rl >> 3) & 1);
  uint32_t left = (uint32_t)__ballot(id >= 0);  // the halves agree
  for (int q = 0; left; q++) {
    const int r = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
    left &= ~(uint32_t)__ballot(id == r);
    if (q % p.slots != slot) continue;
    const __amdgpu_buffer_rsrc_t ra = rsrc(p.A + ((int64_t)r * p.rank + r0) * p.K,
                                           (uint32_t)min(p.rank - r0, 32 * MR) * pitch);
    uint32_t vx[4];
#pragma unroll
    for (int j = 0; j < 4; j++) vx[j] = idr[j] == r ? vo[j] : kOob;
    v16f acc[MR] = {};
    constexpr int kLoads = 4 * (1 + MR);
    auto load = [&](int c, int st) {  // past the last period nothing is read
      const bool on = c < to;
      uint8_t* dst = ring + st * (kRing / 2);
#pragma unroll
      for (int j = 0; j < 4; j++) load_lds(on ? rx : rnone, dst + j * 1024, vx[j], c * kRowB);
#pragma unroll
      for (int m = 0; m < MR; m++)
#pragma unroll
        for (int j = 0; j < 4; j++)
          load_lds(on ? ra : rnone, dst + (1 + m) * kTile + j * 1024, vo[j] + (uint32_t)(32 * m) * pitch,
                   c * kRowB);
    };
    auto stage = [&](int c, int st) {
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(kLoads));
      wave_lds_order();
      const uint8_t* src = ring + st * (kRing / 2) + rl * kRowB;
      bf16x8 x[4], a[MR][4];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int at = ((2 * i + h) ^ xt) * 16;
        x[i] = *reinterpret_cast<const bf16x8*>(src + at);
#pragma unroll
        for (int m = 0; m < MR; m++)
          a[m][i] = *reinterpret_cast<const bf16x8*>(src + (1 + m) * kTile + at);
      }
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): read before the stage is loaded again
      wave_lds_order();
      load(c + 2 * W, st);
#pragma unroll
      for (int i = 0; i < 4; i++)
#pragma unroll
        for (int m = 0; m < MR; m++)
          acc[m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[m][i], x[i], acc[m], 0, 0, 0);
    };
    __syncthreads();  // the adapter before is stored
    load(from + wave, 0);
    load(from + wave + W, 1);
    for (int c = from + wave; c < to; c += 2 * W) {
      stage(c, 0);
      stage(c + W, 1);  // zeros past the last
    }
    // the last loads read nothing but still write zeros into LDS: drain them before the join
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    float* part = reinterpret_cast<float*>(lds);
    __syncthreads();  // every wave is done with its ring
#pragma unroll
    for (int m = 0; m < MR; m++)
#pragma unroll
      for (int g = 0; g < 4; g++)
        *reinterpret_cast<f32x4*>(part + (wave * MR + m) * kPartBlock + rl * kPartRow + g * 8 + h * 4) =
            f32x4{acc[m][4 * g], acc[m][4 * g + 1], acc[m][4 * g + 2], acc[m][4 * g + 3]};
    __syncthreads();
    const float scale = p.parts && p.scale ? p.scale[r] : 1.0f;
    const int steps = (p.rank + 15) / 16;
    for (int i = threadIdx.x; i < 256 * MR; i += W * 64) {
      const int m = i >> 8, tr = (i >> 3) & 31, j = r0 + 32 * m + (i & 7) * 4;
      if (t0 + tr >= p.tokens || j >= (p.parts ? steps * 16 : p.rank) || p.adapter[t0 + tr] != r) continue;
      f32x4 s = {};  // zero past the rank
#pragma unroll
      for (int w = 0; w < W; w++)
        s += *reinterpret_cast<const f32x4*>(part + (w * MR + m) * kPartBlock + tr * kPartRow + (i & 7) * 4);
      if (!p.parts) {
        *reinterpret_cast<f32x4*>(p.u + slice * p.stride + (int64_t)(t0 + tr) * p.rank + j) = s;
        continue;
      }
      bf16x4 v[NP];
#pragma unroll
      for (int e = 0; e < 4; e++) {
        __bf16 w[NP];
        split_bf16<NP>(s[e] * scale, w);
#pragma unroll
        for (int k = 0; k < NP; k++) v[k][e] = w[k];
      }
      uint16_t* at = p.parts + ((int64_t)(t0 / 32) * steps + j / 16) * (NP * 512) +
                     ((j / 8 & 1) * 32 + tr) * 8 + j % 8;
#pragma unroll
      for (int k = 0; k < NP; k++) *reinterpret_cast<bf16x4*>(at + k * 512) = v[k];
    }
  }
}

// ---------------------------------------------------------------------------------- host

constexpr int kMaxRank = 256;

// How the rank values' kernel fills the chip: 32 rank values and eight waves a workgroup with few
// blocks of tokens, 64 and four with many (4096 tokens, K 4096: rank 64 17.7 against 20.0 us, rank 128
// 25.1 against 32.4); slots up to the distinct adapters that a block can have (a slot that finds none
// leaves); and with one block of tokens k in slices (at least 512 each). More blocks have fewer, longer
// workgroups: rank 16, 40 adapters, K 14336, 32 tokens 8.6 us (256 workgroups), 33 and 64 tokens 18.6
// (64), 128 tokens 19.0 (128).
struct RankShape {
  int mr, slots, slices;
  size_t bytes;
  RankShape(int64_t tokens, int64_t K, int rank) {
    const int64_t blocks = (tokens + 31) / 32;
    mr = blocks >= 32 && rank > 32 ? 2 : 1;
    const int64_t wgs = blocks * ((rank + 32 * mr - 1) / (32 * mr));
    slots = (int)std::clamp<int64_t>(256 / wgs, 1, std::min<int64_t>(tokens, 32));
    slices = tokens > kSliceTokens ? 1 : (int)std::clamp<int64_t>(
        256 / (wgs * slots), 1, std::min<int64_t>(K / 512, kMaxSlices));
    bytes = slices > 1 ? (size_t)slices * (size_t)tokens * (size_t)rank * 4
                       : (size_t)blocks * ((rank + 15) / 16) * 3 * 1024;
    bytes = (bytes + 255) / 256 * 256;
  }
};

template <int MR, int NP, int W>
hipError_t launch_rank(const RankArgs& p, hipStream_t s) {
  const int64_t blocks = (int64_t)((p.tokens + 31) / 32) * ((p.rank + 32 * MR - 1) / (32 * MR)) *
                         p.slots * p.slices;
  hipLaunchKernelGGL((k_adapter_rank<MR, NP, W>), dim3((unsigned)blocks), dim3(W * 64), 0, s, p);
  return hipGetLastError();
}

}  // namespace dqm

extern "C" {

dq_status dq_adapter_workspace_bytes(int64_t tokens, int64_t K, int rank, size_t* bytes) {
  using namespace dqm;
  if (!bytes || tokens < 1 || tokens > INT32_MAX - 256 || K < 512 || K % 512 != 0 || K > (1 << 22) ||
      rank < 8 || rank % 8 != 0 || rank > kMaxRank)
    return DQ_ERR_ARG;
  *bytes = RankShape(tokens, K, rank).bytes;
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
  const RankShape shape(tokens, K, rank);
  RankArgs r{};
  r.X = static_cast<const uint16_t*>(X);
  r.adapter = adapter;
  r.A = static_cast<const uint16_t*>(A);
  r.scale = scale;
  if (shape.slices == 1) r.parts = static_cast<uint16_t*>(workspace);
  else r.u = static_cast<float*>(workspace);
  r.stride = tokens * rank;
  r.K = (int)K;
  r.adapters = (int)adapters;
  r.rank = rank;
  r.slots = shape.slots;
  r.slices = shape.slices;
  // rounds of tokens so that no grid passes 2^31 threads
  const int64_t chunk = 1 << 20;
  for (int64_t t = 0; t < tokens; t += chunk) {
    RankArgs p = r;
    p.X += t * K;
    p.adapter += t;
    if (p.parts) p.parts += t / 32 * ((rank + 15) / 16) * ((yt == DQ_F32 ? 3 : 2) * 512);
    else p.u += t * rank;
    p.tokens = (int)std::min(chunk, tokens - t);
    const bool f32 = yt == DQ_F32;
    const hipError_t e =
        shape.mr == 1 ? (f32 ? launch_rank<1, 3, 8>(p, stream) : launch_rank<1, 2, 8>(p, stream))
                      : (f32 ? launch_rank<2, 3, 4>(p, stream) : launch_rank<2, 2, 4>(p, stream));
    if (e != hipSuccess) return DQ_ERR_HIP;
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
  x.parts = r.parts;
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
