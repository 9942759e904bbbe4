// dq_moe.hip -- a layer of experts on MXFP4 weights: every token's gated products and down products
// with its own experts' weights, and their weighted sum.
//
// The rows of the products are pairs of a token and one of its experts. A workgroup takes a tile of
// the pairs of one expert (find_tile in dq_mlp_kernels.h), so an expert's weights are read once per
// tile, and the kernels are those of the dense MLP with gathered rows. Three launches:
//   gated products of the pairs, quantized     -> q (pairs x inner) in the workspace
//   down products of the pairs, in fp32        -> y (pairs x out) in the workspace
//   weighted sums over each token's pairs      -> Y
// With more than kInlinePairs pairs a small launch before them sorts the pairs by expert.
//
// Few tokens read every expert that they name once: memory bounds them. Prompts are bound as the dense
// products are, and by tiles that an expert's last rows leave unfilled. Measured, us:
//   experts, top k, K -> inner -> K, tokens             sort   gated   down   sum   in all
//   64, 8, 2048 -> 1024, 1 token (27 MB)                       7.3     5.8    2.3   15.4
//   64, 8, 4096 -> 1536, 24 tokens (618 MB)                    67      43     4.6   114, 5.4 TB/s
//   8, 2, 4096 -> 14336, 5 tokens, MXFP8 (572 MB)              67      39     4.6   93 - 111, 5.1 - 6.1 TB/s
//   32, 4, 4096 -> 1536, 700 tokens (335 MB)            4.6    56      48     12    119, 0.89 PFLOP/s
#include "../../include/dq_layer.h"
#include "dq_mlp_kernels.h"

namespace dqm {

// counts[e], and the pairs of expert e in ascending order behind those of the experts before it.
// Workgroup e looks at every id: those below e give its place, its own their order. Wave w takes the
// w-th sixteenth of the pairs. 65536 pairs of 64 experts: two sweeps of 64 loads a wave.
__global__ __launch_bounds__(1024) void k_moe_plan(const int* ids, int pairs, int experts, int* counts,
                                                   int* order) {
  __shared__ int own[16], below[16];
  const int e = blockIdx.x, lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int share = ((pairs + 1023) / 1024) * 64;
  const int from = min(wave * share, pairs), to = min(from + share, pairs);
  int mine = 0, less = 0;
  for (int i = from; i < to; i += 256) {  // four loads in flight
    int id[4];
#pragma unroll
    for (int k = 0; k < 4; k++) id[k] = i + 64 * k + lane < to ? ids[i + 64 * k + lane] : -1;
#pragma unroll
    for (int k = 0; k < 4; k++) {
      mine += __popcll(__ballot(id[k] == e));
      less += __popcll(__ballot(id[k] >= 0 && id[k] < e));
    }
  }
  if (lane == 0) {
    own[wave] = mine;
    below[wave] = less;
  }
  __syncthreads();
  int at = 0, total = 0;
  for (int w = 0; w < 16; w++) {
    at += below[w];
    total += own[w];
    if (w < wave) at += own[w];
  }
  if (threadIdx.x == 0) counts[e] = total;
  for (int i = from; i < to; i += 256) {
    bool is[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const int at = i + 64 * k + lane;
      is[k] = at < to && ids[min(at, to - 1)] == e;
    }
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const uint64_t m = __ballot(is[k]);
      if (is[k])
        order[at + __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32),
                                             __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u))] =
            i + 64 * k + lane;
      at += __popcll(m);
    }
  }
}

struct SumArgs {
  const float* y;        // tokens x top_k x out
  const int* ids;
  const float* weights;
  const void* res;       // or null
  void* Y;
  int64_t tokens;
  int out, top_k, experts;
};

// Y = res + sum_s w_s y_s, 4 channels a thread
template <bool BF>
__global__ __launch_bounds__(256) void k_moe_sum(SumArgs p) {
  typedef typename std::conditional<BF, __bf16, float>::type T;
  typedef typename std::conditional<BF, bf16x4, f32x4>::type T4;
  const int per = (p.out + 1023) / 1024;
  const int64_t t = blockIdx.x / per;
  const int ch = (blockIdx.x % per) * 1024 + threadIdx.x * 4;
  if (ch >= p.out) return;
  const float* y = p.y + t * p.top_k * p.out + ch;
  f32x4 sum = {};
  // eight experts at a time, all their loads in flight; one out of range has no y
  constexpr int kAt = 8;
  for (int s0 = 0; s0 < p.top_k; s0 += kAt) {
    f32x4 v[kAt];
    float w[kAt];
    bool in[kAt];
#pragma unroll
    for (int s = 0; s < kAt; s++) {
      const int at = min(s0 + s, p.top_k - 1);
      w[s] = p.weights[t * p.top_k + at];
      in[s] = s0 + s < p.top_k && (unsigned)p.ids[t * p.top_k + at] < (unsigned)p.experts;
      v[s] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(y + (int64_t)at * p.out));
    }
#pragma unroll
    for (int s = 0; s < kAt; s++)
#pragma unroll
      for (int k = 0; k < 4; k++) sum[k] = in[s] ? sum[k] + w[s] * v[s][k] : sum[k];
  }
  const int64_t off = t * p.out + ch;
  if (p.res) {
    const T4 r = *reinterpret_cast<const T4*>(static_cast<const T*>(p.res) + off);
#pragma unroll
    for (int k = 0; k < 4; k++) sum[k] = (float)r[k] + sum[k];
  }
  *reinterpret_cast<T4*>(static_cast<T*>(p.Y) + off) = T4{(T)sum[0], (T)sum[1], (T)sum[2], (T)sum[3]};
}

// ---------------------------------------------------------------------------------- host

constexpr int kMaxTopK = 32;

// The most tokens that a round of launches takes: every array's bytes stay below 2^31 (offsets are
// 32-bit in the kernels) and every grid below 2^31 threads.
int64_t moe_chunk(int64_t tokens, int64_t K, int64_t inner, int64_t out, int64_t experts, int top_k) {
  const int64_t row = std::max({K, top_k * inner, top_k * out * 4});
  const int64_t blocks = std::max(inner, out) / 32;
  int64_t n = std::min(tokens, (int64_t)INT32_MAX / row);
  while (n > 1 && blocks * (std::min(n * top_k, experts) + n * top_k / 32) > (1 << 23)) n = (n + 1) / 2;
  return n;
}

// The workspace of a round of n tokens
struct MoeSpace {
  size_t codes, scales, y, counts, order, bytes;
  MoeSpace(int64_t n, int64_t inner, int64_t out, int64_t experts, int top_k) {
    const size_t pairs = (size_t)n * top_k;
    size_t at = 0;
    auto take = [&](size_t b) {
      const size_t here = at;
      at += (b + 255) / 256 * 256;
      return here;
    };
    codes = take(pairs * inner);
    scales = take(pairs * (inner / 32));
    y = take(pairs * out * 4);
    counts = take(experts * 4);
    order = take(pairs * 4);
    bytes = at;
  }
};

bool moe_sizes(int64_t tokens, int64_t K, int64_t inner, int64_t out, int64_t experts, int top_k) {
  constexpr int64_t kMost = 1 << 22;
  return tokens >= 1 && tokens <= INT32_MAX - 256 && K >= 512 && K % 512 == 0 && K <= kMost &&
         inner >= 512 && inner % 512 == 0 && inner <= kMost && out >= 32 && out % 32 == 0 &&
         out <= kMost && experts >= 1 && experts <= kMaxExperts && top_k >= 1 && top_k <= kMaxTopK;
}

// Which kernel: the tile kernel, of 64 rows of an expert or 128, where an expert has a few rows and
// there are tiles for the whole chip, or many rows; else tiles of 32 rows with k split over the waves.
// Measured, us, gated and down product (number of workgroups of the tiles):
//   experts, top k, K -> inner, tokens (mean rows)   split, 32 rows   tiles of 64             of 128
//   64, 8, 2048 -> 1024, 32 (4)                      63 in all        51 in all
//   64, 8, 4096 -> 1536, 24 (3)                      119 in all       114 in all
//   64, 8, 4096 -> 1536, 40 (5)                      79 + 58          72 (828) + 46 (1104)
//   64, 8, 2048 -> 1024, 60 (7)                      40 + 31          31 (568) + 21 (568)
//   8, 2, 4096 -> 4096, 32 (8)                       29 + 17          30 (288) + 30 (144)
//   32, 4, 4096 -> 1536, 64 (8)                      42 + 33          44 (432) + 24 (576)
//   32, 4, 4096 -> 1536, 128 (16)                    51 + 40          48 (480) + 29 (640)     51 + 32
//   8, 2, 4096 -> 4096, 100 (25)                     37 + 25          33 (352) + 32 (176)     35 + 37
//   4, 2, 4096 -> 2048, 100 (50)                     15 + 12          17 (112) + 15 (112)
//   8, 2, 4096 -> 2048, 200 (50)                     28 + 25          25 (224) + 21 (224)
//   8, 2, 2048 -> 1024, 300 (75)                     14 + 12          14 (136) + 12 (136)
//   4, 2, 4096 -> 4096, 300 (150)                    55 + 38          34 (416) + 33 (208)     30 (256) + 39 (128)
//   8, 2, 4096 -> 14336, 600 (150)                   344 + 186        166 (2912) + 127 (416)  147 (1904) + 117 (272)
//   8, 2, 2048 -> 2048, 600 (150)                    30 + 22          17 (416) + 16 (208)     17 (272) + 21 (136)
//   64, 8, 2048 -> 1024, 3000 (375)                  246 + 243        103 (3512) + 110 (3512) 93 (2008) + 102 (2008)
// The gated product of MXFP8 activations, which takes two matrix instructions for one:
//   4, 2, 4096 -> 2048, 100 (50)                     18               34 (112)                61
//   8, 2, 4096 -> 2048, 200 (50)                     37               43 (224)                65
//   4, 4, 6144 -> 1536, 151 (151)                    39               53 (192)                93
//   4, 2, 4096 -> 4096, 300 (150)                    73               58 (416)                70
//   8, 2, 4096 -> 14336, 600 (150)                   457              295 (2912)              352
//   64, 8, 2048 -> 1024, 3000 (375)                  342              210 (3512)              201
// Both products, by the kernel of each (* the rule's):
//   gated, down:                                     split, split  tiles, split  split, tiles  tiles, tiles
//   8, 2, 4096 -> 14336, 12 (3)                      121           131 *         170           180
//   8, 2, 4096 -> 14336, 32 (8)                      139           143 *         183           187
//   16, 2, 4096 -> 6144, 32 (4)                      109           113 *         116           119
//   32, 4, 4096 -> 1536, 64 (8)                      80            84            72            76 *
//   64, 8, 4096 -> 1536, 40 (5)                      144           140           131           126 *
//   64, 8, 2048 -> 1024, 60 (7)                      74            66            65            57 *
//   MXFP8: 8, 2, 4096 -> 14336, 12 (3)               125           147 *         173           195
//   64, 8, 4096 -> 1536, 24 (3)                      128           150           120           141 *
//   64, 8, 2048 -> 1024, 60 (7)                      76            69            66            59 *
// The rule goes by the mean of even routing and by the tiles. It does not know K: at K 4096 few rows of
// few or of MXFP8 activations' experts would be up to 18% faster with split gated products, which lose
// about as much at K 2048.
template <bool ACT8, bool GATED, int OUT>
hipError_t launch_experts(const MlpArgs& p, Experts x, hipStream_t s) {
  constexpr int kRows = GATED ? 128 : 256;
  constexpr bool kTwice = ACT8 && GATED;
  const int used = std::min(x.pairs, x.experts), mean = x.pairs / used;
  auto slots = [&](int tile) { return used + x.pairs / tile; };
  auto tiles = [&](int tile) { return (int64_t)slots(tile) * ((p.out + kRows - 1) / kRows); };
  if constexpr (!kTwice) {
    if (mean > 128 && tiles(128) >= 256) {
      x.slots = slots(128);
      return launch_tile<ACT8, GATED, OUT, 4>(p, x, s);
    }
  }
  if (mean >= 3 && tiles(64) >= (mean < 40 ? 340 : kTwice ? 256 : 128)) {
    x.slots = slots(64);
    return launch_tile<ACT8, GATED, OUT, 2>(p, x, s);
  }
  x.slots = slots(32);
  return launch_split<ACT8, GATED, OUT, 2, 1>(p, x, s);
}

}  // namespace dqm

extern "C" {

dq_status dq_moe_workspace_bytes(int64_t tokens, int64_t K, int64_t inner, int64_t out,
                                 int64_t experts, int top_k, size_t* bytes) {
  using namespace dqm;
  if (!bytes || !moe_sizes(tokens, K, inner, out, experts, top_k)) return DQ_ERR_ARG;
  *bytes = MoeSpace(moe_chunk(tokens, K, inner, out, experts, top_k), inner, out, experts, top_k).bytes;
  return DQ_OK;
}

dq_status dq_moe_mx(const uint8_t* act_codes, const uint8_t* act_scales, dq_format act_fmt,
                    int64_t tokens, int64_t K, const int32_t* ids, const float* weights, int top_k,
                    int64_t experts, const uint8_t* gate_codes, const uint8_t* gate_scales,
                    const float* a_gate, const uint8_t* up_codes, const uint8_t* up_scales,
                    const float* a_up, dq_activation activation, int64_t inner,
                    const float* b_inner, dq_format inner_fmt, const uint8_t* down_codes,
                    const uint8_t* down_scales, const float* a_down, const void* residual,
                    int64_t out, dq_dtype yt, void* Y, void* workspace, size_t workspace_bytes,
                    hipStream_t stream) {
  using namespace dqm;
  if (inner_fmt != DQ_FMT_MXFP4 && inner_fmt != DQ_FMT_MXFP8) return DQ_ERR_UNSUPPORTED;
  if (yt != DQ_F32 && yt != DQ_BF16) return DQ_ERR_UNSUPPORTED;
  if (yt == DQ_F32 && (act_fmt == DQ_FMT_MXFP8 || inner_fmt == DQ_FMT_MXFP8)) return DQ_ERR_UNSUPPORTED;
  if (!moe_sizes(tokens, K, inner, out, experts, top_k)) return DQ_ERR_ARG;
  dq_status st = check_product(act_codes, act_scales, act_fmt, tokens, K, gate_codes, gate_scales,
                               a_gate, inner, activation);
  if (st == DQ_OK)
    st = check_product(act_codes, act_scales, act_fmt, tokens, K, up_codes, up_scales, a_up, inner,
                       activation);
  if (st == DQ_OK)
    st = check_product(act_codes, act_scales, act_fmt, tokens, inner, down_codes, down_scales, a_down,
                       out, activation);
  if (st != DQ_OK) return st;
  if (!ids || !weights || !Y || !workspace) return DQ_ERR_ARG;
  if (((uintptr_t)ids | (uintptr_t)weights) & 3u) return DQ_ERR_ARG;
  if (((uintptr_t)b_inner | (uintptr_t)Y | (uintptr_t)residual) & 15u) return DQ_ERR_ARG;
  if ((uintptr_t)workspace & 255u) return DQ_ERR_ARG;
  const int64_t chunk = moe_chunk(tokens, K, inner, out, experts, top_k);
  const MoeSpace space(chunk, inner, out, experts, top_k);
  if (workspace_bytes < space.bytes) return DQ_ERR_WORKSPACE;
  const int esz = yt == DQ_BF16 ? 2 : 4;
  const size_t wb = packed_bytes(experts * inner, K), db = packed_bytes(experts * out, inner);
  const size_t vb = (size_t)(experts * inner) * 4, yb = (size_t)tokens * (size_t)out * esz;
  if (dq::any_overlap({{Y, yb}, {workspace, space.bytes}},
                      {{residual == Y ? nullptr : residual, yb},
                       {act_codes, act_bytes(act_fmt, tokens, K)},
                       {act_scales, (size_t)(tokens * (K / 32))},
                       {ids, (size_t)tokens * top_k * 4},
                       {weights, (size_t)tokens * top_k * 4},
                       {gate_codes, wb},
                       {gate_scales, wb / 16},
                       {up_codes, wb},
                       {up_scales, wb / 16},
                       {down_codes, db},
                       {down_scales, db / 16},
                       {a_gate, vb},
                       {a_up, vb},
                       {b_inner, vb},
                       {a_down, (size_t)(experts * out) * 4}}))
    return DQ_ERR_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const bool act8 = act_fmt == DQ_FMT_MXFP8, mid8 = inner_fmt == DQ_FMT_MXFP8;
  for (int64_t t = 0; t < tokens; t += chunk) {
    const int n = (int)std::min(chunk, tokens - t), pairs = n * top_k;
    Experts x{};
    x.ids = ids + t * top_k;
    x.pairs = pairs;
    x.experts = (int)experts;
    if (pairs > kInlinePairs) {
      int *counts = reinterpret_cast<int*>(ws + space.counts),
          *order = reinterpret_cast<int*>(ws + space.order);
      hipLaunchKernelGGL(k_moe_plan, dim3((unsigned)experts), dim3(1024), 0, stream, x.ids, pairs,
                         (int)experts, counts, order);
      if (hipGetLastError() != hipSuccess) return DQ_ERR_HIP;
      x.counts = counts;
      x.order = order;
    }
    MlpArgs g{};
    g.xc = act_codes + t * (act8 ? K : K / 2);
    g.xs = act_scales + t * (K / 32);
    g.wc[0] = gate_codes;
    g.wc[1] = up_codes;
    g.ws[0] = gate_scales;
    g.ws[1] = up_scales;
    g.a[0] = a_gate;
    g.a[1] = a_up;
    g.b = b_inner;
    g.codes = ws + space.codes;
    g.scales = ws + space.scales;
    g.tokens = pairs;
    g.out = (int)inner;
    g.K = (int)K;
    g.act = activation;
    x.div = top_k;
    x.src_rows = (uint32_t)n;
    hipError_t e;
    if (act8) e = mid8 ? launch_experts<true, true, kOutFp8>(g, x, stream)
                       : launch_experts<true, true, kOutFp4>(g, x, stream);
    else e = mid8 ? launch_experts<false, true, kOutFp8>(g, x, stream)
                  : launch_experts<false, true, kOutFp4>(g, x, stream);
    if (e != hipSuccess) return DQ_ERR_HIP;
    MlpArgs d{};
    d.xc = g.codes;
    d.xs = g.scales;
    d.wc[0] = down_codes;
    d.ws[0] = down_scales;
    d.a[0] = a_down;
    d.y = ws + space.y;
    d.tokens = pairs;
    d.out = (int)out;
    d.K = (int)inner;
    d.act = DQ_ACTIVATION_NONE;
    x.div = 1;
    x.src_rows = (uint32_t)pairs;
    e = mid8 ? launch_experts<true, false, kOutF32>(d, x, stream)
             : launch_experts<false, false, kOutF32>(d, x, stream);
    if (e != hipSuccess) return DQ_ERR_HIP;
    SumArgs s{};
    s.y = static_cast<const float*>(d.y);
    s.ids = x.ids;
    s.weights = weights + t * top_k;
    s.res = residual ? static_cast<const char*>(residual) + t * out * esz : nullptr;
    s.Y = static_cast<char*>(Y) + t * out * esz;
    s.tokens = n;
    s.out = (int)out;
    s.top_k = top_k;
    s.experts = (int)experts;
    const dim3 grid((unsigned)(n * ((out + 1023) / 1024)));
    if (yt == DQ_BF16) hipLaunchKernelGGL(k_moe_sum<true>, grid, dim3(256), 0, stream, s);
    else hipLaunchKernelGGL(k_moe_sum<false>, grid, dim3(256), 0, stream, s);
    if (hipGetLastError() != hipSuccess) return DQ_ERR_HIP;
  }
  return DQ_OK;
}

}  // extern "C"
