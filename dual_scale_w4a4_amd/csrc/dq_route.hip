// dq_route.hip -- the router of a layer of experts: each token's scores of the experts, its top_k of
// them and their weights.
//
// Which experts a token takes must not depend on the order of a sum, so a logit is the fp64 sum of
// the exact products rounded once to fp32, and scores and selection keys are fp64.
//
// Two launches. The logits: for small products a wave takes one expert and up to 4 tokens, k over its
// lanes; for larger ones the fp64 matrix instruction takes tiles of 16 or 32 tokens by as many experts,
// k over the workgroup's waves. Then a wave per token selects.
//
// For large products of bf16 values the fp64 instruction is what bounds that (4096 tokens, 128 experts,
// K 4096: 82 us of 90, 52 TFLOP/s), so the first launch takes the bf16 instruction instead and gives each
// logit with a bound on its error, and the second computes in fp64 the few experts of each token
// that the bounds leave in question, the chosen ones among them: the same result. Where scores of other
// experts enter the result (the softmax's sum with a bias or without renormalization), or a value is
// not finite, that is every expert. That takes 18 + 27 us: the bf16 products wait for their operands'
// way through LDS; the selection's 8.1 experts a token (8 asked for) are 1.4 10^8 exact products at
// 4.4 vector instructions each, and about 14 us that do not depend on K. One token, 64 experts: 4.0 + 3.0
// us, latency.
#include <float.h>
#include <limits.h>

#include <algorithm>

#include "../../include/dq_layer.h"
#include "dq_mlp_kernels.h"

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

// Workgroup of 16 waves: 16 M tokens by 16 M experts, wave w taking channels 32 w .. of every 512 (the
// waves' partial sums joined in wave order; with 4 waves 640 tokens, 128 experts, K 4096 in fp32 take 55
// us, with 8 44, with 16 41). V_MFMA_F64_16X16X4: lane l holds row (column) l % 16, k l / 16; result v
// of lane l is D[4 v + l / 16][l % 16]. The order of k inside a sum is free, so lane quarter q takes
// channels 8 q .. 8 q + 7 of the 32, in 8 steps.
template <bool XB, bool WB, int M>
__global__ __launch_bounds__(1024) void k_logits_many(LogitArgs p) {
  constexpr int W = 16, T = 16 * M;
  __shared__ double part[W][M * M][4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int rl = lane & 15, q = lane >> 4;
  const int ne = (p.experts + T - 1) / T;
  const int e0 = (blockIdx.x % ne) * T;
  const int64_t t0 = (int64_t)(blockIdx.x / ne) * T;
  // rows past the end read the last one; their results are not stored
  int64_t xo[M], wo[M];
#pragma unroll
  for (int m = 0; m < M; m++) {
    xo[m] = min(t0 + 16 * m + rl, p.tokens - 1) * p.cols;
    wo[m] = (int64_t)min(e0 + 16 * m + rl, p.experts - 1) * p.cols;
  }
  f64x4 acc[M][M] = {};
  for (int c0 = wave * 32; c0 < p.cols; c0 += W * 32) {
    const int c = c0 + 8 * q;
    float x[M][8] = {}, w[M][8] = {};
    if (c < p.cols) {
#pragma unroll
      for (int m = 0; m < M; m++) {
        load8<XB>(p.X, xo[m] + c, x[m]);
        load8<WB>(p.W, wo[m] + c, w[m]);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; k++)
#pragma unroll
      for (int m = 0; m < M; m++)
#pragma unroll
        for (int n = 0; n < M; n++)
          acc[m][n] = __builtin_amdgcn_mfma_f64_16x16x4f64((double)x[m][k], (double)w[n][k],
                                                           acc[m][n], 0, 0, 0);
  }
#pragma unroll
  for (int m = 0; m < M; m++)
#pragma unroll
    for (int n = 0; n < M; n++)
#pragma unroll
      for (int v = 0; v < 4; v++) part[wave][M * m + n][v][lane] = acc[m][n][v];
  __syncthreads();
  for (int i = threadIdx.x; i < T * T; i += W * 64) {
    const int b = i >> 8, v = (i >> 6) & 3, l = i & 63;
    double s = 0.0;
    for (int w = 0; w < W; w++) s += part[w][b][v][l];
    const int64_t t = t0 + 16 * (b / M) + 4 * v + (l >> 4);
    const int e = e0 + 16 * (b % M) + (l & 15);
    if (t < p.tokens && e < p.experts) p.logits[t * p.experts + e] = (float)s;
  }
}

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

// Logits within a bound: {l, d} with |l - the exact sum| <= d. A workgroup takes 32 tokens and 64
// experts; its waves share the two blocks of 32 experts and, in periods of 64 k, the channels. Each
// runs by itself through two LDS stages of its own (rows of one cache line, pieces swizzled), as the
// adapters' rank kernel does. Products of bf16 values are exact in fp32; a period's 64 are added in
// fp32, with at most 64 roundings of 2^-23 of the sum of their magnitudes, which a second product of
// the magnitudes gives; the periods' sums are added in fp64.
constexpr int kFastWaves = 8, kFastCols = 1 << 16;

struct FastArgs {
  const uint16_t* X;
  const uint16_t* W;
  float* out;        // tokens x experts x 2
  int64_t tokens;
  int cols, experts;
};

__global__ __launch_bounds__(kFastWaves * 64) void k_logits_fast(FastArgs p) {
  using namespace dqm;
  constexpr int kTile = 32 * kRowB, kRing = 4 * kTile, kShare = kFastWaves / 2;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kFastWaves * kRing];
  const int lane = threadIdx.x & 63, rl = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ne = (p.experts + 63) / 64;
  const int e0 = (blockIdx.x % ne) * 64 + (wave & 1) * 32;
  const int64_t t0 = (int64_t)(blockIdx.x / ne) * 32;
  const uint32_t pitch = (uint32_t)p.cols * 2u;
  // rows past the end read zeros
  const int nt = (int)min((int64_t)32, p.tokens - t0), nx = max(min(32, p.experts - e0), 0);
  const __amdgpu_buffer_rsrc_t rx = rsrc(p.X + t0 * p.cols, (uint32_t)nt * pitch);
  const __amdgpu_buffer_rsrc_t rw = rsrc(p.W + (int64_t)(nx ? e0 : 0) * p.cols, (uint32_t)nx * pitch);
  const __amdgpu_buffer_rsrc_t rnone = rsrc(p.X, 0u);
  const int periods = (p.cols + 63) / 64, first = wave >> 1;
  uint32_t vo[4], vend[4];  // vend: in the last period, whose pieces past the row's end read zeros
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const int r = 8 * j + (lane >> 3), piece = (lane & 7) ^ (r & 7) ^ ((r >> 3) & 1);
    vo[j] = (uint32_t)r * pitch + (uint32_t)(piece * 16);
    vend[j] = (periods - 1) * 64 + piece * 8 < p.cols ? vo[j] : kOob;
  }
  uint8_t* ring = lds + wave * kRing;
  const int xt = (rl & 7) ^ ((rl >> 3) & 1);
  double sum[16] = {};
  v16f size = {};
  auto load = [&](int c, int st) {  // past the last period nothing is read
    const bool on = c < periods, end = c == periods - 1;
    uint8_t* dst = ring + st * (2 * kTile);
#pragma unroll
    for (int j = 0; j < 4; j++)
      load_lds(on ? rx : rnone, dst + j * 1024, end ? vend[j] : vo[j], c * kRowB);
#pragma unroll
    for (int j = 0; j < 4; j++)
      load_lds(on ? rw : rnone, dst + kTile + j * 1024, end ? vend[j] : vo[j], c * kRowB);
  };
  auto stage = [&](int c, int st) {
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(8));
    wave_lds_order();
    const uint8_t* src = ring + st * (2 * kTile) + rl * kRowB;
    u32x4 x[4], w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int at = ((2 * i + h) ^ xt) * 16;
      x[i] = *reinterpret_cast<const u32x4*>(src + at);
      w[i] = *reinterpret_cast<const u32x4*>(src + kTile + at);
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): read before the stage is loaded again
    wave_lds_order();
    load(c + 2 * kShare, st);
    v16f acc = {};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x[i]),
                                                    __builtin_bit_cast(bf16x8, w[i]), acc, 0, 0, 0);
      const u32x4 ax = x[i] & 0x7FFF7FFFu, aw = w[i] & 0x7FFF7FFFu;
      size = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, ax),
                                                     __builtin_bit_cast(bf16x8, aw), size, 0, 0, 0);
    }
#pragma unroll
    for (int v = 0; v < 16; v++) sum[v] += (double)acc[v];
  };
  load(first, 0);
  load(first + kShare, 1);
  for (int c = first; c < periods; c += 2 * kShare) {
    stage(c, 0);
    stage(c + kShare, 1);  // zeros past the last
  }
  // the last loads read nothing but still write zeros into LDS: drain them before the join
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
  __syncthreads();
  // join: value v of a lane is token 8 (v / 4) + 4 h + v % 4, expert lane % 32
  double* part = reinterpret_cast<double*>(lds);                            // [wave][v][lane]
  float* part2 = reinterpret_cast<float*>(lds + kFastWaves * 16 * 64 * 8);  // likewise
  static_assert(kFastWaves * 16 * 64 * 12 <= kFastWaves * kRing, "the join's LDS");
#pragma unroll
  for (int v = 0; v < 16; v++) {
    part[(wave * 16 + v) * 64 + lane] = sum[v];
    part2[(wave * 16 + v) * 64 + lane] = size[v];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * 16 * 64; i += kFastWaves * 64) {
    const int b = i >> 10, v = (i >> 6) & 15, l = i & 63;
    double s = 0.0;
    float m = 0.0f;
#pragma unroll
    for (int w = 0; w < kShare; w++) {
      s += part[((2 * w + b) * 16 + v) * 64 + l];
      m += part2[((2 * w + b) * 16 + v) * 64 + l];
    }
    const int64_t t = t0 + 8 * (v / 4) + 4 * (l >> 5) + v % 4;
    const int e = (blockIdx.x % ne) * 64 + b * 32 + (l & 31);
    if (t < p.tokens && e < p.experts) {
      // the magnitudes' sum is itself off by up to cols / 2^23 of it, at most 1 / 128; the logit is
      // rounded here and once more to compare; products below fp32's range may be lost. Without any
      // magnitude it stands as 0: products below 2^-126 add up to 2^-110 at most, and where all of a
      // token's experts are such their scores are equal in fp64 either way.
      float2 o;
      o.x = (float)s;
      o.y = m == 0.0f ? 0.0f : m * (1.02f / (1 << 17)) + fabsf(o.x) * 0x1p-22f + 0x1p-100f;
      *reinterpret_cast<float2*>(p.out + (t * p.experts + e) * 2) = o;
    }
  }
}

struct SelectArgs {
  const float* logits; // tokens x experts, or tokens x experts x {logit, bound}
  const float* bias;   // experts, or null
  int* ids;
  float* weights;
  int64_t tokens;
  int experts, top_k, renormalize;
  float scale;
  const uint16_t* X;   // with bounds: bf16 tokens x cols
  const uint16_t* W;   // and experts x cols
  int cols;
};

// v of a lane that is the same for the whole wave
__device__ __forceinline__ double of_lane(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return dq::u2d((uint64_t)(uint32_t)__builtin_amdgcn_readlane((uint32_t)(u >> 32), lane) << 32 |
                 (uint32_t)__builtin_amdgcn_readlane((uint32_t)u, lane));
}

// the largest of the wave's values, none of them NaN
__device__ __forceinline__ double wave_max(double v) {
  v = fmax(v, dq::dpp_f64<dq::kDppQuadXor1>(v));
  v = fmax(v, dq::dpp_f64<dq::kDppQuadXor2>(v));
  v = fmax(v, dq::dpp_f64<dq::kDppRowHalfMirror>(v));
  v = fmax(v, dq::dpp_f64<dq::kDppRowMirror>(v));
  return fmax(fmax(of_lane(v, 0), of_lane(v, 16)), fmax(of_lane(v, 32), of_lane(v, 48)));
}

__device__ __forceinline__ double wave_add(double v) {
  v = dq::sum16_dpp(v);
  return ((of_lane(v, 0) + of_lane(v, 16)) + of_lane(v, 32)) + of_lane(v, 48);
}

// The next of the largest keys among those still free, ties to the lowest index: its index, no longer
// free.
template <int N>
__device__ __forceinline__ int take_largest(const double (&key)[N], bool (&is_free)[N], double& best) {
  const int lane = threadIdx.x & 63;
  double mine = -INFINITY;
#pragma unroll
  for (int n = 0; n < N; n++)
    if (is_free[n]) mine = fmax(mine, key[n]);
  best = wave_max(mine);
  int at = -1;
#pragma unroll
  for (int n = 0; n < N; n++) {
    const uint64_t m = __ballot(is_free[n] && key[n] == best);
    if (at < 0 && m) {
      at = n * 64 + __builtin_ctzll(m);
      if (lane == (at & 63)) is_free[n] = false;
    }
  }
  return at;
}

__device__ __forceinline__ double sigmoid64(double l) { return 1.0 / (1.0 + exp(-l)); }

// The k-th of two bf16 values in a word, finite, times 2^-896 as fp64: its exponent field is taken as
// fp64's (a subnormal one's too), by a shift that leaves copies of the sign to be masked out. Two or
// three instructions, where a conversion takes the time of four.
constexpr int kShift = 896;
__device__ __forceinline__ double shifted(uint32_t r, int k) {
  const uint32_t u = (uint32_t)((int32_t)(k ? r : r << 16) >> 3) & 0x8FFFE000u;
  return dq::u2d((unsigned long long)u << 32);
}

constexpr int kDppRowRor4 = 0x124, kDppRowRor8 = 0x128;  // lane i from i - 4, i - 8 within each 16 lanes

// The sum over the wave of one of eight values a lane: v[l % 8] in lane l. Halves of the values are
// exchanged with lane l ^ 1 and l ^ 2, and a lane four away takes the other half (3/4 fewer steps than a
// sum for each).
__device__ __forceinline__ double wave_add8(const double (&v)[8]) {
  const int lane = threadIdx.x & 63;
  double a[4], b[2];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const double keep = lane & 1 ? v[2 * i + 1] : v[2 * i], send = lane & 1 ? v[2 * i] : v[2 * i + 1];
    a[i] = keep + dq::dpp_f64<dq::kDppQuadXor1>(send);
  }
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const double keep = lane & 2 ? a[2 * i + 1] : a[2 * i], send = lane & 2 ? a[2 * i] : a[2 * i + 1];
    b[i] = keep + dq::dpp_f64<dq::kDppQuadXor2>(send);
  }
  const double keep = lane & 4 ? b[1] : b[0], send = lane & 4 ? b[0] : b[1];
  double s = keep + dq::dpp_f64<kDppRowRor4>(send);
  s += dq::dpp_f64<kDppRowRor8>(s);
  s += __shfl_xor(s, 16, 64);
  return s + __shfl_xor(s, 32, 64);
}

// fp64 dot products of a token's row with G experts' rows: with 8 that of e[l % 8] in lane l, with
// fewer the sums in v of every lane. FINITE: all values are. U 512-channel pieces of all rows are
// loaded at once.
template <int G, int U, bool FINITE>
__device__ __forceinline__ double dots(const SelectArgs& p, const uint16_t* x, const int (&e)[G],
                                       double (&s)[G]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int g = 0; g < G; g++) s[g] = 0.0;
  for (int c0 = lane * 8; c0 < p.cols; c0 += 512 * U) {
    u32x4 xr[U], wr[U][G];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int c = c0 + 512 * u;
      const bool in = c < p.cols;
      xr[u] = in ? *reinterpret_cast<const u32x4*>(x + c) : u32x4{};
#pragma unroll
      for (int g = 0; g < G; g++)
        wr[u][g] = in ? *reinterpret_cast<const u32x4*>(p.W + (int64_t)e[g] * p.cols + c) : u32x4{};
    }
    __builtin_amdgcn_sched_barrier(0);  // all of them in flight
    auto value = [](const u32x4& r, int k) { return u2f(k & 1 ? r[k / 2] & 0xFFFF0000u : r[k / 2] << 16); };
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int k = 0; k < 8; k++) {
        const double xv = FINITE ? shifted(xr[u][k / 2], k & 1) * 0x1p896 : (double)value(xr[u], k);
#pragma unroll
        for (int g = 0; g < G; g++)
          s[g] = fma(xv, FINITE ? shifted(wr[u][g][k / 2], k & 1) : (double)value(wr[u][g], k), s[g]);
      }
  }
  if constexpr (G == 8) {
    const double v = wave_add8(s);
    return FINITE ? ldexp(v, kShift) : v;
  } else {
#pragma unroll
    for (int g = 0; g < G; g++) {
      s[g] = wave_add(s[g]);
      if (FINITE) s[g] = ldexp(s[g], kShift);
    }
    return 0.0;
  }
}

// The bits of v in an order of unsigned numbers; a NaN is the largest
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = dq::f2u(v);
  return v == v ? u ^ (u >> 31 ? 0xFFFFFFFFu : 0x80000000u) : 0xFFFFFFFFu;
}
__device__ __forceinline__ float of_order(uint32_t u) {
  return u2f(u ^ (u >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}

// The token's experts that can be among the top_k (or more), in ascending order, the j-th in slot j / 64
// of lane j % 64: their exact logits and numbers; returns how many.
//
// Keys grow with the logits, so an expert whose key at its upper bound lies below the top_k-th
// largest of the keys at the lower bounds cannot. The keys of the bounds are fp32, widened by more
// than fp32's roundings and exp's last bits (where fp64 keys can tie): a logit's bound holds
// 2^-22 of it for three roundings of 2^-24, a score is off by less than 5 10^-7 of itself. A bound
// that is no number leaves its expert in question.
// WPT waves share the token's sums and hand them on in LDS.
template <bool SIGMOID, int N, int WPT>
__device__ __forceinline__ int recheck(const SelectArgs& p, int64_t t, double (&l)[N], int (&id)[N]) {
  constexpr int G = WPT == 1 ? 8 : 2;
  __shared__ float exact[WPT == 1 ? 1 : 64 * N];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t lo[N], hi[N];
  bool wild = false, zeros = true;
  float top = -INFINITY;
#pragma unroll
  for (int n = 0; n < N; n++) {
    const int e = n * 64 + lane;
    lo[n] = hi[n] = 0u;
    id[n] = 0;
    l[n] = -INFINITY;
    if (e < p.experts) {
      const float2 v = *reinterpret_cast<const float2*>(p.logits + (t * p.experts + e) * 2);
      float from = v.x - v.y, to = v.x + v.y, slack = 1e-7f;
      top = fmaxf(top, to);
      wild |= !(fabsf(v.x) + v.y < 1e38f);
      zeros &= v.y == 0.0f;
      if (SIGMOID) {
        const float b = p.bias ? p.bias[e] : 0.0f;
        from = __builtin_amdgcn_rcpf(1.0f + expf(-from));
        to = __builtin_amdgcn_rcpf(1.0f + expf(-to));
        slack = 1e-6f * (to + fabsf(b)) + 1e-37f;
        from += b;
        to += b;
      }
      from -= slack;
      lo[n] = from == from ? ordered(from) : 0u;
      hi[n] = ordered(to + slack);
    }
  }
  // A token of zeros (a batch's padding): without a bias every expert is in question, and every logit is
  // known. 4096 tokens, 128 experts, K 4096: 26 us where all are such, 35 with half of them, 46 with none
  // (summing their experts again 297 and 189, more than the 85 of the fp64 instruction).
  if (__all(zeros)) {
#pragma unroll
    for (int n = 0; n < N; n++)
      if (n * 64 + lane < p.experts) {
        id[n] = n * 64 + lane;
        l[n] = 0.0;
      }
    return p.experts;
  }
  // the top_k-th largest of lo, bit by bit until the top_k are apart, then the least of them
  uint32_t kth = 0u;
  for (uint32_t bit = 0x80000000u; bit; bit >>= 1) {
    int above = 0;
#pragma unroll
    for (int n = 0; n < N; n++) above += __popcll(__ballot(lo[n] >= (kth | bit)));
    if (above >= p.top_k) kth |= bit;
    if (above == p.top_k) break;
  }
  uint32_t least = 0xFFFFFFFFu;
#pragma unroll
  for (int n = 0; n < N; n++)
    if (lo[n] >= kth) least = min(least, lo[n]);
  least = min(least, dq::dpp_u32<dq::kDppQuadXor1>(least));
  least = min(least, dq::dpp_u32<dq::kDppQuadXor2>(least));
  least = min(least, dq::dpp_u32<dq::kDppRowHalfMirror>(least));
  least = min(least, dq::dpp_u32<dq::kDppRowMirror>(least));
  auto row = [&](int i) { return (uint32_t)__builtin_amdgcn_readlane(least, 16 * i); };
  kth = min(min(row(0), row(1)), min(row(2), row(3)));
  const bool finite = !__any(wild);
  // softmax scores that underflow are equal, and one logit that is not finite is in every score
  if (!SIGMOID && (!finite || __any(!(top - 700.0f < of_order(kth))))) kth = 0u;
  // their sums in fp64, G experts at a time and the last ones singly; a logit's magnitude and bound
  // are not finite where one of its values is not
  const uint16_t* x = p.X + t * p.cols;
  uint64_t m[N];
  int count = 0;
#pragma unroll
  for (int n = 0; n < N; n++) {
    m[n] = __ballot(n * 64 + lane < p.experts && hi[n] >= kth);
    count += __popcll(m[n]);
  }
  auto next = [&] {
    int e = -1;
#pragma unroll
    for (int n = 0; n < N; n++)
      if (e < 0 && m[n]) {
        e = n * 64 + __builtin_ctzll(m[n]);
        m[n] &= m[n] - 1;
      }
    return e;
  };
  for (int j = 0, q = 0; j < count; q++) {
    const bool mine = WPT == 1 || q % WPT == wave;
    const int width = finite && count - j >= G ? G : 1;
    auto set = [&](int at, int e, double sum, bool here) {
      if (WPT > 1 && lane == 0 && here) exact[at] = (float)sum;
#pragma unroll
      for (int n = 0; n < N; n++)
        if (n == at >> 6 && lane == (at & 63)) {
          id[n] = e;
          if (WPT == 1) l[n] = (double)(float)sum;
        }
    };
    if (width == G) {
      int e[G];
      double v[G];
#pragma unroll
      for (int g = 0; g < G; g++) e[g] = next();
      double sum = 0.0;
      if (mine) sum = dots<G, G == 8 ? 2 : 4, true>(p, x, e, v);
#pragma unroll
      for (int g = 0; g < G; g++) set(j + g, e[g], G == 8 ? sum : v[g], mine);
    } else {
      const int e[1] = {next()};
      double v[1];
      if (mine) {
        if (finite) dots<1, 8, true>(p, x, e, v);
        else dots<1, 1, false>(p, x, e, v);
      }
      set(j, e[0], v[0], mine);
    }
    j += width;
  }
  if (WPT > 1) {
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; n++)
      if (n * 64 + lane < count) l[n] = (double)exact[n * 64 + lane];
  }
  return count;
}

// The token's top_k of the experts that the wave holds (in ascending order, slot after slot) and their
// weights. NaN keys rank as -inf. RANKED: `count` experts, one a lane, each of which counts those before
// it; else the largest is taken top_k times.
template <bool SIGMOID, int N, bool RANKED>
__device__ __forceinline__ void finish(const SelectArgs& p, int64_t t, double (&score)[N],
                                       const int (&id)[N], bool (&is_free)[N], int count) {
  const int lane = threadIdx.x & 63;
  double key[N];
  if (SIGMOID) {
#pragma unroll
    for (int n = 0; n < N; n++) score[n] = sigmoid64(score[n]);
  } else {
    double top = -INFINITY;
#pragma unroll
    for (int n = 0; n < N; n++) top = fmax(top, score[n]);
    top = wave_max(top);
    double sum = 0.0;
#pragma unroll
    for (int n = 0; n < N; n++) {
      score[n] = is_free[n] ? exp(score[n] - top) : 0.0;
      sum += score[n];
    }
    const double total = wave_add(sum);
#pragma unroll
    for (int n = 0; n < N; n++) score[n] = score[n] / total;
  }
#pragma unroll
  for (int n = 0; n < N; n++) {
    key[n] = score[n] + (p.bias && is_free[n] ? (double)p.bias[id[n]] : 0.0);
    if (!(key[n] == key[n])) key[n] = -INFINITY;
  }
  double chosen = 0.0, mine = 0.0;  // the sum of the chosen scores
  int place = kMaxExperts, expert = 0;
  if constexpr (RANKED) {
    int rank = 0;
    for (int j = 0; j < count; j++) {
      const double other = of_lane(key[0], j);
      rank += other > key[0] || (other == key[0] && j < lane);
    }
    for (int k = 0; k < p.top_k; k++)
      chosen += of_lane(score[0], __builtin_ctzll(__ballot(lane < count && rank == k)));
    if (lane < count) place = rank;
    mine = score[0];
    expert = id[0];
  } else {
    for (int k = 0; k < p.top_k; k++) {  // the k-th goes to lane k
      double best;
      const int at = __builtin_amdgcn_readfirstlane(take_largest<N>(key, is_free, best));
      double s = 0.0;
      int e = 0;
#pragma unroll
      for (int n = 0; n < N; n++)
        if (n == at >> 6) {
          s = score[n];
          e = id[n];
        }
      s = of_lane(s, at & 63);
      e = __builtin_amdgcn_readlane(e, at & 63);
      chosen += s;
      if (lane == k) {
        place = k;
        mine = s;
        expert = e;
      }
    }
  }
  if (place < p.top_k) {
    double w = mine;
    if (p.renormalize) w = chosen == 0.0 ? 0.0 : mine / chosen;
    p.ids[t * p.top_k + place] = expert;
    p.weights[t * p.top_k + place] = (float)(w * (double)p.scale);
  }
}

// Wave: one token; lane l holds experts l, l + 64, ... N of them. BOUNDS: the logits come with bounds;
// only the experts in question are held, and the softmax's sum cancels in the weights.
template <bool SIGMOID, int N, bool BOUNDS, int WPT = 1>
__global__ __launch_bounds__(256) void k_select(SelectArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t t = WPT == 4 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= p.tokens) return;
  double score[N];
  int id[N];
  bool is_free[N];
  int count = p.experts;
  if (BOUNDS) count = recheck<SIGMOID, N, WPT>(p, t, score, id);
  if (WPT > 1 && threadIdx.x >= 64) return;
#pragma unroll
  for (int n = 0; n < N; n++) {
    is_free[n] = n * 64 + lane < count;
    if (!BOUNDS) {
      id[n] = n * 64 + lane;
      score[n] = is_free[n] ? (double)p.logits[t * p.experts + id[n]] : -INFINITY;
    }
  }
  if (BOUNDS && count <= 64) {
    double s[1] = {score[0]};
    const int i[1] = {id[0]};
    bool f[1] = {is_free[0]};
    finish<SIGMOID, 1, true>(p, t, s, i, f, count);
  } else {
    finish<SIGMOID, N, false>(p, t, score, id, is_free, count);
  }
}

// ---------------------------------------------------------------------------------- host

constexpr int kMaxTopK = 32;

// Which kernels; logits + selection measured, us, 8 experts, sigmoid:
//   experts, K     tokens   a wave an    fp64 instruction,    .. of 32   bounds, and the sums
//                           expert       tiles of 16                     in question (bf16)
//   128, 4096      96       15 + 5       17 + 5                          14 + 8
//                  192      21 + 5       18 + 5                          14 + 9
//                  512      46 + 5       18 + 5                          14 + 11
//                  640      57 + 5       32 + 5               41 + 5     14 + 12
//                  1024                  32 + 6               41 + 6     14 + 15
//                  1500                  45 + 6               41 + 6
//                  4096                  118 + 8              82 + 8     18 + 27
//   64, 2048       256      10 + 4       11 + 4                          9 + 6
//                  512      16 + 4       11 + 4                          9 + 7
//                  1300                  17 + 4               22 + 4     10 + 11
//                  4096                  31 + 6               22 + 6     10 + 18
//   256, 7168      64       23 + 8       27 + 8                          21 + 12
//                  128      45 + 8       28 + 8                          21 + 12
//                  256                   28 + 8                          21 + 15
//                  320                   52 + 8               70 + 8
//   128, 1024      160      8 + 5        6 + 5
//                  4096                                       20 + 8     9 + 15
// So by tokens x experts, nearly whatever K: the fp64 instruction from 5 2^12 on, in tiles of 16 as long
// as those of 32 are at most 160. Bounds, where they can be had, above 2^16 (more tiles of 16 than CUs)
// and from 2^28 products on.
// Whether they can: bf16 values, and a result that only the chosen experts' scores enter.
bool with_bounds(dq_dtype xt, dq_dtype wt, int64_t tokens, int64_t cols, int64_t experts,
                 const float* bias, dq_score score, int renormalize) {
  return xt == DQ_BF16 && wt == DQ_BF16 && cols <= kFastCols &&
         (score == DQ_SCORE_SIGMOID || (renormalize && !bias)) &&
         tokens * experts > (1 << 16) && tokens * experts * cols >= (1 << 28);
}

template <bool XB, bool WB>
hipError_t launch_logits(const LogitArgs& p, hipStream_t s) {
  if (p.tokens * p.experts < 5 << 12) {
    const int64_t ne = (p.experts + 3) / 4;
    if (p.tokens == 1)
      hipLaunchKernelGGL((k_logits_few<XB, WB, 1>), dim3((unsigned)ne), dim3(256), 0, s, p);
    else
      hipLaunchKernelGGL((k_logits_few<XB, WB, 4>), dim3((unsigned)(ne * ((p.tokens + 3) / 4))),
                         dim3(256), 0, s, p);
  } else {
    auto tiles = [&](int t) { return ((p.experts + t - 1) / t) * ((p.tokens + t - 1) / t); };
    if (tiles(32) <= 160)
      hipLaunchKernelGGL((k_logits_many<XB, WB, 1>), dim3((unsigned)tiles(16)), dim3(1024), 0, s, p);
    else
      hipLaunchKernelGGL((k_logits_many<XB, WB, 2>), dim3((unsigned)tiles(32)), dim3(1024), 0, s, p);
  }
  return hipGetLastError();
}

hipError_t launch_logits_fast(const LogitArgs& l, hipStream_t s) {
  FastArgs p{};
  p.X = static_cast<const uint16_t*>(l.X);
  p.W = static_cast<const uint16_t*>(l.W);
  p.out = l.logits;
  p.tokens = l.tokens;
  p.cols = l.cols;
  p.experts = l.experts;
  const int64_t n = (int64_t)((p.experts + 63) / 64) * ((p.tokens + 31) / 32);
  hipLaunchKernelGGL(k_logits_fast, dim3((unsigned)n), dim3(kFastWaves * 64), 0, s, p);
  return hipGetLastError();
}

template <bool SIGMOID, int N>
hipError_t launch_select_n(const SelectArgs& p, bool bounds, hipStream_t s) {
  const dim3 grid((unsigned)((p.tokens + 3) / 4)), block(256);
  // up to 1024 tokens, so above 64 experts: fewer waves than the chip holds; four share a token's sums
  constexpr int kShare = N > 1 ? 4 : 1;
  if (!bounds)
    hipLaunchKernelGGL((k_select<SIGMOID, N, false>), grid, block, 0, s, p);
  else if (kShare > 1 && p.tokens <= 1024)
    hipLaunchKernelGGL((k_select<SIGMOID, N, true, kShare>), dim3((unsigned)p.tokens), block, 0, s, p);
  else
    hipLaunchKernelGGL((k_select<SIGMOID, N, true>), grid, block, 0, s, p);
  return hipGetLastError();
}

template <bool SIGMOID>
hipError_t launch_select(const SelectArgs& p, bool bounds, hipStream_t s) {
  if (p.experts <= 64) return launch_select_n<SIGMOID, 1>(p, bounds, s);
  if (p.experts <= 128) return launch_select_n<SIGMOID, 2>(p, bounds, s);
  if (p.experts <= 256) return launch_select_n<SIGMOID, 4>(p, bounds, s);
  return launch_select_n<SIGMOID, 16>(p, bounds, s);
}

}  // namespace dqr

extern "C" {

dq_status dq_moe_route_workspace_bytes(int64_t tokens, int64_t experts, size_t* bytes) {
  using namespace dqr;
  if (!bytes || tokens < 1 || tokens > INT32_MAX - 256 || experts < 1 || experts > kMaxExperts)
    return DQ_ERR_ARG;
  *bytes = ((size_t)tokens * (size_t)experts * 8 + 255) / 256 * 256;
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
  const int64_t chunk = 1 << 20;
  const bool bounds = with_bounds(xt, wt, tokens, cols, experts, bias, score, renormalize);
  for (int64_t t = 0; t < tokens; t += chunk) {
    LogitArgs l{};
    l.X = static_cast<const char*>(X) + t * cols * (xt == DQ_BF16 ? 2 : 4);
    l.W = W;
    l.logits = static_cast<float*>(workspace) + t * experts * 2;
    l.tokens = std::min(chunk, tokens - t);
    l.cols = (int)cols;
    l.experts = (int)experts;
    hipError_t e;
    if (bounds) e = launch_logits_fast(l, stream);
    else if (xt == DQ_BF16) e = wt == DQ_BF16 ? launch_logits<true, true>(l, stream)
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
    s.X = static_cast<const uint16_t*>(l.X);
    s.W = static_cast<const uint16_t*>(W);
    s.cols = l.cols;
    e = score == DQ_SCORE_SIGMOID ? launch_select<true>(s, bounds, stream)
                                  : launch_select<false>(s, bounds, stream);
    if (e != hipSuccess) return DQ_ERR_HIP;
  }
  return DQ_OK;
}

}  // extern "C"
