// dq_block_norm.hip -- the norm after a block, the block's gate, the scaled residual, the norm
// before the next block, column scales and the group quantizer in one kernel.
//
//   m = fl(fl(X r1) post) (or X),  m = fl(fl(m gate_j) tgate_t)
//   h = round_xt(fl(fl(rs R) + m)) (stored),  n = fl(fl(h r2) w) (stored as x_out where asked for)
//   x = fl(n b), then Q in groups of G channels.
//
// As for the single norm (dq_norm.hip) codes have to be the definition's bit for bit: one fp32
// rounding per step, sums of squares and roots in fp64.
//
// Memory bounds it: every array moves once, and the rest is kept below that (exact bf16 squares in
// fp32, roots by Newton steps, packed stores: with fp64 conversions, square roots and quotients
// 8192 x 4096 took 66 us). 8192 x 4096 bf16 with post norm, gate and x_out to MXFP8: 54 - 56 us for
// 303 MB, 5.4 - 5.5 TB/s. 1003 x 8160 fp32 with a token gate to MXFP8: 22 us for 107 MB, 4.8 TB/s. One
// token of 4096: 4.2 us. The other formats at 8192 x 4096 in bf16: MXFP4 52 us, MXINT4 53, INT4 56, NVFP4
// 81, whose quantizer does not fit the registers (13 spilled; in fp32 71, and 155 us against 117).
// 8192 rows of other widths, as the first, TB/s in bf16 and fp32: 1024 channels 2.8 and 4.2, 2048 4.3 and
// 5.4, 2880 5.0 and 4.3, 5120 4.5 and 4.6, 8192 5.3 and 5.1, 12288 5.3 and 5.3: where a workgroup has fewer
// waves than its LDS is laid out for, fewer loads are in flight (below).
#include <limits.h>

#include "../../include/dq_layer.h"
#include "dq_norm_device.h"

namespace dq {

struct BlockNormArgs {
  const void* X;
  const void* R;        // or null
  void* h;
  const void* post;     // channels, or null
  const float* gate;    // channels, or null
  const float* tgate;   // tokens, or null
  const void* w;        // channels, or null
  const float* b;       // channels, or null
  void* xo;             // n, or null
  int64_t m, n;
  double post_eps, eps;
  float rs;
  float g;              // NVFP4
  uint8_t* codes;
  void* scales;
  int* status;
  bool norm1;           // whether the block's output is normed
  bool wbf, xobf;       // post and w, xo are bf16
};

// a vector of 16 channels, ones where there is none (a product with 1 is exact)
__device__ __forceinline__ void load_ones(const void* p, bool bf, int64_t c, float (&v)[kNormEpl]) {
#pragma unroll
  for (int k = 0; k < kNormEpl; k++) v[k] = 1.0f;
  if (p) {
    if (bf) load16<true>(p, c, v);
    else load16<false>(p, c, v);
  }
}

// v rounded to bf16 (or as it is), stored
template <bool BF>
__device__ __forceinline__ void store_rounded(float (&v)[kNormEpl], void* p, int64_t off, bool act) {
  if (BF) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    Raw16<true> o;
#pragma unroll
    for (int k = 0; k < kNormEpl / 2; k++)
      o.v[k / 4][k % 4] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)v[2 * k], (__bf16)v[2 * k + 1]});
    if (act)
#pragma unroll
      for (int k = 0; k < 2; k++) reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + off)[k] = o.v[k];
    o.unpack(v);
  } else if (act) {
    store16<false>(p, off, v);
  }
}

// fl32(1 / sqrt(sum / n + eps)): the hardware's approximation (measured 2^-24.2) and two Newton steps
// in fp64 (2^-47.7 after one; the second costs nothing that shows), fewer instructions than a square
// root and a quotient
__device__ __forceinline__ float rstd_of(double sum, double rn, double eps) {
  const double v = fma(sum, rn, eps), y = __builtin_amdgcn_rsq(v);
  const double e = fma(-v * y, y, 1.0), z = fma(0.5 * e, y, y);
  return (float)fma(0.5 * fma(-v * z, z, 1.0), z, z);
}

// The largest |v| of 16 values as bits: above every finite value's for an infinity or a NaN
__device__ __forceinline__ uint32_t top_bits(const float (&v)[kNormEpl]) {
  uint32_t m = 0u;
#pragma unroll
  for (int k = 0; k < kNormEpl; k++) m = max(m, f2u(v[k]) & 0x7FFFFFFFu);
  return m;
}
constexpr uint32_t kInfBits = 0x7F800000u;

// Sum of squares of 16 values, exact but for the additions. bf16 values are squared in fp32 where that
// is exact (16 bits) and become fp64 values times 2^-896 by a shift of their bits: three instructions
// each, where the conversion alone costs four times one. A square below fp32's normal range keeps a
// multiple of 2^-146; with a largest value above 2^-44 fifteen of them lose less than 2^-54 of its square,
// an addition's rounding.
template <bool BF>
__device__ __forceinline__ double squares16(const float (&h)[kNormEpl], uint32_t top) {
  if (BF && top < 0x5F000000u && (top > 0x29800000u || top == 0u)) {  // 2^-44 .. 2^63, or all zero
    double s[2] = {};
#pragma unroll
    for (int k = 0; k < kNormEpl; k++)
      s[k & 1] += u2d((unsigned long long)(f2u(h[k] * h[k]) >> 3) << 32);
    return (s[0] + s[1]) * 0x1p896;
  }
  return sum_squares(h);
}

// h = rs R + m of 16 channels, rounded to the stream's type and stored
template <bool BF>
__device__ __forceinline__ void join16(float (&m)[kNormEpl], const float (&r)[kNormEpl], float rs,
                                       void* p, int64_t off, bool act) {
#pragma unroll
  for (int k = 0; k < kNormEpl; k++) m[k] = r[k] * rs + m[k];
  store_rounded<BF>(m, p, off, act);
}

// n = h r2 w; stores n rounded to x_out's type and returns whether a stored value is not finite
__device__ __forceinline__ bool norm16(float (&h)[kNormEpl], float r2, const float (&w)[kNormEpl],
                                       const BlockNormArgs& p, int64_t off, bool act) {
#pragma unroll
  for (int k = 0; k < kNormEpl; k++) h[k] = h[k] * r2 * w[k];
  if (!p.xo) return false;
  float v[kNormEpl];
#pragma unroll
  for (int k = 0; k < kNormEpl; k++) v[k] = h[k];
  if (p.xobf) store_rounded<true>(v, p.xo, off, act);
  else store_rounded<false>(v, p.xo, off, act);
  return act && top_bits(v) >= kInfBits;
}

// A workgroup of up to NW waves has a thread per 16 channels and takes row after row, each array
// read and written once: X of the next row is loaded before the first of the row's two sums, its
// residual before the second. post and w stay in registers. gate and b lie in LDS, 16 values that
// each thread writes and reads alone: with all four in registers 128 of them do not suffice (100
// spilled), and sixteen waves a CU, which 128 registers allow, cover the loads best. That LDS is laid
// out for NW waves whatever the workgroup has, and there without gate and b too: four workgroups of up to
// 4 waves fit a CU, two of up to 8 and one of up to 16, so that rows up to 1024 channels have 4 waves a CU,
// up to 2048 8 and those of 5 waves (up to 5120) 10.
template <int FMT, int G, bool BF, int NW>
__global__ __launch_bounds__(NW * kWave, 4) void k_block_norm(BlockNormArgs p) {
  __shared__ double red[2][NW];
  __shared__ u32x4 own[2][4][NW * kWave];  // gate, b
  // Lanes past the row's end hold zeros: they load nothing (where h replaces X or R another wave
  // may have stored already what they would read), and they store and report nothing.
  const int64_t c = threadIdx.x * kNormEpl;
  const bool act = c < p.n;
  const int waves = blockDim.x / kWave;
  const QuantConst q = quant_const(p.g);
  float post[kNormEpl], w[kNormEpl];
  Raw16<BF> xr = {}, rr = {};
  int64_t row = blockIdx.x;
  if (act) {
    xr.load(p.X, row * p.n + c);
    if (p.R) rr.load(p.R, row * p.n + c);
  }
  const int64_t lc = act ? c : 0;
  Raw16<false> v;
  if (p.gate) {
    v.load(p.gate, lc);
#pragma unroll
    for (int k = 0; k < 4; k++) own[0][k][threadIdx.x] = v.v[k];
  }
  if (p.b) {
    v.load(p.b, lc);
#pragma unroll
    for (int k = 0; k < 4; k++) own[1][k][threadIdx.x] = v.v[k];
  }
  load_ones(p.post, p.wbf, lc, post);
  load_ones(p.w, p.wbf, lc, w);
  auto times = [&](float (&x)[kNormEpl], int which) {
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const u32x4 u = own[which][k][threadIdx.x];
#pragma unroll
      for (int e = 0; e < 4; e++) x[4 * k + e] = x[4 * k + e] * u2f(u[e]);
    }
  };
  const double rn = 1.0 / (double)p.n;
  constexpr int kInput = 1 << 30;  // this lane's X or R of the row is not finite
  int flags = 0, turn = 0;  // the sums take the two arrays in turn: one barrier lies between a read
                            // of an array and its next use
  for (; row < p.m; row += gridDim.x) {
    const int64_t off = row * p.n + c, next = row + gridDim.x;
    float h[kNormEpl], r[kNormEpl];
    xr.unpack(h);
    if (act && next < p.m) xr.load(p.X, next * p.n + c);
    const uint32_t topx = top_bits(h);
    if (p.norm1) {
      const double sum1 = block_sum(squares16<BF>(h, topx), red[turn], waves);
      turn ^= 1;
      const float r1 = rstd_of(sum1, rn, p.post_eps);
#pragma unroll
      for (int k = 0; k < kNormEpl; k++) h[k] = h[k] * r1 * post[k];
    }
    if (p.gate) times(h, 0);
    if (p.tgate) {
      const float tg = p.tgate[row];
#pragma unroll
      for (int k = 0; k < kNormEpl; k++) h[k] = h[k] * tg;
    }
    rr.unpack(r);
    join16<BF>(h, r, p.rs, p.h, off, act);
    const uint32_t toph = top_bits(h);
    // rare: what is not finite in X or R is not in h either
    if (toph >= kInfBits && (topx >= kInfBits || top_bits(r) >= kInfBits)) flags |= kInput;
    if (act && p.R && next < p.m) rr.load(p.R, next * p.n + c);
    const double sum2 = block_sum(squares16<BF>(h, toph), red[turn], waves);
    turn ^= 1;
    if (!(sum2 <= DBL_MAX)) {  // a value of h that is not finite, which any lane's X or R explains
      const bool in = block_sum(flags & kInput ? 1.0 : 0.0, red[turn], waves) > 0.0;
      turn ^= 1;
      flags = (flags & ~kInput) | (in ? kStNonFinite : kStRange);
    }
    bool over = norm16(h, rstd_of(sum2, rn, p.eps), w, p, off, act);
    if (p.b) times(h, 1);
    over |= quantize16<FMT, G>(h, act, p, off, q);
    if (over && sum2 <= DBL_MAX) flags |= kStRange;  // a value of n or x that is not finite
  }
  if (flags) atomicOr(p.status, flags);
}

// Wider rows: three sweeps of 256 threads, h read back by the thread that stored it.
template <int FMT, int G, bool BF>
__global__ __launch_bounds__(kBlock) void k_block_norm_wide(BlockNormArgs p) {
  __shared__ double red[2][kWaves];
  const int64_t row = (int64_t)blockIdx.x * p.n;
  int flags = 0;
  bool wild = false;  // X or R is not finite
  double sum1 = 0.0, sum2 = 0.0;
  if (p.norm1) {
    for (int64_t c = threadIdx.x * kNormEpl; c < p.n; c += kBlock * kNormEpl) {
      float x[kNormEpl];
      load16<BF>(p.X, row + c, x);
      sum1 += squares16<BF>(x, top_bits(x));
    }
    sum1 = block_sum(sum1, red[0], kWaves);
  }
  const double rn = 1.0 / (double)p.n;
  const float r1 = rstd_of(sum1, rn, p.post_eps), tg = p.tgate ? p.tgate[blockIdx.x] : 1.0f;
  for (int64_t c = threadIdx.x * kNormEpl; c < p.n; c += kBlock * kNormEpl) {
    float h[kNormEpl], r[kNormEpl] = {}, v[kNormEpl];
    load16<BF>(p.X, row + c, h);
    wild |= top_bits(h) >= kInfBits;
    if (p.R) {
      load16<BF>(p.R, row + c, r);
      wild |= top_bits(r) >= kInfBits;
    }
    if (p.norm1) {
      load_ones(p.post, p.wbf, c, v);
#pragma unroll
      for (int k = 0; k < kNormEpl; k++) h[k] = h[k] * r1 * v[k];
    }
    load_ones(p.gate, false, c, v);
#pragma unroll
    for (int k = 0; k < kNormEpl; k++) h[k] = h[k] * v[k] * tg;
    join16<BF>(h, r, p.rs, p.h, row + c, true);
    sum2 += squares16<BF>(h, top_bits(h));
  }
  sum2 = block_sum(sum2, red[1], kWaves);
  // a value of h that is not finite: any lane's X or R explains it
  if (!(sum2 <= DBL_MAX))
    flags |= block_sum(wild ? 1.0 : 0.0, red[0], kWaves) > 0.0 ? kStNonFinite : kStRange;
  const float r2 = rstd_of(sum2, rn, p.eps);
  const QuantConst q = quant_const(p.g);
  // every lane of a wave runs the same trips (the group maxima exchange lanes); lanes past the
  // row's end read its start and store nothing
  for (int64_t c0 = 0; c0 < p.n; c0 += kBlock * kNormEpl) {
    const int64_t c = c0 + threadIdx.x * kNormEpl;
    const bool act = c < p.n;
    const int64_t lc = act ? c : 0;
    float x[kNormEpl], w[kNormEpl], b[kNormEpl];
    load16<BF>(p.h, row + lc, x);
    load_ones(p.w, p.wbf, lc, w);
    load_ones(p.b, false, lc, b);
    bool over = norm16(x, r2, w, p, row + lc, act);
#pragma unroll
    for (int k = 0; k < kNormEpl; k++) x[k] = x[k] * b[k];
    over |= quantize16<FMT, G>(x, act, p, row + lc, q);
    if (over && sum2 <= DBL_MAX) flags |= kStRange;
  }
  if (flags) atomicOr(p.status, flags);
}

constexpr int kBlockNormCols = 16 * kWave * kNormEpl;  // the widest rows of k_block_norm

template <int FMT, int G, bool BF>
static hipError_t block_norm_launch(const BlockNormArgs& p, hipStream_t s) {
  if (p.n > kBlockNormCols) {
    hipLaunchKernelGGL((k_block_norm_wide<FMT, G, BF>), dim3((unsigned)p.m), dim3(kBlock), 0, s, p);
    return hipGetLastError();
  }
  const int waves = (int)((p.n + kWave * kNormEpl - 1) / (kWave * kNormEpl));
  // sixteen waves a CU; what does not fit beside each other by its LDS follows (workgroups of 1, 2, 3 and 5
  // waves)
  const int64_t most = 256 * (16 / waves);
  const dim3 grid((unsigned)(p.m < most ? p.m : most)), block(waves * kWave);
  if (waves <= 4)
    hipLaunchKernelGGL((k_block_norm<FMT, G, BF, 4>), grid, block, 0, s, p);
  else if (waves <= 8)
    hipLaunchKernelGGL((k_block_norm<FMT, G, BF, 8>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((k_block_norm<FMT, G, BF, 16>), grid, block, 0, s, p);
  return hipGetLastError();
}

template <int FMT, int G>
static hipError_t block_norm_type(bool bf16, const BlockNormArgs& p, hipStream_t s) {
  return bf16 ? block_norm_launch<FMT, G, true>(p, s) : block_norm_launch<FMT, G, false>(p, s);
}

template <int FMT>
static hipError_t block_norm_group(int G, bool bf16, const BlockNormArgs& p, hipStream_t s) {
  switch (G) {
    case 16: return block_norm_type<FMT, 16>(bf16, p, s);
    case 32: return block_norm_type<FMT, 32>(bf16, p, s);
    case 64: return block_norm_type<FMT, 64>(bf16, p, s);
    default: return hipErrorInvalidValue;
  }
}

// Launches over chunks of rows so that no grid passes 2^31 threads.
static hipError_t launch_block_norm(int fmt, int G, bool bf16, const BlockNormArgs& whole,
                                    hipStream_t s) {
  constexpr int64_t kRows = 1 << 22;
  for (int64_t t = 0; t < whole.m; t += kRows) {
    BlockNormArgs p = whole;
    p.m = whole.m - t < kRows ? whole.m - t : kRows;
    const int64_t off = t * p.n, in = off * (bf16 ? 2 : 4);
    p.X = static_cast<const char*>(p.X) + in;
    if (p.R) p.R = static_cast<const char*>(p.R) + in;
    p.h = static_cast<char*>(p.h) + in;
    if (p.tgate) p.tgate += t;
    if (p.xo) p.xo = static_cast<char*>(p.xo) + off * (p.xobf ? 2 : 4);
    p.codes += fmt == kMxFp8 ? off : off / 2;
    p.scales = static_cast<char*>(p.scales) + off / G * (fmt == kInt4Bf16 ? 2 : 1);
    hipError_t e;
    switch (fmt) {
      case kInt4Bf16: e = block_norm_group<kInt4Bf16>(G, bf16, p, s); break;
      case kMxInt4: e = block_norm_group<kMxInt4>(G, bf16, p, s); break;
      case kMxFp4: e = block_norm_group<kMxFp4>(G, bf16, p, s); break;
      case kNvFp4: e = block_norm_group<kNvFp4>(G, bf16, p, s); break;
      default: e = block_norm_group<kMxFp8>(G, bf16, p, s); break;
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

static bool is_type(dq_dtype t) { return t == DQ_F32 || t == DQ_BF16; }

// The host-side checks of both forms, and the kernel's arguments but the status word. `word`: the
// status word, or the workspace that holds it (null: neither is the caller's).
static dq_status block_norm_args(const void* X, dq_dtype xt, int post_norm, const void* post_weight,
                                 double post_eps, const float* gate, const float* token_gate,
                                 const void* residual, float residual_scale, void* residual_out,
                                 int64_t tokens, int64_t cols, const void* weight, dq_dtype wt,
                                 double eps, void* x_out, dq_dtype xot, const float* b,
                                 dq_format fmt, int group, float g, uint8_t* codes,
                                 void* inner_scales, const Span& word, BlockNormArgs* p) {
  if ((int)fmt < 0 || (int)fmt > kMxFp8 || !is_type(xt)) return DQ_ERR_UNSUPPORTED;
  if ((weight || post_weight) && !is_type(wt)) return DQ_ERR_UNSUPPORTED;
  if (x_out && !is_type(xot)) return DQ_ERR_UNSUPPORTED;
  if (post_norm != 0 && post_norm != 1) return DQ_ERR_ARG;
  if (!X || !residual_out || !codes || !inner_scales || (post_weight && !post_norm)) return DQ_ERR_ARG;
  if (tokens < 1 || cols < 1 || (group != 16 && group != 32 && group != 64) || cols % group != 0)
    return DQ_ERR_ARG;
  if (tokens > INT32_MAX || cols > ((int64_t)1 << 40) / tokens) return DQ_ERR_ARG;
  if (!(eps > 0.0) || eps > DBL_MAX) return DQ_ERR_ARG;
  if (post_norm && (!(post_eps > 0.0) || post_eps > DBL_MAX)) return DQ_ERR_ARG;
  if (!(fabsf(residual_scale) <= FLT_MAX)) return DQ_ERR_ARG;
  if (fmt == DQ_FMT_NVFP4 && (!(g > 0.0f) || g > FLT_MAX)) return DQ_ERR_ARG;
  if (((uintptr_t)X | (uintptr_t)residual | (uintptr_t)residual_out | (uintptr_t)post_weight |
       (uintptr_t)gate | (uintptr_t)weight | (uintptr_t)b | (uintptr_t)x_out) & 15u)
    return DQ_ERR_ARG;
  if ((uintptr_t)token_gate & 3u) return DQ_ERR_ARG;
  if ((uintptr_t)codes & (fmt == DQ_FMT_MXFP8 ? 15u : 7u)) return DQ_ERR_ARG;
  if (fmt == DQ_FMT_INT4_BF16 && ((uintptr_t)inner_scales & 1u)) return DQ_ERR_ARG;
  const size_t n = (size_t)tokens * (size_t)cols, bytes = n * (xt == DQ_BF16 ? 2 : 4);
  const size_t vb = (size_t)cols * 4, wb = wt == DQ_BF16 ? vb / 2 : vb;
  if (any_overlap({{codes, fmt == DQ_FMT_MXFP8 ? n : n / 2},
                   {inner_scales, n / (size_t)group * (fmt == DQ_FMT_INT4_BF16 ? 2 : 1)},
                   {residual_out, bytes},
                   {x_out, n * (xot == DQ_BF16 ? 2 : 4)},
                   word},
                  {{X == residual_out ? nullptr : X, bytes},
                   {residual == residual_out ? nullptr : residual, bytes},
                   {post_weight, wb},
                   {gate, vb},
                   {token_gate, (size_t)tokens * 4},
                   {weight, wb},
                   {b, vb}}))
    return DQ_ERR_ARG;
  p->X = X;
  p->R = residual;
  p->h = residual_out;
  p->post = post_weight;
  p->gate = gate;
  p->tgate = token_gate;
  p->w = weight;
  p->b = b;
  p->xo = x_out;
  p->m = tokens;
  p->n = cols;
  p->post_eps = post_norm ? post_eps : 1.0;
  p->eps = eps;
  p->rs = residual_scale;
  p->g = fmt == DQ_FMT_NVFP4 ? g : 1.0f;
  p->codes = codes;
  p->scales = inner_scales;
  p->status = static_cast<int*>(const_cast<void*>(word.p));
  p->norm1 = post_norm != 0;
  p->wbf = wt == DQ_BF16;
  p->xobf = xot == DQ_BF16;
  return DQ_OK;
}

}  // namespace dq

extern "C" {

dq_status dq_block_norm_quantize_act_async(
    const void* X, dq_dtype xt, int post_norm, const void* post_weight, double post_eps,
    const float* gate, const float* token_gate, const void* residual, float residual_scale,
    void* residual_out, int64_t tokens, int64_t cols, const void* weight, dq_dtype wt, double eps,
    void* x_out, dq_dtype xot, const float* b, dq_format fmt, int group, float g, uint8_t* codes,
    void* inner_scales, int* status, hipStream_t stream) {
  using namespace dq;
  BlockNormArgs p{};
  const dq_status st = block_norm_args(X, xt, post_norm, post_weight, post_eps, gate, token_gate,
                                       residual, residual_scale, residual_out, tokens, cols, weight,
                                       wt, eps, x_out, xot, b, fmt, group, g, codes, inner_scales,
                                       {status, sizeof *status}, &p);
  if (st != DQ_OK) return st;
  if (!status || ((uintptr_t)status & 3u)) return DQ_ERR_ARG;
  return launch_block_norm(fmt, group, xt == DQ_BF16, p, stream) == hipSuccess ? DQ_OK : DQ_ERR_HIP;
}

dq_status dq_block_norm_quantize_act(
    const void* X, dq_dtype xt, int post_norm, const void* post_weight, double post_eps,
    const float* gate, const float* token_gate, const void* residual, float residual_scale,
    void* residual_out, int64_t tokens, int64_t cols, const void* weight, dq_dtype wt, double eps,
    void* x_out, dq_dtype xot, const float* b, dq_format fmt, int group, float g, uint8_t* codes,
    void* inner_scales, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  using namespace dq;
  if (workspace && workspace_bytes < DQ_NORM_WORKSPACE_BYTES) return DQ_ERR_WORKSPACE;
  BlockNormArgs p{};
  dq_status st = block_norm_args(X, xt, post_norm, post_weight, post_eps, gate, token_gate,
                                 residual, residual_scale, residual_out, tokens, cols, weight, wt,
                                 eps, x_out, xot, b, fmt, group, g, codes, inner_scales,
                                 {workspace, DQ_NORM_WORKSPACE_BYTES}, &p);
  if (st != DQ_OK) return st;
  if ((uintptr_t)workspace & 255u) return DQ_ERR_ARG;
  void* ws = workspace;
  if (!ws && hipMallocAsync(&ws, DQ_NORM_WORKSPACE_BYTES, stream) != hipSuccess) return DQ_ERR_HIP;
  p.status = static_cast<int*>(ws);
  int host = 0;
  if (launch_clear(p.status, 1, stream) != hipSuccess ||
      launch_block_norm(fmt, group, xt == DQ_BF16, p, stream) != hipSuccess ||
      hipMemcpyAsync(&host, p.status, sizeof host, hipMemcpyDeviceToHost, stream) != hipSuccess ||
      hipStreamSynchronize(stream) != hipSuccess)
    st = DQ_ERR_HIP;
  if (!workspace) (void)hipFreeAsync(ws, stream);
  if (st != DQ_OK) return st;
  if (host & kStNonFinite) return DQ_ERR_NONFINITE;
  return (host & kStRange) ? DQ_ERR_RANGE : DQ_OK;
}

}  // extern "C"
