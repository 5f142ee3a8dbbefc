// What stands between two blocks of a decoder layer, for gfx950: the norm of a
// block's output, its gate, the scaled residual stream and the next block's norm, in
// one pass with the quantization of that norm's output; and SiLU(gate) x up with
// block-wise quantized output.
//
//   n  = post norm of y (or y);  t = fl32(n * gate) (or n)
//   h' = bf16(fl32(fl32(res h) + t))                          (the new residual stream)
//   z  = norm of h' with the next block's gain (UAQ's s folded in) -> codes, or bf16
//
// The norms' roundings are the norm producer's: statistics in float64, mean and r rounded
// once to fp32, fp32 products in a fixed order (contraction is off in this file). A call
// gives the same bits on every run, and the producer's unless a statistic's exact value
// lies within about 2^-45 of an fp32 rounding boundary: sums are taken in another order
// here, LayerNorm's variance loses up to 6 bits to cancellation (2^-47), 1 / sqrt is good
// to 2^-48.
#include "qr_internal.h"
#include "qr_mx.h"

#pragma clang fp contract(off)

namespace qr {
namespace {

// Sum / maximum over a wave, every lane getting it: within 16 lanes by lane permutes of
// the vector ALU, then across the four groups through LDS permutes.
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)b, CTRL, 0xf, 0xf, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(b >> 32), CTRL, 0xf, 0xf, true);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp<0xB1>(v);   // quad_perm [1, 0, 3, 2]
  v += dpp<0x4E>(v);   // quad_perm [2, 3, 0, 1]
  v += dpp<0x141>(v);  // row_half_mirror
  v += dpp<0x140>(v);  // row_mirror
  v += __shfl_xor(v, 16, 64);
  v += __shfl_xor(v, 32, 64);
  return v;
}

// Sums / maximum over the block, whose waves leave theirs in `red` (not used by another
// reduction of the kernel, so one barrier each).
template <int N>
__device__ __forceinline__ void row_sum(double (&v)[N], double (*red)[16]) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    v[n] = wave_sum(v[n]);
    if ((threadIdx.x & 63) == 0) red[n][threadIdx.x >> 6] = v[n];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    v[n] = red[n][0];
    for (uint32_t w = 1; w < blockDim.x >> 6; ++w) v[n] += red[n][w];
  }
}

__device__ __forceinline__ float row_max(float v, float* red) {
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
  for (uint32_t w = 1; w < blockDim.x >> 6; ++w) v = fmaxf(v, red[w]);
  return v;
}

__device__ __forceinline__ void load8(const float* p, int64_t c, float* v) {
  const float4 a = reinterpret_cast<const float4*>(p)[2 * c];
  const float4 b = reinterpret_cast<const float4*>(p)[2 * c + 1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
}

// Eight INT8 codes rint(fl32(v / t)), |v| <= 127 t, inv = fl32(1 / t) finite: v inv is
// within 2^-15 of fl32(v / t) and rounds to the same integer unless it lies that close to
// a half; only then (one value in 8000) is the division done. Adding 1.5 2^23 rounds to
// an integer (ties to even) and leaves it in the low byte.
__device__ __forceinline__ uint2 int8_codes8(const float* v, float t, float inv) {
  constexpr float kMagic = 12582912.0f;
  uint32_t b[8];
  float far = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float q = v[e] * inv, m = q + kMagic;
    far = fmaxf(far, fabsf(q - (m - kMagic)));
    b[e] = __float_as_uint(m);
  }
  if (far > 0.5f - 0x1p-14f)
    return make_uint2(quant_codes4<kQInt8>(v[0], v[1], v[2], v[3], t),
                      quant_codes4<kQInt8>(v[4], v[5], v[6], v[7], t));
  auto pack = [](uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
    // bytes: 4 .. 7 of the first operand, 0 .. 3 of the second
    const uint32_t lo = __builtin_amdgcn_perm(a1, a0, 0x0c0c0400u), hi = __builtin_amdgcn_perm(a3, a2, 0x04000c0cu);
    return lo | hi;
  };
  return make_uint2(pack(b[0], b[1], b[2], b[3]), pack(b[4], b[5], b[6], b[7]));
}

// 1 / sqrt(x) in float64 to 2^-48: the instruction's estimate (2^-24) and two Newton steps
// (the second for the estimate's last bits); 0 and infinity as the estimate gives them.
__device__ __forceinline__ double rsqrt64(double x) {
  const double y0 = __builtin_amdgcn_rsq(x);
  double y = y0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const double h = 0.5 * y;
    y = fma(h, fma(-x * y, y, 1.0), y);
  }
  return x > 0.0 && x < __builtin_inf() ? y : y0;
}

// Norm of the row held as v[i][8] (chunk c(i) = lt + i tpr of thread lt) in place;
// `live(i)` says which chunks exist. inv_k = 1 / K; red: three arrays of 16.
//
// LayerNorm's sum of (v - mu)^2 is s2 - mu (2 s1 - K mu) with s1, s2 the sums of v and v^2,
// all in float64: one pass and one barrier instead of two. The cancellation costs
// s2 / that of its 53 bits; where it is more than 6 (a mean of eight deviations) the
// second pass is made.
//
// The mean's quotient by K is a product with fl64(1 / K) and one correction by its remainder
// (exact in an fma): a mean that float64 holds comes out as it is. One row in a hundred has a
// mean half way between two fp32 numbers (short sums over a K with few odd factors), and the
// product alone falls beside it for K of some odd factors, to be rounded to the wrong one.
template <int KIND, int MAXC, typename Live>
__device__ __forceinline__ void norm_row(float (&v)[MAXC][8], const Live& live, int lt, int tpr, double inv_k,
                                         double k, const float* gamma, const float* beta, float eps,
                                         double (*red)[16]) {
  float mu = 0.0f;
  double var;
  if constexpr (KIND == 1) {
    double s[2] = {0.0, 0.0};
#pragma unroll
    for (int i = 0; i < MAXC; ++i)
      if (live(i))
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const double d = (double)v[i][e];
          s[0] += d;
          s[1] = fma(d, d, s[1]);
        }
    row_sum<2>(s, red);
    const double q = s[0] * inv_k;
    mu = (float)fma(fma(-q, k, s[0]), inv_k, q);
    const double m = (double)mu;
    var = s[1] - m * (2.0 * s[0] - k * m);
    if (!(var * 64.0 > s[1])) {  // the same for every thread of the block
      double t[1] = {0.0};
#pragma unroll
      for (int i = 0; i < MAXC; ++i)
        if (live(i))
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const double d = (double)v[i][e] - (double)mu;
            t[0] = fma(d, d, t[0]);
          }
      row_sum<1>(t, red + 2);
      var = t[0];
    }
  } else {
    double s[1] = {0.0};
#pragma unroll
    for (int i = 0; i < MAXC; ++i)
      if (live(i))
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const double d = (double)v[i][e];
          s[0] = fma(d, d, s[0]);
        }
    row_sum<1>(s, red);
    var = s[0];
  }
  const float r = (float)rsqrt64(var * inv_k + (double)eps);
#pragma unroll
  for (int i = 0; i < MAXC; ++i) {
    if (!live(i)) continue;
    const int64_t c = lt + (int64_t)i * tpr;
    float g[8];
    load8(gamma, c, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = KIND == 1 ? v[i][e] - mu : v[i][e];
      v[i][e] = (d * r) * g[e];
    }
    if (beta) {
      load8(beta, c, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] + g[e];
    }
  }
}

// One row per block of tpr threads, held in registers, so one pass over memory: K <= 8 MAXC
// tpr. 4096 x 5120 to INT8: 35 us with RMS (147 MB, 4.2 TB/s), 47 - 50 with LayerNorm, biases
// and a gate per token (189 MB, 3.8 - 4.0 TB/s; 5 us of it the four parameter rows, 80 KB that each
// block reads from the L2). Two or four rows a block, which share those, took 44 (RMS with
// biases and gate; 48 here) and 54 us (LayerNorm). The residual row
// is loaded with the block's output, but with four chunks a thread after the post norm. At
// most 64 registers, eight waves a SIMD (RMS keeps to that by itself; LayerNorm, 4096 x 3584
// to INT8: 24.7 us, and 30.3 with the 68 registers it would take). Every output row is read
// by the thread that writes it before it does, so Hout may be an input's rows.
template <int KIND, int MAXC>
__global__ __launch_bounds__(1024, KIND == 1 ? 8 : 4) void block_norm_kernel(const BlockNormArgs p) {
  __shared__ double red[6][16];
  __shared__ float redf[16];
  const int tpr = (int)blockDim.x, lt = (int)threadIdx.x;
  // an XCD takes a contiguous range of rows: their scale bytes share lines
  const uint32_t g8 = gridDim.x & ~7u;
  const uint32_t blk = blockIdx.x < g8 ? (blockIdx.x & 7u) * (g8 >> 3) + (blockIdx.x >> 3) : blockIdx.x;
  const int64_t row = p.row0 + blk, K = p.K;
  const double inv_k = p.inv_k, k = (double)K;
  const int nch = (int)(K >> 3), niter = (nch + tpr - 1) / tpr;
  const uint4* yr = reinterpret_cast<const uint4*>(p.Y + row * p.ldy);
  const uint4* hr = reinterpret_cast<const uint4*>(p.H + row * p.ldh);
  auto live = [&](int i) { return lt + i * tpr < nch; };

  constexpr bool kLateH = MAXC > 2;
  uint4 hraw[MAXC];
  float v[MAXC][8];
#pragma unroll
  for (int i = 0; i < MAXC; ++i) {
    if (i >= niter) continue;
    const int c = lt + i * tpr, cc = c < nch ? c : nch - 1;
    bf16x8(yr[cc], v[i]);
    if constexpr (!kLateH) hraw[i] = hr[cc];
  }
  if (p.post_gamma)
    norm_row<KIND, MAXC>(v, live, lt, tpr, inv_k, k, p.post_gamma, p.post_beta, p.eps, red);

#pragma unroll
  for (int i = 0; i < MAXC; ++i) {
    if (!live(i)) continue;
    const int c = lt + i * tpr;
    if constexpr (kLateH) hraw[i] = hr[c];
    if (p.gate) {
      float g[8];
      if (p.gate_rows)
        bf16x8(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.gate) + row * p.ldgate)[c], g);
      else
        load8(static_cast<const float*>(p.gate), c, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] * g[e];
    }
    float h[8];
    bf16x8(hraw[i], h);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = h[e] * p.res + v[i][e];
    const uint4 o = pack8(v[i]);
    reinterpret_cast<uint4*>(p.Hout + row * p.ldo)[c] = o;
    bf16x8(o, v[i]);
  }

  norm_row<KIND, MAXC>(v, live, lt, tpr, inv_k, k, p.gamma, p.beta, p.eps, red + 3);

  if (p.fmt == kActMxFp4 || p.fmt == kActMxFp8) {
    // every lane takes part in the block maxima
    uint8_t* s = static_cast<uint8_t*>(p.scales);
#pragma unroll
    for (int i = 0; i < MAXC; ++i) {
      if (i >= niter) continue;
      const int64_t c = lt + i * tpr;
      const bool on = live(i);
      if (!on)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
      if (p.fmt == kActMxFp4) mx_store_row8<true>(v[i], on, row, p.M, c, K, p.codes, s);
      else mx_store_row8<false>(v[i], on, row, p.M, c, K, p.codes, s);
    }
    return;
  }
  if (p.fmt == kActBf16) {
#pragma unroll
    for (int i = 0; i < MAXC; ++i)
      if (live(i)) reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.codes) + row * K)[lt + i * tpr] = pack8(v[i]);
    return;
  }
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < MAXC; ++i)
    if (live(i))
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[i][e]));
  amax = row_max(amax, redf);
  const bool i8 = p.fmt == kActInt8;
  const float t = amax / (i8 ? qmax<kQInt8>() : qmax<kQFp8>()), inv = 1.0f / t;
  if (lt == 0) static_cast<float*>(p.scales)[row] = t;
#pragma unroll
  for (int i = 0; i < MAXC; ++i) {
    if (!live(i)) continue;
    uint2 q = make_uint2(0u, 0u);
    if (t != 0.0f) {
      if (i8 && inv < 3.0e38f) {
        q = int8_codes8(v[i], t, inv);
      } else if (i8) {
        q.x = quant_codes4<kQInt8>(v[i][0], v[i][1], v[i][2], v[i][3], t);
        q.y = quant_codes4<kQInt8>(v[i][4], v[i][5], v[i][6], v[i][7], t);
      } else {
        q.x = quant_codes4<kQFp8>(v[i][0], v[i][1], v[i][2], v[i][3], t);
        q.y = quant_codes4<kQFp8>(v[i][4], v[i][5], v[i][6], v[i][7], t);
      }
    }
    reinterpret_cast<uint2*>(p.codes + row * K)[lt + i * tpr] = q;
  }
}

// g u / (1 + exp(-g)) in float64, relative error below 2^-40 (so its fp32 rounding is the
// exact value's unless that lies as close to a rounding boundary). With x = -g log2(e)
// (off by at most 2^-43), n = rint(x), exp(-g) = 2^n 2^f, |f| <= 1/2, 2^f by its Taylor
// polynomial of degree 10 (remainder (ln 2 / 2)^11 / 11! < 2^-42); the quotient by the
// reciprocal instruction (relative error at most 2^-23) and a Newton step (2^-46). g is
// clamped to +-700 for the exponential, where the value is g u or rounds to zero. Of the
// order of half the operations of the library's exp and an IEEE division.
__device__ __forceinline__ float silu_mul(float g, float u) {
  const double x = (double)__builtin_amdgcn_fmed3f(g, -700.0f, 700.0f) * -1.4426950408889634;
  const double n = rint(x), f = x - n;
  double p = 7.054911620801121e-09;  // ln(2)^k / k!, k = 10 .. 0
  p = fma(p, f, 1.0178086009239696e-07);
  p = fma(p, f, 1.3215486790144305e-06);
  p = fma(p, f, 1.5252733804059838e-05);
  p = fma(p, f, 0.00015403530393381606);
  p = fma(p, f, 0.0013333558146428441);
  p = fma(p, f, 0.009618129107628477);
  p = fma(p, f, 0.055504108664821576);
  p = fma(p, f, 0.2402265069591007);
  p = fma(p, f, 0.6931471805599453);
  p = fma(p, f, 1.0);
  const double d = 1.0 + ldexp(p, (int)n);
  double r = __builtin_amdgcn_rcp(d);
  r = fma(r, fma(-d, r, 1.0), r);
  return (float)(((double)g * (double)u) * r);
}

// The same in fp32 for g >= -80, off by less than 2^-21.3 of it where nothing underflows
// (the sigmoid by at most 2^-22.4, the largest error over all bf16 g; two products):
// exp(-g) = 2^(-g c) (1 - g d) with c the 15 leading bits of log2(e), so that g c is exact,
// and d = (log2(e) - c) ln 2, |g d| < 2^-11.3.
__device__ __forceinline__ float silu_mul_fast(float g, float u) {
  const float e = __builtin_amdgcn_exp2f(g * -1.44268798828125f) * fmaf(g, -4.888495152e-06f, 1.0f);
  return (g * __builtin_amdgcn_rcpf(1.0f + e)) * u;
}

// Rows [row0, row0 + w.rows), eight outputs a thread, block-wise codes: those of silu_mul's
// values. Rounding to codes is monotone, and so is the scale in the block's maximum: where
// the values times 1 - 2^-19 and times 1 + 2^-19 give the same codes and scale, so does
// silu_mul's value, which the fp32 form comes closer to than 2^-20 (2^-21.3, and the
// roundings to fp32 of that value and of the product with the factor). Else (one wave in 60
// for E4M3 codes), or if a block is not finite or its maximum below 2^-100, or a g < -80, the
// wave evaluates silu_mul. 1001 x 27648 to E4M3, 138 MB: 25.8 us, 5.4 TB/s (39.3 with
// silu_mul for all, bound by its float64 operations); 256 x 18944 to E2M1 8.3 us (10.8).
template <bool FP4>
__global__ __launch_bounds__(256) void silu_mx_kernel(const uint16_t* __restrict__ G,
                                                      const uint16_t* __restrict__ U, int64_t M,
                                                      int64_t N, int64_t ldg, int64_t ldu,
                                                      uint8_t* __restrict__ codes,
                                                      uint8_t* __restrict__ scales, int64_t row0,
                                                      ChunkWalk w) {
  constexpr float kLow = 1.0f - 0x1p-19f, kHigh = 1.0f + 0x1p-19f;
  const uint32_t i = w.first(1), r = w.row(i), c = i - r * w.cpr;
  const int64_t row = row0 + r;
  const bool live = i < w.rows * w.cpr && c < (uint32_t)(N >> 3);
  uint4 g = make_uint4(0u, 0u, 0u, 0u), u = g;
  if (live) {
    g = *reinterpret_cast<const uint4*>(G + row * ldg + 8 * c);
    u = *reinterpret_cast<const uint4*>(U + row * ldu + 8 * c);
  }
  float a[8], b[8], t[8], least = 0.0f;
  bf16x8(g, a);
  bf16x8(u, b);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    t[e] = silu_mul_fast(a[e], b[e]);
    least = fminf(least, a[e]);
  }
  const uint32_t m = mx_block_max(t);  // a NaN or an infinity is above every number
  const float amax = __uint_as_float(m);
  uint32_t sb = mx_scale_byte<FP4>(__float_as_uint(amax * kHigh));
  const float inv = mx_inv_scale(sb);
  uint2 q = mx_codes8_times<FP4>(t, inv * kLow);
  const uint2 high = mx_codes8_times<FP4>(t, inv * kHigh);
  const bool sure = m >= 0x0d800000u && m < 0x7f000000u && least >= -80.0f && q.x == high.x && q.y == high.y &&
                    sb == mx_scale_byte<FP4>(__float_as_uint(amax * kLow));
  if (__builtin_amdgcn_ballot_w64(live && !sure) != 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = silu_mul(a[e], b[e]);
    sb = mx_block_scale<FP4>(a);
    q = mx_codes8<FP4>(a, sb);
  }
  mx_store_codes8<FP4>(q, live ? sb : 0u, live, row, M, c, N, codes, scales);
}

template <int MAXC>
void launch_rows(BlockNormArgs p, int kind, hipStream_t st) {
  constexpr int64_t kBlocks = (int64_t)1 << 21;  // per launch
  const int nch = (int)(p.K >> 3), waves = ((nch + MAXC - 1) / MAXC + 63) >> 6;
  const int threads = 64 * (waves > 0 ? waves : 1);
  p.inv_k = 1.0 / (double)p.K;
  for (p.row0 = 0; p.row0 < p.M; p.row0 += kBlocks) {
    const int64_t blocks = p.M - p.row0 < kBlocks ? p.M - p.row0 : kBlocks;
    const dim3 g((unsigned)blocks), b(threads);
    if (kind == 0) hipLaunchKernelGGL((block_norm_kernel<0, MAXC>), g, b, 0, st, p);
    else hipLaunchKernelGGL((block_norm_kernel<1, MAXC>), g, b, 0, st, p);
  }
}

}  // namespace

// Chunks a thread, from the time of 3584-wide RMS rows to MXFP4 with one / two / four:
// few rows want many threads a row (256 rows 4.3 / 5.0 / 6.7 us), many rows few, whose
// barriers cost less (1200 rows 10.5 / 9.6 / 10.5; 4096 rows 27.9 / 24.1 / 22.2). Rows under
// 2048 values leave four chunks a thread no full wave (4096 x 512 5.5 / 5.5 / 5.9).
hipError_t launch_block_norm(const BlockNormArgs& p, int kind, hipStream_t st) {
  const bool per_token = p.fmt == kActInt8 || p.fmt == kActFp8;  // rows of no values have scale 0
  if (p.M == 0 || (p.K == 0 && !per_token)) return hipSuccess;
  const int64_t nch = p.K >> 3;
  if (nch <= 1024 && p.M <= 512) launch_rows<1>(p, kind, st);
  else if (nch <= 2048 && (p.M < 2048 || nch < 256)) launch_rows<2>(p, kind, st);
  else launch_rows<4>(p, kind, st);
  return hipGetLastError();
}

hipError_t launch_silu_mx(const void* G, const void* U, int64_t M, int64_t N, int64_t ldg, int64_t ldu,
                          int fmt, void* codes, uint8_t* scales, hipStream_t st) {
  const uint16_t *g = static_cast<const uint16_t*>(G), *u = static_cast<const uint16_t*>(U);
  uint8_t* q = static_cast<uint8_t*>(codes);
  const dim3 b(256);
  return chunk_launches(M, ((N + 127) >> 7) << 4, 1, [&](int64_t r, ChunkWalk w, dim3 gr) {
    if (fmt == kActMxFp4) hipLaunchKernelGGL(silu_mx_kernel<true>, gr, b, 0, st, g, u, M, N, ldg, ldu, q, scales, r, w);
    else hipLaunchKernelGGL(silu_mx_kernel<false>, gr, b, 0, st, g, u, M, N, ldg, ldu, q, scales, r, w);
  });
}

}  // namespace qr
