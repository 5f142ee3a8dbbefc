// What stands between two blocks of a decoder layer, for gfx950: the norm of a
// block's output, its gate, the scaled residual stream and the next block's norm, in
// one pass with the quantization of that norm's output; and SiLU(gate) x up with
// block-wise quantized output.
//
//   n  = post norm of y (or y);  t = fl32(n * gate) (or n)
//   h' = bf16(fl32(fl32(res h) + t))                          (the new residual stream)
//   z  = norm of h' with the next block's gain (UAQ's s folded in) -> codes, or bf16
//
// The norms' arithmetic is the norm producer's: statistics in float64, r rounded
// once to fp32, fp32 products in a fixed order (contraction is off in this file), so
// codes are reproducible bit for bit.
#include "qr_internal.h"
#include "qr_mx.h"

#pragma clang fp contract(off)

namespace qr {
namespace {

constexpr int block_threads(int tpr) { return tpr < 256 ? 256 : tpr; }

template <int TPR>
__device__ __forceinline__ double row_sum(double v, double* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if constexpr (TPR > 64) {
    __syncthreads();  // red may still be read from the last reduction
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = red[0];
#pragma unroll
    for (int w = 1; w < TPR / 64; ++w) s += red[w];
    v = s;
  }
  return v;
}

template <int TPR>
__device__ __forceinline__ float row_max(float v, double* red) {
  v = wave_max(v);
  if constexpr (TPR > 64) {
    float* redf = reinterpret_cast<float*>(red);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) redf[threadIdx.x >> 6] = v;
    __syncthreads();
    float m = redf[0];
#pragma unroll
    for (int w = 1; w < TPR / 64; ++w) m = fmaxf(m, redf[w]);
    v = m;
  }
  return v;
}

__device__ __forceinline__ void load8(const float* p, int64_t c, float* v) {
  const float4 a = reinterpret_cast<const float4*>(p)[2 * c];
  const float4 b = reinterpret_cast<const float4*>(p)[2 * c + 1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ uint4 pack8(const float* v) {
  uint32_t h[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = f32_to_bf16_any(v[e]);
  return make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
}

// Norm of the row held as v[i][8] (chunk lt + i TPR of thread lt) in place; `live(i)`
// says which chunks exist.
template <int KIND, int TPR, int MAXC, typename Live>
__device__ __forceinline__ void norm_row(float (&v)[MAXC][8], const Live& live, int lt, int64_t K,
                                         const float* gamma, const float* beta, float eps, double* red) {
  float mu = 0.0f;
  if constexpr (KIND == 1) {
    double s1 = 0.0;
#pragma unroll
    for (int i = 0; i < MAXC; ++i)
      if (live(i))
#pragma unroll
        for (int e = 0; e < 8; ++e) s1 += (double)v[i][e];
    mu = (float)(row_sum<TPR>(s1, red) / (double)K);
  }
  double s2 = 0.0;
#pragma unroll
  for (int i = 0; i < MAXC; ++i)
    if (live(i))
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const double d = KIND == 1 ? (double)v[i][e] - (double)mu : (double)v[i][e];
        s2 += d * d;
      }
  s2 = row_sum<TPR>(s2, red);
  const float r = (float)(1.0 / sqrt(s2 / (double)K + (double)eps));
#pragma unroll
  for (int i = 0; i < MAXC; ++i) {
    if (!live(i)) continue;
    const int64_t c = lt + (int64_t)i * TPR;
    float g[8];
    load8(gamma, c, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = KIND == 1 ? v[i][e] - mu : v[i][e];
      v[i][e] = (d * r) * g[e];
    }
    if (beta) {
      float b[8];
      load8(beta, c, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] + b[e];
    }
  }
}

// One row per TPR threads, held in registers: K <= 8 MAXC TPR. The residual row is
// loaded with the block's output, but by the 1024-thread blocks of the longest rows,
// which have 128 registers a thread, after the post norm.
template <int KIND, int TPR, int MAXC>
__global__ __launch_bounds__(block_threads(TPR)) void block_norm_kernel(const BlockNormArgs p) {
  constexpr int RPB = block_threads(TPR) / TPR;
  __shared__ double red[16];
  const int lt = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  const bool valid = row < p.M;
  const int64_t K = p.K, nch = K >> 3, rr = valid ? row : p.M - 1;
  const int niter = (int)((nch + TPR - 1) / TPR);
  const uint4* yr = reinterpret_cast<const uint4*>(p.Y + rr * p.ldy);
  const uint4* hr = reinterpret_cast<const uint4*>(p.H + rr * p.ldh);
  auto live = [&](int i) { return valid && i < niter && lt + (int64_t)i * TPR < nch; };

  constexpr bool kLateH = TPR == 1024 && MAXC > 2;
  uint4 hraw[MAXC];
  float v[MAXC][8];
#pragma unroll
  for (int i = 0; i < MAXC; ++i) {
    if (i >= niter) continue;
    const int64_t c = lt + (int64_t)i * TPR, cc = c < nch ? c : nch - 1;
    bf16x8(yr[cc], v[i]);
    if constexpr (!kLateH) hraw[i] = hr[cc];
  }
  if (p.post_gamma) norm_row<KIND, TPR, MAXC>(v, live, lt, K, p.post_gamma, p.post_beta, p.eps, red);

#pragma unroll
  for (int i = 0; i < MAXC; ++i) {
    if (!live(i)) continue;
    const int64_t c = lt + (int64_t)i * TPR;
    if (p.gate) {
      float g[8];
      if (p.gate_rows)
        bf16x8(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.gate) + rr * p.ldgate)[c], g);
      else
        load8(static_cast<const float*>(p.gate), c, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] * g[e];
    }
    float h[8];
    if constexpr (kLateH) hraw[i] = hr[c];
    bf16x8(hraw[i], h);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = h[e] * p.res + v[i][e];
    const uint4 o = pack8(v[i]);
    reinterpret_cast<uint4*>(p.Hout + rr * p.ldo)[c] = o;
    bf16x8(o, v[i]);
  }

  norm_row<KIND, TPR, MAXC>(v, live, lt, K, p.gamma, p.beta, p.eps, red);

  if (p.fmt == kActMxFp4 || p.fmt == kActMxFp8) {
    // every lane takes part in the block maxima
#pragma unroll
    for (int i = 0; i < MAXC; ++i) {
      if (i >= niter) continue;
      const int64_t c = lt + (int64_t)i * TPR;
      const bool on = live(i);
      if (!on)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
      uint8_t* s = static_cast<uint8_t*>(p.scales);
      if (p.fmt == kActMxFp4) mx_store_row8<true>(v[i], on, row, p.M, c, K, p.codes, s);
      else mx_store_row8<false>(v[i], on, row, p.M, c, K, p.codes, s);
    }
    return;
  }
  if (p.fmt == kActBf16) {
#pragma unroll
    for (int i = 0; i < MAXC; ++i)
      if (live(i))
        reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.codes) + row * K)[lt + (int64_t)i * TPR] =
            pack8(v[i]);
    return;
  }
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < MAXC; ++i)
    if (live(i))
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[i][e]));
  amax = row_max<TPR>(amax, red);
  if (!valid) return;
  const bool i8 = p.fmt == kActInt8;
  const float t = amax / (i8 ? qmax<kQInt8>() : qmax<kQFp8>());
  if (lt == 0) static_cast<float*>(p.scales)[row] = t;
#pragma unroll
  for (int i = 0; i < MAXC; ++i) {
    if (!live(i)) continue;
    uint2 q = make_uint2(0u, 0u);
    if (t != 0.0f) {
      if (i8) {
        q.x = quant_codes4<kQInt8>(v[i][0], v[i][1], v[i][2], v[i][3], t);
        q.y = quant_codes4<kQInt8>(v[i][4], v[i][5], v[i][6], v[i][7], t);
      } else {
        q.x = quant_codes4<kQFp8>(v[i][0], v[i][1], v[i][2], v[i][3], t);
        q.y = quant_codes4<kQFp8>(v[i][4], v[i][5], v[i][6], v[i][7], t);
      }
    }
    reinterpret_cast<uint2*>(p.codes + row * K)[lt + (int64_t)i * TPR] = q;
  }
}

// Eight outputs per lane: a = fl32(g u / (1 + exp(-g))) in float64, block-wise codes.
template <bool FP4>
__global__ __launch_bounds__(256) void silu_mx_kernel(const uint16_t* __restrict__ G,
                                                      const uint16_t* __restrict__ U, int64_t M,
                                                      int64_t N, int64_t ldg, int64_t ldu,
                                                      uint8_t* __restrict__ codes,
                                                      uint8_t* __restrict__ scales) {
  const int64_t cpr = ((N + 127) >> 7) << 4;
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = idx / cpr, c = idx - row * cpr;
  const bool live = row < M && 8 * c < N;
  float v[8] = {};
  if (live) {
    float g[8], u[8];
    bf16x8(*reinterpret_cast<const uint4*>(G + row * ldg + 8 * c), g);
    bf16x8(*reinterpret_cast<const uint4*>(U + row * ldu + 8 * c), u);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double gd = g[e];
      v[e] = (float)((gd * (double)u[e]) / (1.0 + exp(-gd)));
    }
  }
  mx_store_row8<FP4>(v, live, row, M, c, N, codes, scales);
}

template <int TPR, int MAXC>
void launch_rows(const BlockNormArgs& p, int kind, hipStream_t st) {
  constexpr int NT = block_threads(TPR), RPB = NT / TPR;
  const dim3 g((unsigned)((p.M + RPB - 1) / RPB)), b(NT);
  if (kind == 0) hipLaunchKernelGGL((block_norm_kernel<0, TPR, MAXC>), g, b, 0, st, p);
  else hipLaunchKernelGGL((block_norm_kernel<1, TPR, MAXC>), g, b, 0, st, p);
}

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs& p, int kind, hipStream_t st) {
  if (p.M == 0 || p.K == 0) return hipSuccess;
  if (p.K <= 2048) launch_rows<64, 4>(p, kind, st);
  else if (p.K <= 4096) launch_rows<256, 2>(p, kind, st);
  else if (p.K <= 8192) launch_rows<512, 2>(p, kind, st);
  else if (p.K <= 16384) launch_rows<1024, 2>(p, kind, st);
  else launch_rows<1024, 4>(p, kind, st);
  return hipGetLastError();
}

hipError_t launch_silu_mx(const void* G, const void* U, int64_t M, int64_t N, int64_t ldg, int64_t ldu,
                          int fmt, void* codes, uint8_t* scales, hipStream_t st) {
  const int64_t total = M * (((N + 127) >> 7) << 4);
  if (total == 0) return hipSuccess;
  const dim3 gr((unsigned)((total + 255) / 256)), b(256);
  const uint16_t *g = static_cast<const uint16_t*>(G), *u = static_cast<const uint16_t*>(U);
  uint8_t* q = static_cast<uint8_t*>(codes);
  if (fmt == kActMxFp4) hipLaunchKernelGGL(silu_mx_kernel<true>, gr, b, 0, st, g, u, M, N, ldg, ldu, q, scales);
  else hipLaunchKernelGGL(silu_mx_kernel<false>, gr, b, 0, st, g, u, M, N, ldg, ldu, q, scales);
  return hipGetLastError();
}

}  // namespace qr
