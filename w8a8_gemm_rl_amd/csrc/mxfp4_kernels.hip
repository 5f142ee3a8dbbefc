// Microscaled 4-bit floating point (MXFP4) for gfx950: quantization of weights and
// tokens, values back from codes, and the product with MXFP4 weights. Formats and
// the layout of scales: qr_mx.h.
//
//   Y[m,n] = sum_b 2^(Xx[m,b] + Xw[n,b]) sum_{k in block b} x[m,k] w[n,k]
//
// runs on v_mfma_scale_f32_16x16x128_f8f6f4 with weights on operand A (E2M1) and
// tokens on operand B (E2M1 or E4M3). Operand layouts (measured): lane l holds row
// l % 16; with g = l / 16, E2M1: elements [32 g, 32 g + 32) of the 128, 16 bytes;
// E4M3: elements [16 g, 16 g + 16) and [64 + 16 g, 64 + 16 g + 16); in both the
// lane's scale byte is that of block g. Register i of the result is weight row
// 4 g + i, token l % 16.
#include "qr_internal.h"
#include "qr_mx.h"

namespace qr {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

// One chunk of eight values per lane, four lanes a block; 256 chunks per block of
// threads, rows padded to whole 16-chunk panels so that lanes keep their place.
template <bool FP4, bool BF16>
__global__ __launch_bounds__(256) void mx4_quant_kernel(const void* __restrict__ A, int64_t R,
                                                        int64_t K, int64_t lda,
                                                        uint8_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales) {
  const int64_t cpr = ((K + 127) >> 7) << 4;  // chunks per row, padded
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = idx / cpr, c = idx - row * cpr;
  const bool live = row < R && 8 * c < K;
  float v[8] = {};
  if (live) {
    if constexpr (BF16) {
      bf16x8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(A) + row * lda + 8 * c), v);
    } else {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(A) + row * lda + 8 * c);
      const float4 a = p[0], b = p[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  }
  mx_store_row8<FP4>(v, live, row, R, c, K, codes, scales);
}

// Eight values per lane from their codes and the block's scale byte.
template <bool FP4, bool BF16>
__global__ __launch_bounds__(256) void mx_dequant_kernel(const uint8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales,
                                                         int64_t R, int64_t K, void* __restrict__ out,
                                                         int64_t ldo) {
  const int64_t cpr = K >> 3;
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (idx >= R * cpr) return;
  const int64_t row = idx / cpr, c = idx - row * cpr;
  const int64_t b = c >> 2;
  const float s = mx_scale_value(scales[((b >> 2) * R + row) * 4 + (b & 3)]);
  float v[8];
  if constexpr (FP4) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + row * (K >> 1) + 4 * c);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // |v| = m / 2 for codes 0 and 1, else (1 + m / 2) 2^(e - 1)
      const uint32_t q = (w >> (4 * e)) & 15u, ex = (q >> 1) & 3u, m = q & 1u;
      const uint32_t mag = ex == 0u ? (m ? 0x3f000000u : 0u) : ((ex + 126u) << 23) | (m << 22);
      v[e] = __uint_as_float(mag | ((q & 8u) << 28)) * s;
    }
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(codes + row * K + 8 * c);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t q = (e < 4 ? w.x >> (8 * e) : w.y >> (8 * (e - 4))) & 255u;
      const uint32_t ex = (q >> 3) & 15u, m = q & 7u;
      const float mag = ex == 0u ? (float)m * 0x1p-9f : __uint_as_float(((ex + 120u) << 23) | (m << 20));
      v[e] = ((q & 127u) == 127u ? __uint_as_float(0x7fc00000u) : ((q & 128u) ? -mag : mag)) * s;
    }
  }
  if constexpr (BF16) {
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = f32_to_bf16_any(v[e]);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + row * ldo + 8 * c) =
        make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
  } else {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + row * ldo + 8 * c);
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

struct Mx4Params {
  const uint8_t* Xq;
  const uint8_t* sx;
  const uint8_t* Wq;
  const uint8_t* sw;
  int64_t M, N, K;
  void* Y;
  int64_t ldy;
  int out_raw;
};

// Store of a lane's four consecutive output channels of one token.
__device__ __forceinline__ void mx4_store4(const Mx4Params& p, int64_t m, int64_t n, const float* a) {
  if (m >= p.M || n >= p.N) return;
  const bool full = n + 3 < p.N && (p.ldy & 3) == 0;
  if (p.out_raw) {
    float* y = static_cast<float*>(p.Y) + m * p.ldy + n;
    if (full) *reinterpret_cast<float4*>(y) = make_float4(a[0], a[1], a[2], a[3]);
    else
      for (int r = 0; r < 4 && n + r < p.N; ++r) y[r] = a[r];
  } else {
    uint32_t b[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) b[r] = f32_to_bf16_any(a[r]);
    uint16_t* y = static_cast<uint16_t*>(p.Y) + m * p.ldy + n;
    if (full) *reinterpret_cast<uint2*>(y) = make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
    else
      for (int r = 0; r < 4 && n + r < p.N; ++r) y[r] = (uint16_t)b[r];
  }
}

// A block owns 16 weight rows x 16 tokens; its 8 waves take the 128-element panels
// of K in turn (operands straight from memory to registers), and the waves' partial
// sums are added in a fixed order.
template <bool XFP4>
__global__ __launch_bounds__(512) void mx4_stream_kernel(const Mx4Params p) {
  __shared__ float4 red[8][64];
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int64_t tiles_m = (p.M + 15) >> 4;
  const int64_t tn = blockIdx.x / tiles_m, tm = blockIdx.x % tiles_m;
  const int64_t n = tn * 16 + r < p.N ? tn * 16 + r : p.N - 1;
  const int64_t m = tm * 16 + r < p.M ? tm * 16 + r : p.M - 1;
  const uint8_t* wr = p.Wq + n * (p.K >> 1) + 16 * g;
  const uint8_t* xr = p.Xq + (XFP4 ? m * (p.K >> 1) : m * p.K) + 16 * g;
  v4f acc = {};
  const int64_t np = p.K >> 7;
  for (int64_t k = wid; k < np; k += 8) {
    const uint4 a = *reinterpret_cast<const uint4*>(wr + k * 64);
    const int ea = p.sw[(k * p.N + n) * 4 + g];
    const int eb = p.sx[(k * p.M + m) * 4 + g];
    const v8i A = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    if constexpr (XFP4) {
      const uint4 b = *reinterpret_cast<const uint4*>(xr + k * 64);
      const v8i B = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, acc, 4, 4, 0, ea, 0, eb);
    } else {
      const uint4 b = *reinterpret_cast<const uint4*>(xr + k * 128);
      const uint4 c = *reinterpret_cast<const uint4*>(xr + k * 128 + 64);
      const v8i B = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, (int)c.x, (int)c.y, (int)c.z, (int)c.w};
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, acc, 4, 0, 0, ea, 0, eb);
    }
  }
  red[wid][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
  __syncthreads();
  if (wid != 0) return;
  float s[4] = {};
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const float4 v = red[w][lane];
    s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
  }
  mx4_store4(p, tm * 16 + r, tn * 16 + 4 * g, s);
}

}  // namespace

hipError_t launch_mx4_quant(const void* A, int64_t R, int64_t K, int64_t lda, int bf16, int fmt,
                            void* codes, uint8_t* scales, hipStream_t st) {
  const int64_t total = R * (((K + 127) >> 7) << 4);
  if (total == 0) return hipSuccess;
  const dim3 g((unsigned)((total + 255) / 256)), b(256);
  uint8_t* q = static_cast<uint8_t*>(codes);
  if (fmt == kActMxFp4) {
    if (bf16) hipLaunchKernelGGL((mx4_quant_kernel<true, true>), g, b, 0, st, A, R, K, lda, q, scales);
    else hipLaunchKernelGGL((mx4_quant_kernel<true, false>), g, b, 0, st, A, R, K, lda, q, scales);
  } else {
    if (bf16) hipLaunchKernelGGL((mx4_quant_kernel<false, true>), g, b, 0, st, A, R, K, lda, q, scales);
    else hipLaunchKernelGGL((mx4_quant_kernel<false, false>), g, b, 0, st, A, R, K, lda, q, scales);
  }
  return hipGetLastError();
}

hipError_t launch_mx_dequant(const void* codes, const uint8_t* scales, int64_t R, int64_t K, int fmt,
                             void* out, int64_t ldo, int bf16, hipStream_t st) {
  const int64_t total = R * (K >> 3);
  if (total == 0) return hipSuccess;
  const dim3 g((unsigned)((total + 255) / 256)), b(256);
  const uint8_t* q = static_cast<const uint8_t*>(codes);
  if (fmt == kActMxFp4) {
    if (bf16) hipLaunchKernelGGL((mx_dequant_kernel<true, true>), g, b, 0, st, q, scales, R, K, out, ldo);
    else hipLaunchKernelGGL((mx_dequant_kernel<true, false>), g, b, 0, st, q, scales, R, K, out, ldo);
  } else {
    if (bf16) hipLaunchKernelGGL((mx_dequant_kernel<false, true>), g, b, 0, st, q, scales, R, K, out, ldo);
    else hipLaunchKernelGGL((mx_dequant_kernel<false, false>), g, b, 0, st, q, scales, R, K, out, ldo);
  }
  return hipGetLastError();
}

hipError_t launch_mx4_gemm(const void* Xq, const uint8_t* sx, int xfmt, const void* Wq,
                           const uint8_t* sw, int64_t M, int64_t N, int64_t K, int out_raw, void* Y,
                           int64_t ldy, void* /*ws*/, hipStream_t st) {
  if (M == 0 || N == 0) return hipSuccess;
  const Mx4Params p{static_cast<const uint8_t*>(Xq), sx, static_cast<const uint8_t*>(Wq), sw,
                    M, N, K, Y, ldy, out_raw};
  const dim3 g((unsigned)(((N + 15) / 16) * ((M + 15) / 16))), b(512);
  if (xfmt == kActMxFp4) hipLaunchKernelGGL(mx4_stream_kernel<true>, g, b, 0, st, p);
  else hipLaunchKernelGGL(mx4_stream_kernel<false>, g, b, 0, st, p);
  return hipGetLastError();
}

size_t mx4_gemm_ws_bytes(int64_t, int64_t, int64_t, int) { return 0; }

// The workspace holds the token codes, then their scales (each 256-byte aligned).
hipError_t launch_mx4_linear(const void* X, int64_t ldx, int xfmt, const void* Wq, const uint8_t* sw,
                             int64_t M, int64_t N, int64_t K, void* Y, int64_t ldy, void* ws,
                             hipStream_t st) {
  if (M == 0 || N == 0) return hipSuccess;
  const size_t cb = (size_t)(xfmt == kActMxFp4 ? M * (K >> 1) : M * K);
  uint8_t* xq = static_cast<uint8_t*>(ws);
  uint8_t* sx = xq + ((cb + 255) & ~(size_t)255);
  const hipError_t e = launch_mx4_quant(X, M, K, ldx, 1, xfmt, xq, sx, st);
  if (e != hipSuccess) return e;
  return launch_mx4_gemm(xq, sx, xfmt, Wq, sw, M, N, K, 0, Y, ldy, nullptr, st);
}

}  // namespace qr
