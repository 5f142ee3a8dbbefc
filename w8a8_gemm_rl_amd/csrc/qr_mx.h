// Block-scaled (microscaled) formats: device helpers shared by the kernels that
// write or read 32-element blocks with one power-of-two scale.
//
//   E2M1   S.EE.M, bias 1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives; two to
//          a byte, element 2 i in the low half.
//   E4M3   as in qr_device.h, a byte each.
//   scale  byte X + 127 for 2^X (E8M0), 255 for a block that holds a NaN or an
//          infinity. X is the smallest integer in [-127, 127] with
//          max |v| <= top 2^X (top = 6 or 448), so no element is clipped.
//
// Scale bytes lie in panels of 128 elements of K, [ceil(K / 128)][rows][4].
#pragma once

#include "qr_device.h"

namespace qr {

// Formats of token codes (the header's QR_ACT_*).
constexpr int kActInt8 = 0, kActFp8 = 1, kActMxFp8 = 2, kActMxFp4 = 3, kActBf16 = 4;

// Scale byte of a block from the bits of max |v| (sign cleared). amax = 1.m 2^(E - 127);
// 6 = 1.5 2^2 and 448 = 1.75 2^8, so X + 127 is E - 2 (E - 8), one more where the
// mantissa exceeds top's. Integers only: subnormal and zero blocks give 0 (X = -127).
template <bool FP4>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t abits) {
  if (abits >= 0x7f800000u) return 255u;
  const int s = (int)(abits >> 23) - (FP4 ? 2 : 8) +
                ((abits & 0x7fffffu) > (FP4 ? 0x400000u : 0x600000u) ? 1 : 0);
  return (uint32_t)(s < 0 ? 0 : s);
}

// 2^-X for a scale byte other than 255 (a normal fp32: the byte is at most 253).
// Products with it are exact unless they fall below fp32's normal range, far under
// half of the formats' smallest step.
__device__ __forceinline__ float mx_inv_scale(uint32_t sb) {
  return __uint_as_float((254u - sb) << 23);
}

// 2^X (byte 0 is the subnormal 2^-127), NaN for byte 255.
__device__ __forceinline__ float mx_scale_value(uint32_t sb) {
  return __uint_as_float(sb == 0u ? 0x400000u : (sb == 255u ? 0x7fc00000u : sb << 23));
}

// Eight E2M1 codes of values already divided by the scale (|v| <= 6), packed low
// half first; v_cvt_scalef32_pk_fp4_f32 rounds to nearest, ties to even, and keeps
// the sign of values that round to zero.
__device__ __forceinline__ uint32_t mx_fp4_codes8(const float* v) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], 1.0f, 3);
  return w;
}

__device__ __forceinline__ uint2 mx_fp8_codes8(const float* v) {
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}

__device__ __forceinline__ uint32_t abs_bits_max8(const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t a = __float_as_uint(v[e]) & 0x7fffffffu;
    m = a > m ? a : m;
  }
  return m;
}

// Bits of max |v| and the scale byte of the 32-element block that lanes 4 j .. 4 j + 3
// hold, eight values each (every lane of the four gets them). Integer maximum of the sign-cleared bits:
// the order of non-negative floats, with NaN above infinity above every number.
__device__ __forceinline__ uint32_t mx_block_max(const float* v) {
  uint32_t m = abs_bits_max8(v);
  uint32_t o = (uint32_t)__shfl_xor((int)m, 1, 64);
  m = o > m ? o : m;
  o = (uint32_t)__shfl_xor((int)m, 2, 64);
  return o > m ? o : m;
}

template <bool FP4>
__device__ __forceinline__ uint32_t mx_block_scale(const float* v) {
  return mx_scale_byte<FP4>(mx_block_max(v));
}

// Codes of eight values times inv.
template <bool FP4>
__device__ __forceinline__ uint2 mx_codes8_times(const float* v, float inv) {
  float t[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) t[e] = v[e] * inv;
  if constexpr (FP4) return make_uint2(mx_fp4_codes8(t), 0u);
  else return mx_fp8_codes8(t);
}

// Codes of eight values of a block with scale byte sb (zero codes in a NaN block).
template <bool FP4>
__device__ __forceinline__ uint2 mx_codes8(const float* v, uint32_t sb) {
  if (sb == 255u) return make_uint2(0u, 0u);
  return mx_codes8_times<FP4>(v, mx_inv_scale(sb));
}

// Stores the codes and scale bytes of a row when every lane holds those of eight
// consecutive values: chunk c (values 8 c .. 8 c + 7) of row `row`, c ascending with
// the lane and c % 16 == lane % 16. `live` lanes hold values (whole blocks of 32),
// the others zeros. A panel's four scale bytes are stored as one word; the bytes of a
// last panel that no block owns come out zero.
template <bool FP4>
__device__ __forceinline__ void mx_store_codes8(uint2 q, uint32_t sb, bool live, int64_t row, int64_t R,
                                                int64_t c, int64_t K, uint8_t* codes, uint8_t* scales) {
  const int lane = threadIdx.x & 63;
  uint32_t w = sb << (8 * ((lane >> 2) & 3));
  w |= (uint32_t)__shfl_xor((int)w, 4, 64);
  w |= (uint32_t)__shfl_xor((int)w, 8, 64);
  if (!live) return;
  if constexpr (FP4) *reinterpret_cast<uint32_t*>(codes + row * (K >> 1) + 4 * c) = q.x;
  else *reinterpret_cast<uint2*>(codes + row * K + 8 * c) = q;
  if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(scales + ((c >> 4) * R + row) * 4) = w;
}

// The same from the lanes' values.
template <bool FP4>
__device__ __forceinline__ void mx_store_row8(const float* v, bool live, int64_t row, int64_t R,
                                              int64_t c, int64_t K, uint8_t* codes, uint8_t* scales) {
  const uint32_t sb = mx_block_scale<FP4>(v);
  mx_store_codes8<FP4>(mx_codes8<FP4>(v, sb), sb, live, row, R, c, K, codes, scales);
}

// Elementwise passes over rows of 16-byte-aligned chunks of eight values: a block of 256
// threads takes U * 256 consecutive chunks (lane order = chunk order, a thread's chunks
// 256 apart), rows counting `cpr` chunks. Blocks are numbered so that an XCD takes a
// contiguous range: neighbouring rows' scale bytes share lines.
struct ChunkWalk {
  uint32_t rows, cpr;     // rows of this launch, chunks per row; rows * cpr < 2^31
  uint32_t magic, shift;  // i / cpr = mulhi(i, magic) >> shift for i < 2^31
  // With 2^(s-1) < cpr <= 2^s, magic = floor(2^(31+s) / cpr) + 1 exceeds 2^(31+s) / cpr by
  // at most 1, so i magic / 2^(31+s) exceeds i / cpr by less than 1 / cpr.
  static ChunkWalk of(int64_t rows, int64_t cpr) {  // cpr >= 2
    uint32_t s = 1;
    while (((int64_t)1 << s) < cpr) ++s;
    return {(uint32_t)rows, (uint32_t)cpr, (uint32_t)(((uint64_t)1 << (31 + s)) / (uint64_t)cpr + 1), s - 1};
  }
  __device__ __forceinline__ uint32_t row(uint32_t i) const { return __umulhi(i, magic) >> shift; }
  __device__ __forceinline__ uint32_t first(int u) const {
    const uint32_t g8 = gridDim.x & ~7u, b = blockIdx.x;
    const uint32_t blk = b < g8 ? (b & 7u) * (g8 >> 3) + (b >> 3) : b;
    return (blk * (uint32_t)u) * 256u + threadIdx.x;
  }
};

// Host: launches `launch(row0, walk, grid)` over row ranges of at most 2^30 chunks.
template <typename F>
hipError_t chunk_launches(int64_t rows, int64_t cpr, int u, const F& launch) {
  if (rows == 0 || cpr == 0) return hipSuccess;
  const int64_t step = ((int64_t)1 << 30) / cpr > 0 ? ((int64_t)1 << 30) / cpr : 1;
  for (int64_t r = 0; r < rows; r += step) {
    const int64_t n = rows - r < step ? rows - r : step;
    launch(r, ChunkWalk::of(n, cpr), dim3((unsigned)((n * cpr + u * 256 - 1) / (u * 256))));
  }
  return hipGetLastError();
}

// fp32 -> bf16 bits, round to nearest even; NaN stays NaN.
__device__ __forceinline__ uint32_t f32_to_bf16_any(float f) {
  const uint32_t u = __float_as_uint(f);
  return (u & 0x7fffffffu) > 0x7f800000u ? ((u >> 16) | 0x40u) : f32_to_bf16_rne(f);
}

// Two fp32 -> packed bf16 (a low), v_cvt_pk_bf16_f32: nearest even, NaN stays NaN.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 h2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{a, b}), h2));
}

__device__ __forceinline__ void bf16x8(const uint4 v, float* h) {
  h[0] = bf16_lo(v.x); h[1] = bf16_hi(v.x); h[2] = bf16_lo(v.y); h[3] = bf16_hi(v.y);
  h[4] = bf16_lo(v.z); h[5] = bf16_hi(v.z); h[6] = bf16_lo(v.w); h[7] = bf16_hi(v.w);
}

}  // namespace qr
