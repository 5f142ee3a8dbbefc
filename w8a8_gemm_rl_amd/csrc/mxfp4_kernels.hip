// Microscaled 4-bit floating point (MXFP4) for gfx950: quantization of weights and
// tokens, values back from codes, and the product with MXFP4 weights. Formats and
// the layout of scales: qr_mx.h.
//
//   Y[m,n] = sum_b 2^(Xx[m,b] + Xw[n,b]) sum_{k in block b} x[m,k] w[n,k]
//
// runs on v_mfma_scale_f32_16x16x128_f8f6f4 and v_mfma_scale_f32_32x32x64_f8f6f4 with
// weights on operand A (E2M1) and tokens on operand B (E2M1 or E4M3). Operand layouts of
// the T x T x KI instruction (measured): lane l holds row l % T; with g = l / T, E2M1:
// elements [32 g, 32 g + 32) of the KI, 16 bytes; E4M3: elements [16 g, 16 g + 16) and
// [KI / 2 + 16 g, KI / 2 + 16 g + 16); in both the lane's scale byte is that of block g.
// Register 4 q + r of the result is weight row 8 q + 4 g + r, token l % T. On operands that
// stay in registers E2M1 x E2M1 reaches 6.6 - 7.1 PFLOP/s, E2M1 x E4M3 4.0.
#include <type_traits>

#include "qr_copy.h"
#include "qr_internal.h"
#include "qr_mx.h"

namespace qr {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));

// Rows [row0, row0 + w.rows) of A, eight values a thread, four lanes a block of 32; rows
// padded to whole panels of 16 chunks so that lanes keep their place in a block (pad chunks
// hold zeros). One pass, bound by memory: the 7B gate's fp32 master weights, 308 MB in and
// out, take 56 us (5.5 TB/s; 60 with two chunks a thread); 256 bf16 tokens of 3584 values
// take no longer than a launch (2.9 us back to back). The weights are read once and not
// again soon, hence the non-temporal loads.
template <bool FP4, bool BF16>
__global__ __launch_bounds__(256) void mx4_quant_kernel(const void* __restrict__ A, int64_t R,
                                                        int64_t K, int64_t lda,
                                                        uint8_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales, int64_t row0,
                                                        ChunkWalk w) {
  typedef float f4 __attribute__((ext_vector_type(4)));
  const uint32_t i = w.first(1), r = w.row(i), c = i - r * w.cpr;
  const int64_t row = row0 + r;
  const bool live = i < w.rows * w.cpr && c < (uint32_t)(K >> 3);
  float v[8] = {};
  if (live) {
    if constexpr (BF16) {
      bf16x8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(A) + row * lda + 8 * c), v);
    } else {
      const f4* p = reinterpret_cast<const f4*>(static_cast<const float*>(A) + row * lda + 8 * c);
      const f4 a = __builtin_nontemporal_load(p), b = __builtin_nontemporal_load(p + 1);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = a[e];
        v[4 + e] = b[e];
      }
    }
  }
  mx_store_row8<FP4>(v, live, row, R, c, K, codes, scales);
}

// Eight values from their codes (q: four or eight bytes) and their block's scale byte.
template <bool FP4>
__device__ __forceinline__ void mx_values8(const uint2 q, uint32_t sb, float* v) {
  const float s = mx_scale_value(sb);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (FP4) {
      // |v| = m / 2 for codes 0 and 1, else (1 + m / 2) 2^(ex - 1)
      const uint32_t x = (q.x >> (4 * e)) & 15u, ex = (x >> 1) & 3u, m = x & 1u;
      const uint32_t mag = ex == 0u ? (m ? 0x3f000000u : 0u) : ((ex + 126u) << 23) | (m << 22);
      v[e] = __uint_as_float(mag | ((x & 8u) << 28)) * s;
    } else {
      const uint32_t x = (e < 4 ? q.x >> (8 * e) : q.y >> (8 * (e - 4))) & 255u;
      const uint32_t ex = (x >> 3) & 15u, m = x & 7u;
      const float mag = ex == 0u ? (float)m * 0x1p-9f : __uint_as_float(((ex + 120u) << 23) | (m << 20));
      v[e] = ((x & 127u) == 127u ? __uint_as_float(0x7fc00000u) : ((x & 128u) ? -mag : mag)) * s;
    }
  }
}

// Values of rows [row0, row0 + w.rows), two chunks of eight a thread (18944 x 3584 to bf16:
// 28.4 us from E2M1, 31.9 from E4M3, 6.1 and 6.4 TB/s; one or four chunks a thread cost 2 us
// more). NT: bf16 values past the L2s' 32 MB leave non-temporally (1.2 - 1.5 us more otherwise; 1001
// x 27648 12.9 against 15.3); fewer stay there for whoever reads them. A chunk of fp32 values is
// two stores of half a 32-byte piece each, which non-temporally reach memory as such (18944 x 3584
// 108 us from E2M1 against 79, 4096 x 5120 33 against 23): those leave as ordinary stores.
template <bool FP4, bool BF16, bool NT>
__global__ __launch_bounds__(256) void mx_dequant_kernel(const uint8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales,
                                                         int64_t R, int64_t K, void* __restrict__ out,
                                                         int64_t ldo, int64_t row0, ChunkWalk w) {
  constexpr int U = 2;
  const uint32_t total = w.rows * w.cpr, i0 = w.first(U);
  uint2 q[U];
  uint32_t sb[U], c[U];
  int64_t row[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = i0 + u * 256u, ii = i < total ? i : total - 1, r = w.row(ii);
    row[u] = row0 + r;
    c[u] = ii - r * w.cpr;
    q[u].y = 0u;
    if constexpr (FP4) q[u].x = *reinterpret_cast<const uint32_t*>(codes + row[u] * (K >> 1) + 4 * c[u]);
    else q[u] = *reinterpret_cast<const uint2*>(codes + row[u] * K + 8 * c[u]);
    sb[u] = scales[((int64_t)(c[u] >> 4) * R + row[u]) * 4 + ((c[u] >> 2) & 3u)];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (i0 + u * 256u >= total) break;
    float v[8];
    mx_values8<FP4>(q[u], sb[u], v);
    if constexpr (BF16) {
      typedef uint32_t u4 __attribute__((ext_vector_type(4)));
      const u4 b = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
      u4* o = reinterpret_cast<u4*>(static_cast<uint16_t*>(out) + row[u] * ldo + 8 * c[u]);
      if constexpr (NT) __builtin_nontemporal_store(b, o);
      else *o = b;
    } else {
      static_assert(!NT, "half pieces");
      v4f* o = reinterpret_cast<v4f*>(static_cast<float*>(out) + row[u] * ldo + 8 * c[u]);
      o[0] = v4f{v[0], v[1], v[2], v[3]};
      o[1] = v4f{v[4], v[5], v[6], v[7]};
    }
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

// Store of a lane's four consecutive output channels n .. n + 3 (n a multiple of 4) of
// one token.
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

// Few tokens: a weight stream, bound by the time to get it going and then by memory (one
// token, fused: 7B QKV, 8.8 MB of weights and scales, 5.7 us; 7B down, 36 MB, 10.4 us, 3.5
// TB/s; an empty kernel 2.6 us). A block owns 16 weight rows and up to 16 tokens; its NW
// waves take the 256-element pairs of panels of K in turn (a row's pair is one 128-byte
// line), weights straight from memory to registers with D pairs a wave in flight, and
// the waves' partial sums are added in a fixed order. FUSED: the block first quantizes
// the bf16 tokens into LDS itself (the first weights are on their way meanwhile), else
// token codes are read from memory like the weights.
template <bool XFP4, bool FUSED, int NW, int KW, int D>
__global__ __launch_bounds__(64 * NW) void mx4_decode_kernel(const Mx4Params p,
                                                             const uint16_t* __restrict__ X,
                                                             int64_t ldx) {
  extern __shared__ __attribute__((aligned(16))) uint8_t xs[];  // FUSED: codes, then scales
  __shared__ float4 red[KW > 1 ? NW : 1][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wid = wave % KW;  // the wave's part of K
  const int r = lane & 15, g = lane >> 4;
  const int M = (int)p.M, K = (int)p.K, np = K >> 7, npair = (np + 1) >> 1;
  const int64_t n0 = ((int64_t)blockIdx.x * (NW / KW) + wave / KW) * 16;
  const int64_t n = n0 + r < p.N ? n0 + r : p.N - 1;  // rows past N repeat the last, unstored
  const int m = r < M ? r : M - 1;
  const int rb = XFP4 ? K >> 1 : K;
  const uint8_t* wr = p.Wq + n * (K >> 1) + 16 * g;
  const uint8_t* ws = p.sw + n * 4 + g;

  uint4 a[D][2];
  int ea[D][2];
  auto load = [&](int d, int pair) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int k = 2 * pair + e;
      if (k < np) {
        a[d][e] = *reinterpret_cast<const uint4*>(wr + k * 64);
        ea[d][e] = ws[(int64_t)k * p.N * 4];
      }
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (wid + d * KW < npair) load(d, wid + d * KW);

  if constexpr (FUSED) {
    // eight values a thread, four threads a block of 32; XC loads a thread at once
    constexpr int XC = 4;
    const int cpr = K >> 3, total = M * cpr;
    uint8_t* xsc = xs + M * rb;
    for (int c0 = threadIdx.x; c0 < (total + 63) / 64 * 64; c0 += XC * 64 * NW) {
      uint4 x[XC];
#pragma unroll
      for (int u = 0; u < XC; ++u) {
        const int c = c0 + u * 64 * NW, t = M == 1 ? 0 : c / cpr;
        x[u] = make_uint4(0u, 0u, 0u, 0u);
        if (c < total) x[u] = *reinterpret_cast<const uint4*>(X + t * ldx + 8 * (c - t * cpr));
      }
#pragma unroll
      for (int u = 0; u < XC; ++u) {
        const int c = c0 + u * 64 * NW, t = M == 1 ? 0 : c / cpr, q = c - t * cpr;
        float v[8];
        bf16x8(x[u], v);
        const uint32_t sb = mx_block_scale<XFP4>(v);
        if (c < total) {
          const uint2 w = mx_codes8<XFP4>(v, sb);
          if constexpr (XFP4) *reinterpret_cast<uint32_t*>(xs + t * rb + 4 * q) = w.x;
          else *reinterpret_cast<uint2*>(xs + t * rb + 8 * q) = w;
          if ((q & 3) == 0) xsc[t * (K >> 5) + (q >> 2)] = (uint8_t)sb;
        }
      }
    }
    __syncthreads();
  }
  const uint8_t* xr = (FUSED ? xs : p.Xq) + (int64_t)m * rb + 16 * g;
  const uint8_t* xsc = FUSED ? xs + M * rb + m * (K >> 5) + g : p.sx + m * 4 + g;
  const int xstep = FUSED ? 4 : M * 4;

  v4f acc = {};
  for (int i = wid; i < npair; i += D * KW) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int pair = i + d * KW;
      if (pair >= npair) break;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int k = 2 * pair + e;
        if (k >= np) break;
        const uint4 w = a[d][e];
        const v8i A = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
        const int eb = xsc[(int64_t)k * xstep];
        if constexpr (XFP4) {
          const uint4 b = *reinterpret_cast<const uint4*>(xr + k * 64);
          const v8i B = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
          acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, acc, 4, 4, 0, ea[d][e], 0, eb);
        } else {
          const uint4 b = *reinterpret_cast<const uint4*>(xr + k * 128);
          const uint4 c = *reinterpret_cast<const uint4*>(xr + k * 128 + 64);
          const v8i B = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, (int)c.x, (int)c.y, (int)c.z, (int)c.w};
          acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, acc, 4, 0, 0, ea[d][e], 0, eb);
        }
      }
      if (pair + D * KW < npair) load(d, pair + D * KW);
    }
  }
  float s[4] = {acc[0], acc[1], acc[2], acc[3]};
  if constexpr (KW > 1) {
    red[wave][lane] = make_float4(s[0], s[1], s[2], s[3]);
    __syncthreads();
    if (wid != 0) return;
#pragma unroll
    for (int w = 1; w < KW; ++w) {
      const float4 v = red[wave + w][lane];
      s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
    }
  }
  mx4_store4(p, r, n0 + 4 * g, s);
}

// ---------------------------------------------------------------------------
// Tiled product: BN weight rows x BM tokens per block, a ring of S stages in LDS. A
// stage holds KS elements of K: weight rows (KS / 2 bytes each), token rows (KS / 2
// or KS bytes) and the scale bytes of both (4 per row and 128-element panel), moved
// global -> LDS by LDS-DMA copies (16 bytes a lane). The block's waves form a WN x WM
// grid, each owning BN / WN x BM / WM outputs as T x T fragments.
//
// LDS rows of 64 bytes are paired, so that every 128-byte line has eight 16-byte
// chunks; chunk q of line i sits at q ^ (i & 7) (rows of 128 bytes: i = r / 2, as for
// the 8-bit GEMMs), which spreads a fragment's reads over all banks. The swizzle is
// applied on the global side of the copies.
//
// Operands of a fragment's next K step are read from LDS while the matrix cores work
// on the current one, across the stage boundary too: the barrier that opens a stage
// stands before the last K step of the one before, whose operands are already in
// registers, so its slot can be refilled at once.
//
// A T = 32 fragment takes 64 elements per MFMA (T = 16: 128); lane l holds row l % T
// and, with g = l / T, E2M1 elements [32 g, 32 g + 32) or E4M3 elements [16 g, + 16)
// and [KI / 2 + 16 g, + 16), and the scale byte of block g of the KI elements. A
// lane's scale word (the panel's four bytes of its row) is shifted by 8 g, so that
// byte 0 (and for T = 32 byte 2 in the panel's second half) is the one it needs.
//
// Rows past N or M are copied as zeros and not stored. With splits > 1 a block takes one
// contiguous part of its tile's stages and writes fp32 partial sums, which
// mx4_sum_kernel adds in a fixed order.
//
// Stacked 7B gate and up, 75 MB of codes and scales in and out at 33 E4M3 tokens: 15.0 us,
// 5.0 TB/s, what a copy reaches. At 256 E2M1 tokens 93 MB take 26 us: 237 tiles of
// 160 x 256, one round (E4M3 tokens 35). The 32B gate at 4096 E2M1 tokens: 289 - 298 us, 3.9 -
// 4.0 PFLOP/s (two cards, call after call; 310 - 316 in the first dozen), with E4M3 tokens 424.
// There, on 256 x 256 tiles, 20 stages in seven rounds, the products alone take 160 us (the
// clock falls to 1.93 GHz), a fragment's LDS reads alone 164, the copies alone 193 (20 bytes
// a clock and CU; 127 from the L2), any two together 205, all three 250; the rest fills the ring
// and stores the outputs. Measured slower there: a third operand buffer with
// refills a step earlier, 64-byte rows with deeper rings, four waves of 128 x 128, wave
// priorities, non-temporal weight copies, other groupings of tiles.
//
// fp32 outputs and partial sums leave straight from the fragments, 16 bytes a lane (gate and
// up at 256 tokens 34 us with E2M1, 39 with E4M3; the 32B gate at 4096 about 400 and 520).
// ---------------------------------------------------------------------------
// One copy of LANES lanes' 16 bytes (a power of two), exec being all ones before and after.
// The wait state between the write of M0 and the copy (qr_copy.h) is an s_nop, or the write
// of exec.
template <int LANES>
__device__ __forceinline__ void dma_lanes(uint32_t lds_addr, uint32_t vo, __amdgpu_buffer_rsrc_t r) {
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
  if constexpr (LANES == 64)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 : : "s"(lds_addr), "v"(vo), "s"(r) : "memory", "m0");
  else
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_mov_b64 exec, %3\n\t"
        "buffer_load_dwordx4 %1, %2, 0 offen lds\n\t"
        "s_mov_b64 exec, -1"
        : : "s"(lds_addr), "v"(vo), "s"(r), "s"(((uint64_t)1 << (LANES & 63)) - 1) : "memory", "m0");
#pragma clang diagnostic pop
}

constexpr int kCUs = 256;

struct Mx4TileParams {
  Mx4Params g;
  float* part;
  int tiles_m, tiles_n, stages, splits;
  bool nt_out;  // non-temporal output stores
};

template <int T>
struct Mx4Mfma;
template <>
struct Mx4Mfma<16> {
  using acc_t = v4f;
  static constexpr int KI = 128;
  template <bool XFP4, int OP>
  static __device__ __forceinline__ acc_t run(v8i a, v8i b, acc_t c, int sa, int sb) {
    static_assert(OP == 0, "one step per panel");
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, XFP4 ? 4 : 0, 0, sa, 0, sb);
  }
};
template <>
struct Mx4Mfma<32> {
  using acc_t = v16f;
  static constexpr int KI = 64;
  template <bool XFP4, int OP>
  static __device__ __forceinline__ acc_t run(v8i a, v8i b, acc_t c, int sa, int sb) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, XFP4 ? 4 : 0, 2 * OP, sa, 2 * OP, sb);
  }
};

// Whether a slot of the ring can hold a token fragment of each wave's outputs.
template <bool XFP4, int T, int BN, int BM, int WN, int WM, int KS>
struct Mx4Ahead {
  static constexpr int NW = WN * WM, RA = KS / 2, RB = XFP4 ? KS / 2 : KS;
  static constexpr int IA = (BN * RA / 1024 + NW - 1) / NW * NW, IB = (BM * RB / 1024 + NW - 1) / NW * NW;
  static constexpr bool value = (IA + IB) * 1024 + KS / 128 * 2048 >= NW * T * (BN / WN * 2 + 16);
};

template <bool XFP4, int T, int BN, int BM, int WN, int WM, int S, int KS, bool AHEAD>
__global__ __launch_bounds__(64 * WN * WM, 1) void mx4_tile_kernel(const Mx4TileParams p) {
  using MF = Mx4Mfma<T>;
  using acc_t = typename MF::acc_t;
  constexpr int NW = WN * WM;
  constexpr int KI = MF::KI, NKK = KS / KI, PP = KS / 128;  // K steps, panels per stage
  constexpr int RA = KS / 2, RB = XFP4 ? KS / 2 : KS;       // bytes per row and stage
  constexpr int WTN = BN / WN, WTM = BM / WM, FN = WTN / T, FM = WTM / T;
  constexpr int IA = (BN * RA / 1024 + NW - 1) / NW * NW, IB = (BM * RB / 1024 + NW - 1) / NW * NW;
  constexpr int NA = IA / NW, NB = IB / NW, GA = (NA + 3) / 4, GB = (NB + 3) / 4;
  constexpr int CODES = (IA + IB) * 1024, STAGE = CODES + PP * 2048;
  constexpr int SL = 128 * PP / NW;  // lanes of a wave's scale copy
  constexpr int NI = NA + NB + 1;    // copies per wave and stage
  static_assert(RA == 64 || RA == 128, "weight rows of half a line or a line");
  static_assert(RB == 64 || RB == 128 || RB == 256, "token rows of half a line to two");
  static_assert(NKK % 2 == 0, "operand buffers alternate within a stage");
  static_assert(BN * RA % 1024 == 0 && BM * RB % 1024 == 0, "whole copies");
  static_assert(WTN % T == 0 && WTM % T == 0 && BN <= 256 && BM <= 256, "wave tile");
  static_assert(SL >= 1 && SL <= 64 && 64 % SL == 0, "one scale copy per wave");
  static_assert(S >= 2 && (S - 1) * NI <= 63 && S * STAGE <= 160 * 1024, "ring");

  __shared__ __attribute__((aligned(1024))) uint8_t smem[S * STAGE];

  const int64_t N = p.g.N, M = p.g.M, K = p.g.K;
  // An XCD takes one contiguous part of the tiles, each of its blocks every `step`-th of
  // that; groups of up to 8 token tiles share weight tiles.
  const int tiles = p.tiles_m * p.tiles_n, total = tiles * p.splits, xcd = blockIdx.x & 7;
  const int end = (int)((int64_t)total * (xcd + 1) / 8), step = gridDim.x >> 3;
  int cur = (int)((int64_t)total * xcd / 8) + (blockIdx.x >> 3);
  if (cur >= end) return;
  const int split = cur / tiles;  // blocks of several tiles: one split
  auto locate = [&](int b, int& tm, int& tn) {
    b -= split * tiles;
    const int m0 = b / (8 * p.tiles_n) * 8, gm = p.tiles_m - m0 < 8 ? p.tiles_m - m0 : 8;
    b -= m0 * p.tiles_n;
    tm = __builtin_amdgcn_readfirstlane(m0 + b % gm);
    tn = __builtin_amdgcn_readfirstlane(b / gm);
  };
  const int ks0 = __builtin_amdgcn_readfirstlane((int)((int64_t)p.stages * split / p.splits));
  const int nk = __builtin_amdgcn_readfirstlane((int)((int64_t)p.stages * (split + 1) / p.splits)) - ks0;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wid % WN, wm = wid / WN;
  constexpr uint32_t kBig = 0x80000000u;
  const int64_t ra = K >> 1, rb = XFP4 ? K >> 1 : K;  // bytes per row
  const uint32_t spw = (uint32_t)(N * 4), spx = (uint32_t)(M * 4);
  const uint32_t np = (uint32_t)(K >> 7);
  // What the copies read: buffers that begin at the tile's first rows and end with the
  // arrays, so that rows past them come as zeros.
  __amdgpu_buffer_rsrc_t rw, rx, rs;
  const bool sw_w = (wid * SL / 64 & 1) == 0;  // the wave copies weights' scales
  auto copy_from = [&](int tm, int tn) {
    auto part = [](const uint8_t* a, int64_t from, int64_t bytes) {
      return __builtin_amdgcn_make_buffer_rsrc((void*)(a + from), (short)0, (int)(uint32_t)(bytes - from), kBufWord3);
    };
    rw = part(p.g.Wq, tn * BN * ra, N * ra);
    rx = part(p.g.Xq, tm * BM * rb, M * rb);
    if (sw_w) rs = part(p.g.sw, tn * BN * 4, (int64_t)np * spw);
    else rs = part(p.g.sx, tm * BM * 4, (int64_t)np * spx);
  };

  // Copies: instruction i of an operand fills LDS lines 8 i .. 8 i + 7; lane l the
  // physical chunk l % 8 of line 8 i + l / 8.
  const int ll = lane >> 3, pc = lane & 7;
  auto place = [&](int i, int rowbytes, int& row, int& chunk) {
    const int line = i * 8 + ll;
    if (rowbytes == 256) {
      row = line >> 1;
      chunk = ((line & 1) << 3) | (pc ^ (row & 7));
    } else if (rowbytes == 128) {
      row = line;
      chunk = pc ^ ((line >> 1) & 7);
    } else {
      const int q = pc ^ (line & 7);
      row = 2 * line + (q >> 2);
      chunk = q & 3;
    }
  };
  uint32_t oa[NA], ob[NB];
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    int r, c;
    place(wid * NA + i, RA, r, c);
    oa[i] = (r < BN ? (uint32_t)(r * ra + c * 16) : kBig) - 1024u * (uint32_t)(i % 4);
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    int r, c;
    place(wid * NB + i, RB, r, c);
    ob[i] = (r < BM ? (uint32_t)(r * rb + c * 16) : kBig) - 1024u * (uint32_t)(i % 4);
  }
  // Scales: the 2 PP kilobytes of a stage (panel, then weights or tokens: four bytes of
  // each of 256 rows) are split over the waves, SL lanes' 16 bytes each. Words of rows
  // that are not the tile's belong to rows that are not stored, or are past the array:
  // zero.
  const int sp = wid * SL / 64, sl0 = wid * SL % 64;
  const uint32_t os = (uint32_t)(16 * (sl0 + lane));
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
  const uint32_t la0 = lds0 + (uint32_t)(wid * NA) * 1024u;
  const uint32_t lb0 = lds0 + (uint32_t)(IA + wid * NB) * 1024u;
  const uint32_t ls0 = lds0 + (uint32_t)CODES + (uint32_t)(wid * SL * 16);

  // K an odd multiple of 128: the second half of the last stage lies past the rows'
  // ends. Bit i: copy i's lane holds such a chunk.
  uint32_t past_a = 0, past_b = 0;
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    int r, c;
    place(wid * NA + i, RA, r, c);
    past_a |= (c * 32 >= RA ? 1u : 0u) << i;
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    int r, c;
    place(wid * NB + i, RB, r, c);
    past_b |= (c * 32 >= RB ? 1u : 0u) << i;
  }
  constexpr int NG = GA + GB + 1;  // copy groups of a stage: weights, tokens, scales
  auto issue_group = [&](int g, int slot, int ks) {
    const uint32_t so = (uint32_t)(slot * STAGE);
    if (g == NG - 1) {
      const uint32_t panel = (uint32_t)(ks * PP + (sp >> 1));
      const uint32_t vs = panel < np ? os + panel * (sw_w ? spw : spx) : kBig;
      dma_lanes<SL>(ls0 + so, vs, rs);
      return;
    }
    const bool tail = KS == 256 && (ks + 1) * KS > K;
    const bool isA = g < GA;
    const uint32_t past = tail ? (isA ? past_a : past_b) : 0u;
    const int i0 = (isA ? g : g - GA) * 4, n = isA ? NA : NB, cnt = n - i0 < 4 ? n - i0 : 4;
    const uint32_t base = (isA ? la0 : lb0) + so + (uint32_t)i0 * 1024u;
    const int soff = ks * (isA ? RA : RB);
    uint32_t vo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + e < n ? i0 + e : 0;
      vo[e] = isA ? oa[i < NA ? i : 0] : ob[i < NB ? i : 0];
      if (KS == 256) vo[e] = (past >> i) & 1u ? kBig - 1024u * (uint32_t)(i % 4) : vo[e];
    }
    if (cnt == 4) dma_group<4, false>(base, vo, isA ? rw : rx, soff);
    else if (cnt == 3) dma_group<3, false>(base, vo, isA ? rw : rx, soff);
    else if (cnt == 2) dma_group<2, false>(base, vo, isA ? rw : rx, soff);
    else dma_group<1, false>(base, vo, isA ? rw : rx, soff);
  };

  // Operand reads: byte of chunk c of the wave's first fragment row (rows lr, lr + T,
  // ... have the same swizzle, and are T rows' bytes apart). Chunks of one lane differ from
  // its first, lg, in higher bits only: their bytes are the first's, those bits flipped.
  const int lr = lane % T, lg = lane / T;
  auto at = [&](int row0, int c, int rowbytes) {
    if (rowbytes == 256) return (row0 + lr) * 256 + ((c & 8) << 4) + (((c & 7) ^ (lr & 7)) << 4);
    if (rowbytes == 128) return (row0 + lr) * 128 + ((c ^ ((lr >> 1) & 7)) << 4);
    return ((row0 + lr) >> 1) * 128 + ((((lr & 1) * 4 + c) ^ ((lr >> 1) & 7)) << 4);
  };
  const int xa0 = at(wn * WTN, lg, RA), xb0 = IA * 1024 + at(wm * WTM, lg, RB);
  const int xsa = CODES + (wn * WTN + lr) * 4, xsb = CODES + 1024 + (wm * WTM + lr) * 4, sh = 8 * lg;
  acc_t acc[FN][FM];
  v8i opa[2][FN], opb[2][FM];
  int sna[FN], snb[FM], sca[FN], scb[FM];  // scale words: as read, and shifted for use
  auto load_ops = [&](const uint8_t* st, int h, int buf) {
    const int panel = h * KI / 128;
    // chunk of the lane's first 16 bytes: 32 E2M1 elements, 16 E4M3
    const int xa = xa0 ^ (h * (KI / 32) << 4), xb = xb0 ^ (h * (XFP4 ? KI / 32 : KI / 16) << 4);
    const bool fresh = h * KI % 128 == 0;
#pragma unroll
    for (int i = 0; i < FN; ++i) {
      const uint4 u = *reinterpret_cast<const uint4*>(st + xa + i * T * RA);
      opa[buf][i] = v8i{(int)u.x, (int)u.y, (int)u.z, (int)u.w, 0, 0, 0, 0};
      if (fresh) sna[i] = *reinterpret_cast<const int*>(st + xsa + panel * 2048 + i * T * 4);
    }
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const uint4 u = *reinterpret_cast<const uint4*>(st + xb + j * T * RB);
      if constexpr (XFP4) {
        opb[buf][j] = v8i{(int)u.x, (int)u.y, (int)u.z, (int)u.w, 0, 0, 0, 0};
      } else {
        const uint4 w = *reinterpret_cast<const uint4*>(st + (xb ^ (KI / 32 << 4)) + j * T * RB);
        opb[buf][j] = v8i{(int)u.x, (int)u.y, (int)u.z, (int)u.w, (int)w.x, (int)w.y, (int)w.z, (int)w.w};
      }
      if (fresh) snb[j] = *reinterpret_cast<const int*>(st + xsb + panel * 2048 + j * T * 4);
    }
  };
  auto take_scales = [&]() {
#pragma unroll
    for (int i = 0; i < FN; ++i) sca[i] = sna[i] >> sh;
#pragma unroll
    for (int j = 0; j < FM; ++j) scb[j] = snb[j] >> sh;
  };
  auto multiply_row = [&](int h, int buf, int i) {
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      if (h * KI % 128 == 0)
        acc[i][j] = MF::template run<XFP4, 0>(opa[buf][i], opb[buf][j], acc[i][j], sca[i], scb[j]);
      else if constexpr (T == 32)
        acc[i][j] = MF::template run<XFP4, 1>(opa[buf][i], opb[buf][j], acc[i][j], sca[i], scb[j]);
    }
  };
  // Stage j opens when its copies have landed and no wave reads stage j - 1 any more;
  // the S - 2 stages behind it (S - 1 behind the first) may still be in flight. The
  // last step of stage j - 1 is multiplied after that. Each step is kept apart for the
  // scheduler, which would otherwise hold a whole stage's operands in registers.
  int cs = 0, it = 0, kc = 0;  // kc: stage that the next refill copies
  // one MFMA, then the reads that one covers
  auto interleave = [&]() {
    constexpr int NR = FN + FM * (XFP4 ? 1 : 2), NM = FN * FM;
#pragma unroll
    for (int q = 0; q < NM; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, (NR + NM - 1) / NM + 1, 0);
    }
  };
  auto steps = [&](auto refill, auto last) {
    const int ns = cs + 1 == S ? 0 : cs + 1;
#pragma unroll
    for (int h = 0; h < NKK; ++h) {
      const int buf = h & 1;
      if (h * KI % 128 == 0) take_scales();
      if (h + 1 < NKK) {
        load_ops(smem + cs * STAGE, h + 1, buf ^ 1);
#pragma unroll
        for (int i = 0; i < FN; ++i) multiply_row(h, buf, i);
        interleave();
      } else {
        if constexpr (!decltype(last)::value) {
          if constexpr (decltype(refill)::value) wait_vm<(S - 2) * NI>();
          else wait_stages<NI, S - 2>(nk - 2 - it);
          __syncthreads();
          load_ops(smem + ns * STAGE, 0, buf ^ 1);
          __builtin_amdgcn_sched_barrier(0);
        }
        // the copies of the refill between the products
#pragma unroll
        for (int i = 0; i < (FN > NG ? FN : NG); ++i) {
          if (i < FN) multiply_row(h, buf, i);
          if constexpr (decltype(refill)::value) {
            __builtin_amdgcn_sched_barrier(0);
            if (i < NG) issue_group(i, cs, kc);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (decltype(refill)::value) ++kc;
    cs = ns;
  };
  // Register 4 q + r of a fragment: weight row 8 q + 4 lg + r, token lr.
  constexpr int NQ = T == 16 ? 1 : 4;
  // bf16 outputs go through the ring, each wave its own part, so that a wave's stores run
  // along a token's row: 16 bytes a lane, or 4 or 2 where the row stride (and so the rows'
  // alignment) is no multiple of 8 or 2 channels. Rows of 16 bytes more than the wave's
  // channels spread the writes over the banks. With AHEAD a slot holds it, and the copies of
  // the block's next tile run meanwhile.
  constexpr int LD = WTN * 2 + 16;
  constexpr int FIT = (AHEAD ? 1 : S) * STAGE / NW / (T * LD), JC = FIT < FM ? FIT : FM;
  static_assert(JC >= 1, "a token fragment per wave fits");
  const int64_t n4 = (N + 3) & ~(int64_t)3;
  auto store = [&](int tm, int tn, uint8_t* stage) {
    int sl = lane;
    if constexpr (AHEAD) {  // what follows is not to occupy registers during the products
      asm volatile("" : "+v"(sl));
      sl &= 63;
    }
    const int lr = sl % T, lg = sl / T;
    const int64_t n0 = (int64_t)tn * BN;
    const int own = (int)(N - n0 < BN ? N - n0 : BN);
    if (!p.part && !p.g.out_raw) {
      uint8_t* so = stage + wid * (JC * T * LD);
      uint16_t* Y = static_cast<uint16_t*>(p.g.Y) + n0 + wn * WTN;
      const int64_t mw = (int64_t)tm * BM + wm * WTM, ldy = p.g.ldy;
      const int ow = own - wn * WTN;
      auto rows_out = [&](int j0, auto vec, auto nt) {
        constexpr int V = decltype(vec)::value, CPR = WTN / V, PIECES = JC * T * CPR;
        constexpr bool kWhole = 64 % CPR == 0;  // lanes keep their channels, rows go up in steps
        uint16_t* const first = Y + (mw + T * j0) * ldy + (kWhole ? (sl / CPR) * ldy : 0);
#pragma unroll V == 8 ? (PIECES + 63) / 64 : 4
        for (int k = 0; k < (PIECES + 63) / 64; ++k) {
          const int c = sl + 64 * k, ml = c / CPR, nl = V * (c % CPR);
          const int64_t m = mw + T * j0 + ml;
          if ((PIECES % 64 != 0 && c >= PIECES) || m >= M || nl >= ow || T * j0 + ml >= WTM) continue;
          const uint8_t* src = so + ml * LD + nl * 2;
          uint16_t* dst = first + (kWhole ? k * (64 / CPR) : ml) * ldy + nl;
          if constexpr (V == 8) {
            typedef uint32_t u4 __attribute__((ext_vector_type(4)));
            const u4 v = *reinterpret_cast<const u4*>(src);
            if (nl + 8 > ow) {
              for (int e = 0; nl + e < ow; ++e) dst[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
            } else if constexpr (decltype(nt)::value) {
              __builtin_nontemporal_store(v, reinterpret_cast<u4*>(dst));
            } else {
              *reinterpret_cast<u4*>(dst) = v;
            }
          } else if constexpr (V == 2) {
            const uint32_t v = *reinterpret_cast<const uint32_t*>(src);
            if (nl + 2 > ow) dst[0] = (uint16_t)v;
            else *reinterpret_cast<uint32_t*>(dst) = v;
          } else {
            dst[0] = *reinterpret_cast<const uint16_t*>(src);
          }
        }
      };
#pragma unroll
      for (int j0 = 0; j0 < FM; j0 += JC) {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
          for (int j = j0; j < FM && j < j0 + JC; ++j)
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
              const acc_t& v = acc[i][j];
              *reinterpret_cast<uint2*>(so + (T * (j - j0) + lr) * LD + (T * i + 8 * q + 4 * lg) * 2) =
                  make_uint2(bf16_pair(v[4 * q], v[4 * q + 1]), bf16_pair(v[4 * q + 2], v[4 * q + 3]));
            }
        // lanes read what others of the wave wrote: LDS accesses of a wave are in order
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        // (the branch on nt_out around the loop: around the store the two are merged, without nt)
        if ((ldy & 7) != 0) {
          if ((ldy & 1) == 0) rows_out(j0, std::integral_constant<int, 2>{}, std::false_type{});
          else rows_out(j0, std::integral_constant<int, 1>{}, std::false_type{});
        } else if (p.nt_out) {
          rows_out(j0, std::integral_constant<int, 8>{}, std::true_type{});
        } else {
          rows_out(j0, std::integral_constant<int, 8>{}, std::false_type{});
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        const int64_t m = (int64_t)tm * BM + wm * WTM + T * j + lr;
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          const int nl = wn * WTN + T * i + 8 * q + 4 * lg;
          if (m >= M || nl >= own) continue;
          const float a[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          if (p.part)
            *reinterpret_cast<float4*>(p.part + ((int64_t)split * M + m) * n4 + n0 + nl) =
                make_float4(a[0], a[1], a[2], a[3]);
          else
            mx4_store4(p.g, m, n0 + nl, a);
        }
      }
  };

  // The block's tiles. Copies run S stages ahead, and with AHEAD (nk >= S then) into the next
  // tile: its first S - 1 stages are on their way, or there, while this one's last is
  // multiplied and its outputs are stored from the slot of that last stage.
  int tm, tn;
  locate(cur, tm, tn);
  copy_from(tm, tn);
  kc = ks0;
#pragma unroll
  for (int s = 0; s < S; ++s)
    if (s < nk) {
#pragma unroll
      for (int g = 0; g < NG; ++g) issue_group(g, s, kc);
      ++kc;
    }
  if (nk > 0) wait_stages<NI, S - 1>(nk - 1);
  __syncthreads();
  for (;;) {
    const int next = cur + step;
    const bool more = AHEAD && next < end;
    int tm2 = 0, tn2 = 0;
    if (more) locate(next, tm2, tn2);
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[i][j] = acc_t{};
    uint8_t* last_slot = smem;
    if (nk > 0) {
      load_ops(smem + cs * STAGE, 0, 0);
      it = 0;
      const int refills = more ? nk - 1 : nk - S;
      for (; it < refills; ++it) {
        if (AHEAD && it == nk - S) {
          copy_from(tm2, tn2);
          kc = 0;
        }
        steps(std::true_type{}, std::false_type{});
      }
      for (; it < nk - 1; ++it) steps(std::false_type{}, std::false_type{});
      last_slot = smem + cs * STAGE;
      steps(std::false_type{}, std::true_type{});
    }
    if (more) wait_vm<(S - 2) * NI>();  // the next tile's first stage
    __syncthreads();
    store(tm, tn, AHEAD ? last_slot : smem);
    if (!more) break;
    __syncthreads();
#pragma unroll
    for (int g = 0; g < NG; ++g) issue_group(g, cs == 0 ? S - 1 : cs - 1, kc);
    ++kc;
    cur = next;
    tm = tm2;
    tn = tn2;
  }
}

// Sum of the K splits' partial sums ([splits][M][N up to a multiple of 4]), four
// channels a thread, in the order of the splits: 3 us and the partial sums' write and read,
// which the planner counts.
__global__ __launch_bounds__(256) void mx4_sum_kernel(const float* __restrict__ part, int splits,
                                                      const Mx4Params p) {
  const int64_t n4 = (p.N + 3) & ~(int64_t)3, q = n4 >> 2;
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (idx >= p.M * q) return;
  const int64_t m = idx / q, n = 4 * (idx - m * q);
  const float4* s = reinterpret_cast<const float4*>(part) + idx;
  float a[4] = {};
  for (int i = 0; i < splits; ++i) {
    const float4 v = s[(int64_t)i * p.M * q];
    a[0] += v.x; a[1] += v.y; a[2] += v.z; a[3] += v.w;
  }
  mx4_store4(p, m, n, a);
}

// Whether a product of `tiles` tiles takes one block a CU, each for every so many-th tile of
// its XCD with copies running ahead, rather than a block a tile: where they fill more than
// one round. On one card, both in turn, three sets of operands: stacked 7B gate and up at 512,
// 1024 and 2048 E2M1 tokens 51.0, 100 and 144 us against 52.4, 105 and 146; 8192 tokens of 7B QKV
// 84 against 89; 38 E4M3 tokens of 41740 x 3584 25.7 against 27.2. Past five rounds that gains
// nothing (32B gate at 4096, seven rounds: 309 against 306). These kernels keep state across tiles
// that the scalar registers do not hold: 18 to 77 of them (256 x 256) are kept in vector lanes.
// `slots`: the ring's, 0 if none can hold a token fragment of each wave's outputs.
bool mx4_ahead(int64_t tiles, int64_t stages, int splits, int slots, int per_cu) {
  const int64_t need = (tiles + 7) / 8 * 8, round = (int64_t)kCUs * per_cu;
  return slots > 0 && splits == 1 && stages >= slots && need > round && need <= 5 * round;
}

template <bool XFP4, int T, int BN, int BM, int WN, int WM, int S, int KS>
hipError_t launch_tile(const Mx4Params& g, int splits, int per_cu, float* part, hipStream_t st) {
  Mx4TileParams p;
  p.g = g;
  p.part = splits > 1 ? part : nullptr;
  p.tiles_m = (int)((g.M + BM - 1) / BM);
  p.tiles_n = (int)((g.N + BN - 1) / BN);
  p.stages = (int)((g.K + KS - 1) / KS);
  p.splits = splits;
  // Outputs past half the 256 MB of the memory-side cache leave it to the operands. On one card,
  // with and without in turn, three sets of operands: 2048 and 4096 E2M1 tokens of the stacked 7B
  // gate and up (155 and 310 MB) 144 and 291 us against 157 and 327, the 32B gate at 4096 290
  // against 319 (E4M3 tokens 424 against 439); at 1024 tokens (78 MB) the hint cost 5%.
  p.nt_out = 2 * g.M * g.N > ((int64_t)128 << 20);
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  constexpr bool kAhead = Mx4Ahead<XFP4, T, BN, BM, WN, WM, KS>::value;
  const bool ahead = mx4_ahead(tiles, p.stages, splits, kAhead ? S : 0, per_cu);
  if constexpr (kAhead) {
    if (ahead)
      hipLaunchKernelGGL((mx4_tile_kernel<XFP4, T, BN, BM, WN, WM, S, KS, true>), dim3((unsigned)(kCUs * per_cu)),
                         dim3(64 * WN * WM), 0, st, p);
  }
  if (!ahead)
    hipLaunchKernelGGL((mx4_tile_kernel<XFP4, T, BN, BM, WN, WM, S, KS, false>),
                       dim3((unsigned)((tiles * splits + 7) / 8 * 8)), dim3(64 * WN * WM), 0, st, p);
  if (splits > 1) {
    const int64_t total = g.M * ((g.N + 3) >> 2);
    hipLaunchKernelGGL(mx4_sum_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, st, part, splits, g);
  }
  return hipGetLastError();
}

// X: bf16 tokens to quantize in the kernel (stride ldx), or NULL for codes in p.
template <bool XFP4, bool FUSED, int NW, int KW, int D>
hipError_t launch_decode(const Mx4Params& p, const uint16_t* X, int64_t ldx, hipStream_t st) {
  constexpr int rows = 16 * (NW / KW);
  const size_t lds = FUSED ? (size_t)(XFP4 ? p.M * p.K / 2 : p.M * p.K) + p.M * p.K / 32 : 0;
  hipLaunchKernelGGL((mx4_decode_kernel<XFP4, FUSED, NW, KW, D>), dim3((unsigned)((p.N + rows - 1) / rows)),
                     dim3(64 * NW), lds, st, p, X, ldx);
  return hipGetLastError();
}

// Tile configurations and what they cost: us per tile besides its stages, and per stage
// alone on a CU / with a second block there (measured, one full round of 256 blocks at
// K = 1792 .. 7168).
struct Mx4Config {
  int BN, BM, KS, per_cu;
  float base, alone, shared;
  int slots;  // of a ring that can copy into the next tile, else 0
  hipError_t (*run)(const Mx4Params&, int, int, float*, hipStream_t);
};
template <bool XFP4, int T, int BN, int BM, int WN, int WM, int S, int KS>
constexpr Mx4Config config(int per_cu, float base, float alone, float shared = 0.0f) {
  return {BN, BM, KS, per_cu, base, alone, shared, Mx4Ahead<XFP4, T, BN, BM, WN, WM, KS>::value ? S : 0,
          launch_tile<XFP4, T, BN, BM, WN, WM, S, KS>};
}
constexpr Mx4Config kFp4Configs[] = {
    config<true, 32, 256, 256, 2, 4, 2, 256>(1, 8.0f, 2.00f),
    config<true, 16, 160, 256, 2, 4, 2, 256>(1, 5.5f, 1.50f),
    config<true, 16, 160, 128, 2, 4, 3, 256>(1, 5.0f, 0.87f),
    config<true, 32, 128, 128, 2, 4, 4, 256>(1, 5.0f, 0.65f),
    config<true, 16, 160, 64, 2, 4, 4, 256>(1, 4.5f, 0.65f),
    config<true, 16, 128, 64, 4, 2, 4, 256>(1, 4.0f, 0.45f),
    config<true, 16, 64, 64, 2, 2, 4, 256>(2, 4.4f, 0.31f, 0.44f),
    config<true, 16, 64, 32, 4, 1, 4, 256>(2, 3.5f, 0.30f, 0.35f),
};
constexpr Mx4Config kFp8Configs[] = {
    config<false, 32, 256, 256, 2, 4, 3, 128>(1, 8.0f, 1.42f),
    config<false, 32, 160, 256, 1, 8, 3, 128>(1, 5.0f, 1.02f),
    config<false, 16, 160, 128, 2, 4, 2, 256>(1, 4.0f, 1.40f),
    config<false, 32, 128, 128, 2, 4, 4, 128>(1, 4.8f, 0.50f),
    config<false, 16, 160, 64, 2, 4, 3, 256>(1, 4.8f, 0.68f),
    config<false, 16, 64, 64, 2, 2, 3, 256>(1, 4.0f, 0.38f),
    config<false, 16, 64, 32, 4, 1, 4, 256>(2, 3.8f, 0.31f, 0.42f),
};

struct Mx4Plan {
  const Mx4Config* c;  // NULL: the decode kernel on token codes
  int splits;
};

// Up to 16 tokens and matrices up to 8192 x 8192 take the decode kernel (7B O
// projection, 3.8 - 5.0 us against 6.3 - 7.1 on the smallest tiles; beyond, the tiles'
// deeper copy rings win: 15 against 20 - 32 us on the stacked gate and up). Else the
// configuration and the number of K splits whose rounds of blocks over the CUs cost
// least by the table; a split adds a launch and one write and read of its partial sums.
Mx4Plan make_mx4_plan(int64_t M, int64_t N, int64_t K, bool fp4) {
  if (M <= 16 && N <= 8192 && K <= 8192) return {nullptr, 1};
  const Mx4Config* first = fp4 ? kFp4Configs : kFp8Configs;
  const int n = fp4 ? (int)(sizeof(kFp4Configs) / sizeof(Mx4Config)) : (int)(sizeof(kFp8Configs) / sizeof(Mx4Config));
  Mx4Plan best{first, 1};
  float least = 3.0e38f;
  for (int i = 0; i < n; ++i) {
    const Mx4Config& c = first[i];
    const int64_t tiles = ((M + c.BM - 1) / c.BM) * ((N + c.BN - 1) / c.BN);
    const int64_t stages = (K + c.KS - 1) / c.KS;
    for (int s : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (s > 1 && (stages < 4 * s || tiles * s > 2 * kCUs)) break;
      const int64_t blocks = tiles * s, round = (int64_t)kCUs * c.per_cu;
      const float step = blocks > kCUs && c.per_cu > 1 ? c.shared : c.alone;
      float t = (float)((blocks + round - 1) / round) * (c.base + step * (float)((stages + s - 1) / s));
      if (s > 1) t += 3.5f + (float)s * (float)M * (float)N * 1.0e-6f;
      if (t < least) {
        least = t;
        best = {&c, s};
      }
    }
  }
  return best;
}

}  // namespace

hipError_t launch_mx4_quant(const void* A, int64_t R, int64_t K, int64_t lda, int bf16, int fmt,
                            void* codes, uint8_t* scales, hipStream_t st) {
  uint8_t* q = static_cast<uint8_t*>(codes);
  const dim3 b(256);
  return chunk_launches(R, ((K + 127) >> 7) << 4, 1, [&](int64_t r, ChunkWalk w, dim3 g) {
    if (fmt == kActMxFp4) {
      if (bf16) hipLaunchKernelGGL((mx4_quant_kernel<true, true>), g, b, 0, st, A, R, K, lda, q, scales, r, w);
      else hipLaunchKernelGGL((mx4_quant_kernel<true, false>), g, b, 0, st, A, R, K, lda, q, scales, r, w);
    } else {  // bf16 tokens of a product
      hipLaunchKernelGGL((mx4_quant_kernel<false, true>), g, b, 0, st, A, R, K, lda, q, scales, r, w);
    }
  });
}

hipError_t launch_mx_dequant(const void* codes, const uint8_t* scales, int64_t R, int64_t K, int fmt,
                             void* out, int64_t ldo, int bf16, hipStream_t st) {
  const uint8_t* q = static_cast<const uint8_t*>(codes);
  auto run = [&](auto fp4, auto to_bf16, auto past_l2) {
    return chunk_launches(R, K >> 3, 2, [&](int64_t r, ChunkWalk w, dim3 g) {
      hipLaunchKernelGGL((mx_dequant_kernel<decltype(fp4)::value, decltype(to_bf16)::value, decltype(past_l2)::value>),
                         g, dim3(256), 0, st, q, scales, R, K, out, ldo, r, w);
    });
  };
  auto by_type = [&](auto fp4) {
    if (!bf16) return run(fp4, std::false_type{}, std::false_type{});
    if (2.0 * (double)R * (double)K > 32.0 * 1048576.0) return run(fp4, std::true_type{}, std::true_type{});
    return run(fp4, std::true_type{}, std::false_type{});
  };
  return fmt == kActMxFp4 ? by_type(std::true_type{}) : by_type(std::false_type{});
}

hipError_t launch_mx4_gemm(const void* Xq, const uint8_t* sx, int xfmt, const void* Wq,
                           const uint8_t* sw, int64_t M, int64_t N, int64_t K, int out_raw, void* Y,
                           int64_t ldy, void* ws, hipStream_t st) {
  if (M == 0 || N == 0) return hipSuccess;
  const Mx4Params p{static_cast<const uint8_t*>(Xq), sx, static_cast<const uint8_t*>(Wq), sw,
                    M, N, K, Y, ldy, out_raw};
  const bool fp4 = xfmt == kActMxFp4;
  const Mx4Plan plan = make_mx4_plan(M, N, K, fp4);
  if (plan.c) return plan.c->run(p, plan.splits, plan.c->per_cu, static_cast<float*>(ws), st);
  return fp4 ? launch_decode<true, false, 8, 8, 4>(p, nullptr, 0, st)
             : launch_decode<false, false, 8, 8, 4>(p, nullptr, 0, st);
}

void mx4_plan(int64_t M, int64_t N, int64_t K, int xfmt, int* tile_n, int* tile_m, int* splits, int* ahead) {
  const Mx4Plan plan = make_mx4_plan(M, N, K, xfmt == kActMxFp4);
  const Mx4Config* c = plan.c;
  *tile_n = c ? c->BN : 16;
  *tile_m = c ? c->BM : 0;
  *splits = plan.splits;
  *ahead = c && mx4_ahead(((M + c->BM - 1) / c->BM) * ((N + c->BN - 1) / c->BN), (K + c->KS - 1) / c->KS,
                          plan.splits, c->slots, c->per_cu);
}

size_t mx4_gemm_ws_bytes(int64_t M, int64_t N, int64_t K, int xfmt) {
  const Mx4Plan plan = make_mx4_plan(M, N, K, xfmt == kActMxFp4);
  return plan.splits > 1 ? (size_t)plan.splits * (size_t)M * (size_t)((N + 3) & ~(int64_t)3) * 4 : 0;
}

// One launch where the blocks' own quantization of the tokens costs less than a launch
// for it (2.6 us): up to 16384 values (four tokens of the 7B hidden size: 6.8 against
// 7.6 us on QKV; eight: 9.4 against 7.9), and for one or two tokens up to what fits the
// LDS (7B down projection, one token: 10.5 against 13.7 us).
bool mx4_one_launch(int64_t M, int64_t K) {
  return K > 0 && M <= 16 && (M * K <= 16384 || (M <= 2 && M * K <= 40960));
}

// Many rows (the stacked gate and up) take 32 rows a block, half of K a wave (14.3 us; 17.1
// with 16 rows over eight waves). Long rows whose 16-row tiles all find a CU split K over
// 16 waves (7B down projection 10.4 against 11.3 us over eight; the 32B one, 320 tiles,
// 24.0 against 20.5). Rows up to 4096 need no more than two pairs a wave in flight (7B QKV
// 5.7 against 6.0 us).
template <bool XFP4>
hipError_t launch_fused(const Mx4Params& p, const uint16_t* X, int64_t ldx, hipStream_t st) {
  if (p.N > 16384) return launch_decode<XFP4, true, 4, 2, 4>(p, X, ldx, st);
  if (p.K >= 8192 && p.N <= 16 * kCUs) return launch_decode<XFP4, true, 16, 16, 4>(p, X, ldx, st);
  if (p.K <= 4096) return launch_decode<XFP4, true, 8, 8, 2>(p, X, ldx, st);
  return launch_decode<XFP4, true, 8, 8, 4>(p, X, ldx, st);
}

// The workspace holds the product's partial sums, the token codes, then their scales
// (each 256-byte aligned).
hipError_t launch_mx4_linear(const void* X, int64_t ldx, int xfmt, const void* Wq, const uint8_t* sw,
                             int64_t M, int64_t N, int64_t K, void* Y, int64_t ldy, void* ws,
                             hipStream_t st) {
  if (M == 0 || N == 0) return hipSuccess;
  const bool fp4 = xfmt == kActMxFp4;
  if (mx4_one_launch(M, K)) {
    const Mx4Params p{nullptr, nullptr, static_cast<const uint8_t*>(Wq), sw, M, N, K, Y, ldy, 0};
    const uint16_t* x = static_cast<const uint16_t*>(X);
    return fp4 ? launch_fused<true>(p, x, ldx, st) : launch_fused<false>(p, x, ldx, st);
  }
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  uint8_t* xq = static_cast<uint8_t*>(ws) + up(mx4_gemm_ws_bytes(M, N, K, xfmt));
  uint8_t* sx = xq + up((size_t)(fp4 ? M * (K >> 1) : M * K));
  const hipError_t e = launch_mx4_quant(X, M, K, ldx, 1, xfmt, xq, sx, st);
  if (e != hipSuccess) return e;
  return launch_mx4_gemm(xq, sx, xfmt, Wq, sw, M, N, K, 0, Y, ldy, ws, st);
}

}  // namespace qr
