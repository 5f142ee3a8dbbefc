// Losses over a large vocabulary for gfx950: from hidden states X [M, K] and the head
// W [N, K] (bf16) to per-token losses and back, without the logits.
//
//   z[t,v] = c sum_k X[t,k] W[v,k],  lse[t] = log sum_v exp z[t,v]
//   G[t,v] = a_t exp(z[t,v] - lse[t]) - sum_j b_tj [v = id_tj],  dX = G W,  dW = G^T X
//
// The sums and logits are products in bf16, dX and dW of G in two parts of bf16 or in fp16 (kTwice).
//
// A token has a list of ids with weights (one id of weight 1 for a log-probability).
// Tokens without one are masked: the others are numbered in order ("compact" tokens,
// their count nv known to the GPU only) and their rows of X copied together, so masked
// rows cost nothing and what they hold reaches no sum.
//
// Four products share one kernel (vocab_tile): the logits' softmax sums; the same logits
// again with G as output, a piece of the vocabulary at a time; that piece's part of dX
// and its rows of dW. The sums need 2 M N K operations and W once, the gradient 6 M N K and
// W twice (its logits are computed again: held, they would be M N values) beside dW, and beyond 128
// tokens once more for its largest value. Up to about 128 tokens memory bounds both (W of 131072 x 3584 for
// 1 token: 141 us, 6.7 TB/s), beyond about 512 the matrix cores and the power that they take: 4096 tokens
// of 131072 ids, 3584 wide, take 2.83 ms for the sums (1.36 PFLOP/s), 10.1 ms for the gradient (1.14), 5120
// wide 3.98 ms (1.38) and 14.2; a library product in bf16 alone of the sums' shape reaches 1.47.
#include <cmath>
#include <type_traits>

#include "qr_copy.h"
#include "qr_internal.h"
#include "qr_mx.h"
#include "qr_vocab.h"

namespace qr {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr double kLn2 = 0.6931471805599453;
constexpr int kNone = 0x7fffffff;  // list key of no entry: past every id

// Lambdas of a kernel share its state in registers only where they are inlined.
#define QR_INLINE __attribute__((always_inline))

// ---------------------------------------------------------------------------
// Lists and compact tokens
// ---------------------------------------------------------------------------

// One wave per token: weights p of the list's entries and the entries in the order of
// their ids (entries of one id in the order of the list, ids outside [0, N) last).
// p = softmax over the entries, or exp(c s - teacher_lse). L <= kVocabMaxList; ranks by
// counting in LDS. first[b] is the first entry whose id is not below b << shift, where a tile's
// waves begin to look for theirs. 4096 tokens of 64 entries take 9 us, a launch 2 of them.
template <bool BF16>
__global__ __launch_bounds__(256) void vocab_list_kernel(const int64_t* __restrict__ index,
                                                         const void* __restrict__ teacher,
                                                         const float* __restrict__ teacher_lse, int64_t M,
                                                         int64_t N, int L, float scale, int* __restrict__ keys,
                                                         float* __restrict__ wts, float* __restrict__ mass,
                                                         uint16_t* __restrict__ first, int buckets, int shift) {
  extern __shared__ __attribute__((aligned(16))) uint8_t list_smem[];
  // An entry's id and place in the list, in that order of weight: no two alike. N < 2^22, so
  // that ~0 is no entry's.
  static_assert(kVocabMaxList <= 1024, "places of 10 bits");
  constexpr uint32_t kNoCode = ~0u;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, L4 = (L + 3) & ~3;
  uint32_t* code = reinterpret_cast<uint32_t*>(list_smem) + wave * 3 * L4;
  int* sorted = reinterpret_cast<int*>(code + L4);
  float* y = reinterpret_cast<float*>(sorted + L4);  // c s, then the weight
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t >= M) return;
  const uint64_t below = ((uint64_t)1 << lane) - 1;
  float top = -INFINITY, sum = 0.0f;
  int none = 0;  // entries that are none
  for (int j0 = 0; j0 < L4; j0 += 64) {
    const int j = j0 + lane;
    bool ok = false;
    if (j < L) {
      const int64_t id = index[t * L + j];
      float s;
      if constexpr (BF16) s = bf16_lo(static_cast<const uint16_t*>(teacher)[t * L + j]);
      else s = static_cast<const float*>(teacher)[t * L + j];
      ok = id >= 0 && id < N;
      code[j] = ok ? (uint32_t)id << 10 | (uint32_t)j : kNoCode;
      y[j] = scale * s;
      if (ok) top = fmaxf(top, y[j]);
    } else if (j < L4) {
      code[j] = kNoCode;
    }
    none += __popcll(__ballot(j < L && !ok));
  }
  top = wave_max(top);
  // without an entry of weight all weights are zero
  const float norm = teacher_lse ? teacher_lse[t] : top == -INFINITY ? 0.0f : top;
  for (int j = lane; j < L; j += 64) {
    y[j] = code[j] == kNoCode ? 0.0f : expf(y[j] - norm);
    sum += y[j];
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
  const float div = teacher_lse || sum == 0.0f ? 1.0f : sum;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the wave's own part of LDS
  int seen = L - none;  // place of the next one that is none
  for (int j0 = 0; j0 < L; j0 += 64) {
    const int j = j0 + lane;
    const uint32_t mine = j < L ? code[j] : 0u;
    const uint64_t b = __ballot(j < L && mine == kNoCode);
    int rank = 0;
    for (int i = 0; i < L4; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(code + i);
      rank += (v.x < mine) + (v.y < mine) + (v.z < mine) + (v.w < mine);
    }
    if (mine == kNoCode) rank = seen + __popcll(b & below);
    seen += __popcll(b);
    if (j < L) {
      const int k = mine == kNoCode ? kNone : (int)(mine >> 10);
      sorted[rank] = k;
      keys[t * L + rank] = k;
      wts[t * L + rank] = y[j] / div;
    }
  }
  if (lane == 0) mass[t] = sum / div;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  for (int b = lane; b < buckets; b += 64) {
    int lo = 0, hi = L;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sorted[mid] < b << shift) lo = mid + 1;
      else hi = mid;
    }
    first[t * buckets + b] = (uint16_t)lo;
  }
}

// Whether token t has a list (key 0 of its L), or, with `target`, an id in [0, N).
__device__ __forceinline__ bool vocab_live(const int64_t* target, const int* keys, int L, int64_t N, int64_t t) {
  if (!target) return keys[t * L] != kNone;
  const int64_t id = target[t];
  return id >= 0 && id < N;
}

// Parts of a piece's ids whose sums of dX are kept apart: as fill the CUs, unless the sums (4 bytes
// each, written and read at about 4 TB/s) take longer than the stages that another part saves (the least
// of stages us / s + s sums). The tokens that count decide, whom the GPU numbers.
struct DxPlan {
  int tiles_a, bm;  // tiles of the hidden values, rows of a tile
  int stages;       // of a piece
  int cap;          // rows of sums that the workspace holds
  float worth;      // stages us / (time of a row of sums)
  __host__ __device__ int splits(int64_t rows) const {
    if (rows <= 0 || cap <= 0) return 1;
    int64_t s = 256 / (tiles_a * ((rows + bm - 1) / bm));
    const float best = sqrtf(worth / (float)rows);
    if ((float)s > best) s = (int64_t)best;
    if (s > stages / 2) s = stages / 2;
    if (s > cap / rows) s = cap / rows;
    return (int)(s < 1 ? 1 : s);
  }
};

struct VocabCompact {
  const int64_t* target;  // NULL: lists
  int* keys;              // [M][L]; written (L = 1) with `target`
  int L;
  int64_t M, N, K, ldx;
  const uint16_t* X;
  uint16_t* Xc;  // rows of the compact tokens; twice over where nv <= twice
  int twice;
  // gradients
  DxPlan dx;
  const float *g, *mass;
  float gscale;         // scale, with the gradient's sign
  float *factor, *top;  // [M]: G of a compact token by its H, and the largest of its row times that
  const uint16_t* W;
  int64_t ldw;
  float* peaks;
  int peak_blocks, shift;
  bool stream;
  int *nv, *map, *inv;  // nv: their count, and dX's splits
  float *value, *lse;  // losses: masked tokens' results
};

__device__ __forceinline__ void vocab_count(const VocabCompact& p, int n) {
  p.nv[0] = n;
  p.nv[1] = p.dx.splits(n <= p.twice ? 2 * n : n);
}

// H, what G is held as in fp16: 2^kHalf G / (scale g P), P the weight of the token's list. |H| is at most
// 2^kHalf; fp16 ends at 65504, so that an exponential may come out at 3.9 for 1.
constexpr int kHalf = 14;
constexpr int kPeaks = 2048;  // blocks that look for W's largest value, at most

__device__ __forceinline__ uint32_t half_pair(float a, float b) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef _Float16 h2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{a, b}), h2));
}

__device__ __forceinline__ uint32_t max16(uint32_t a, uint32_t b) {  // of two pairs of 16 bits each
  typedef uint16_t u2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u2, a), __builtin_bit_cast(u2, b)));
}

// The largest of pairs of a block's four waves as bf16 without their signs, to all threads.
__device__ __forceinline__ float block_top(uint32_t pair) {
  __shared__ uint32_t tops[4];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) pair = max16(pair, __shfl_xor(pair, o, 64));
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = pair;
  __syncthreads();
  const uint32_t m = max16(max16(tops[0], tops[1]), max16(tops[2], tops[3]));
  return fmaxf(bf16_lo(m), bf16_hi(m));
}

// Token t (live, compact number c of n): its entries of the tables, its rows of Xc. One block.
__device__ __forceinline__ void vocab_take_row(const VocabCompact& p, int64_t t, int c, int n) {
  const uint4* src = reinterpret_cast<const uint4*>(p.X + t * p.ldx);
  uint4* dst = reinterpret_cast<uint4*>(p.Xc + c * p.K);
  const int64_t again = n <= p.twice ? n * p.K / 8 : 0;
  uint32_t top = 0;
  for (int64_t i = threadIdx.x; i < p.K >> 3; i += 256) {
    const uint4 v = src[i];
    dst[i] = v;
    if (again) dst[again + i] = v;
    top = max16(max16(top, v.x & 0x7fff7fff), v.y & 0x7fff7fff);
    top = max16(max16(top, v.z & 0x7fff7fff), v.w & 0x7fff7fff);
  }
  if (!p.factor || n <= p.twice) return;
  const float most = block_top(top);
  if (threadIdx.x == 0) {
    const float f = ldexpf(p.g[t] * p.gscale * (p.mass ? p.mass[t] : 1.0f), -kHalf);
    p.factor[c] = f;
    p.top[c] = fabsf(f) * most;
  }
}

// The largest of W, for fp16 products: `block` of p.peak_blocks, rows of W 256 >> p.shift at a time. In the
// launch that copies the tokens' rows. 131072 x 3584 takes 135 us, 7.0 TB/s, with non-temporal reads, 172
// without; W that the MALL holds is read without, the logits find it there (gradient of 400 tokens of 5000 ids
// 104 us, else 112).
template <bool STREAM>
__device__ __forceinline__ void vocab_peak(const VocabCompact& p, int block) {
  constexpr int U = 4;
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  const int64_t step = (int64_t)p.peak_blocks * (256 >> p.shift);
  const int c0 = threadIdx.x & ((1 << p.shift) - 1);
  uint32_t top = 0;
  for (int64_t r = block * (int64_t)(256 >> p.shift) + (threadIdx.x >> p.shift); r < p.N; r += U * step) {
    for (int64_t c = c0; c < p.K >> 3; c += 1 << p.shift) {
      u4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t row = r + u * step < p.N ? r + u * step : r;
        const u4* src = reinterpret_cast<const u4*>(p.W + row * p.ldw + 8 * c);
        v[u] = STREAM ? __builtin_nontemporal_load(src) : *src;
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max16(top, v[u][e] & 0x7fff7fff);
    }
  }
  const float most = block_top(top);
  if (threadIdx.x == 0) p.peaks[block] = most;
}

__device__ __forceinline__ void vocab_peak(const VocabCompact& p, int block) {
  if (p.stream) vocab_peak<true>(p, block);
  else vocab_peak<false>(p, block);
}

// Compact numbers and rows in one launch, a block a token that counts the live ones itself.
// M reads a block: up to kVocabCount tokens less than another launch (gradients of 5000 ids, 1 token 21 us
// and 22 in two launches; from 300 tokens to 2048 within 1 us of each other, 4096 217 in two and 224).
constexpr int64_t kVocabCount = 512;
__global__ __launch_bounds__(256) void vocab_compact_kernel(const VocabCompact p) {
  __shared__ int below[4], all[4];
  const int64_t t = blockIdx.x;
  int nb = 0, na = 0;
  bool mine = false;
  for (int64_t i = threadIdx.x; i < p.M; i += 256) {
    const bool live = vocab_live(p.target, p.keys, p.L, p.N, i);
    nb += live && i < t;
    na += live;
    mine |= live && i == t;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    nb += __shfl_xor(nb, o, 64);
    na += __shfl_xor(na, o, 64);
  }
  if ((threadIdx.x & 63) == 0) {
    below[threadIdx.x >> 6] = nb;
    all[threadIdx.x >> 6] = na;
  }
  const bool live = __syncthreads_or(mine);
  const int c = below[0] + below[1] + below[2] + below[3], n = all[0] + all[1] + all[2] + all[3];
  if (t >= p.M) {
    if (n > p.twice) vocab_peak(p, (int)(t - p.M));
    return;
  }
  if (threadIdx.x == 0) {
    if (t == 0) vocab_count(p, n);
    if (p.target) p.keys[t] = live ? (int)p.target[t] : kNone;
    p.inv[t] = live ? c : -1;
    if (live) {
      p.map[c] = (int)t;
    } else if (p.value) {
      p.value[t] = 0.0f;
      p.lse[t] = 0.0f;
    }
  }
  if (live) vocab_take_row(p, t, c, n);
}

// The same for more tokens: one block numbers them, then a block a compact token copies.
__global__ __launch_bounds__(1024) void vocab_scan_kernel(const VocabCompact p) {
  __shared__ int wsum[2][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int base = 0, buf = 0;
  for (int64_t t0 = 0; t0 < p.M; t0 += 1024, buf ^= 1) {
    const int64_t t = t0 + threadIdx.x;
    const bool live = t < p.M && vocab_live(p.target, p.keys, p.L, p.N, t);
    const uint64_t b = __ballot(live);
    if (lane == 0) wsum[buf][wave] = __popcll(b);
    __syncthreads();
    int before = base, all = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      if (w < wave) before += wsum[buf][w];
      all += wsum[buf][w];
    }
    const int c = before + __popcll(b & (((uint64_t)1 << lane) - 1));
    if (t < p.M) {
      if (p.target) p.keys[t] = live ? (int)p.target[t] : kNone;
      p.inv[t] = live ? c : -1;
      if (live) {
        p.map[c] = (int)t;
      } else if (p.value) {
        p.value[t] = 0.0f;
        p.lse[t] = 0.0f;
      }
    }
    base += all;
  }
  if (threadIdx.x == 0) vocab_count(p, base);
}

__global__ __launch_bounds__(256) void vocab_gather_kernel(const VocabCompact p) {
  const int c = blockIdx.x, n = *p.nv;
  if (c < n) vocab_take_row(p, p.map[c], c, n);
  else if (c >= p.M && n > p.twice) vocab_peak(p, (int)(c - p.M));
}

// The power of two that brings values of up to `most` below 2^15.
__device__ __forceinline__ int half_exponent(float most) {
  if (!(most > 0.0f && most < INFINITY)) return 0;
  const int e = 14 - ilogbf(most);
  return e < 126 ? e : 126;
}

__device__ __forceinline__ float block_max(float v) {  // not negative, four waves
  __shared__ float tops[4];
  v = wave_max(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = v;
  __syncthreads();
  return fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
}

// Operands of the fp16 products: the exponents (0: W's, 1: that of X with the factors) and X with them.
// Powers of two for a whole tensor keep all of bf16's bits down to 2^-28 of its largest value, and 2^-38 of
// that below; the factors round X to fp16, 2^-11 of each value. One power for all tokens, and the factors with
// X instead of G: dX of a token is then as exact however small its gradient is beside the others'.
__global__ __launch_bounds__(256) void vocab_half_kernel(const uint16_t* __restrict__ Xc, int64_t K,
                                                         const float* __restrict__ factor,
                                                         const float* __restrict__ top, const float* __restrict__ peaks,
                                                         int npeaks, const int* __restrict__ nv, int twice,
                                                         int* __restrict__ expo, uint16_t* __restrict__ Xh) {
  const int n = *nv;
  if (n <= twice) return;
  float m = 0.0f;
  for (int i = threadIdx.x; i < n; i += 256) m = fmaxf(m, top[i]);
  const int kx = half_exponent(block_max(m));
  if (blockIdx.x == 0) {
    float w = 0.0f;
    for (int i = threadIdx.x; i < npeaks; i += 256) w = fmaxf(w, peaks[i]);
    w = block_max(w);
    if (threadIdx.x == 0) {
      expo[0] = half_exponent(w);
      expo[1] = kx;
    }
  }
  if (!Xh) return;
  for (int c = blockIdx.x; c < n; c += gridDim.x) {
    const double f = ldexp((double)factor[c], kx);  // beyond fp32 where a row of X is small
    for (int64_t i = threadIdx.x; i < K >> 3; i += 256) {
      float x[8];
      bf16x8(*reinterpret_cast<const uint4*>(Xc + c * K + 8 * i), x);
      v8h h;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = (_Float16)(float)((double)x[e] * f);
      *reinterpret_cast<v8h*>(Xh + c * K + 8 * i) = h;
    }
  }
}

// ---------------------------------------------------------------------------
// Products
// ---------------------------------------------------------------------------
enum { kSums, kGrad, kDX, kDW };

// Up to so many tokens that count G is held in two parts of bf16, beyond in fp16, with factors and powers of
// two of its own (H, vocab_half_kernel). Either leaves the gradients next to no error but their own rounding to
// bf16: 0.0017 of them against float64, in norm, as the plain fp32 form's; G in one part of bf16 leaves
// 0.0023 - 0.0025. Two parts are two products, which memory hides for few tokens (us in one part and in
// two, 32768 ids, 3584 wide: 1 token 123 and 123, 33 130 and 143, 128 176 and 212; 128 of 131072 584 and 741).
// fp16 needs the largest value of W, a pass over it (1.4% of 4096 tokens' gradient), W's fragments converted
// on their way to the matrix cores (5%), and products that take more power than bf16's (4%): us in two
// parts and in fp16, 131072 ids, 3584 wide, 140 tokens 937 and 887, 256 1185 and 974, 512 2094 and 1627,
// 4096 15265 and 10115 (in one part of bf16 9130); 200 tokens of 5000 ids 78 and 80, 1000 182 and 159, 1000
// tokens 512 wide 75 and 65.
constexpr int kTwice = 128;

struct VocabTile {
  const uint16_t *A, *B;
  int64_t lda, ldb;
  const int* nv;
  int direct;      // kSums, M of them: tokens are numbered by each block, B is X itself
  const int64_t* target;
  int64_t N;       // ids in all
  int64_t ext_a;   // extent of the A side: ids of the piece (kSums, kGrad), K (kDX, kDW)
  int64_t ids;     // ids of the piece
  int64_t id0;     // its first id
  int64_t K;
  int tiles_a;
  const int* map;
  const int* keys;
  const float *wts, *mass, *lse, *g;
  int L;
  const uint16_t* first;  // [M][buckets], L > 1
  int buckets, shift;
  float scale, sign;  // G = sign * ...: -1 for a log-probability
  float2* part;    // kSums: [tiles_a][ldpart]
  int64_t ldpart;
  float* zl;       // kSums: logits of the lists' ids, in base 2
  uint16_t* out16; // kGrad: G [nv][ldo]; kDW: dW + id0 ldo
  int64_t ldo;
  float* out32;    // kDX: [splits][rows of G][K]
  int add;         // kDX: add to what is there
  // kSums, kGrad, kDX: W's copies may carry the non-temporal hint; kDW: stores may. They do where a
  // tile holds all tokens that count: nothing of W is read again, and dW is written to be read later (less
  // time by, 3584 wide, W past the MALL or not there yet: log-probabilities of 1 token, 131072 ids, 12%, 128
  // 8%, 1 of 32768 10%; gradient of 1 of 131072 19%, 33 of 32768 19%). kGrad reads
  // without it where kDX will find W in the MALL (33 x 32768: 3 us), kDX where it finds it in the L2s
  // (gradient, 200 tokens, 3584 wide or 1808: 10000 ids 108 / 110, 5000 68 / 70, 4112 x 1808 50 / 46).
  bool stream;
  int twice;       // up to so many compact tokens G is held in two parts, beyond as H in fp16
  const int* expo; // exponents of the fp16 operands
  const uint16_t* Xh;  // kDW: A of fp16 products
};

// Tokens that a launch's blocks number themselves (vocab_number): 16 tokens of 5000 ids,
// 512 wide, take 13 us, numbered by a launch of their own 15; 128 of 32768, 1024 wide, 27 and 31;
// 256 of 5000 17 and 19.
constexpr int kVocabDirect = 256;

// The compact tokens of p.direct tokens into LDS (int [nv] from the start); their count. All
// waves of the block; the caller synchronizes before it writes there again.
__device__ __forceinline__ int vocab_number(const VocabTile& p, int wid, int lane, int waves, uint8_t* smem) {
  int* const map = reinterpret_cast<int*>(smem);
  uint64_t* const mask = reinterpret_cast<uint64_t*>(smem + kVocabDirect * 4);
  for (int g = wid; g < kVocabDirect / 64; g += waves) {
    const int t = 64 * g + lane;
    const uint64_t b = __ballot(t < p.direct && vocab_live(p.target, p.keys, p.L, p.N, t));
    if (lane == 0) mask[g] = b;
  }
  __syncthreads();
  int n = 0;
#pragma unroll
  for (int g = 0; g < kVocabDirect / 64; ++g) {
    const uint64_t b = mask[g];
    if (g % waves == wid && ((b >> lane) & 1)) map[n + __popcll(b & (((uint64_t)1 << lane) - 1))] = 64 * g + lane;
    n += __popcll(b);
  }
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(n);
}

template <int BN, int BM, int NW, int S>
constexpr int ring_bytes() {  // copies of 8 rows (1 KB), as many by each wave
  return S * ((BN / 8 + NW - 1) / NW + (BM / 8 + NW - 1) / NW) * NW * 1024;
}

// A block: BN x BM outputs, A side by B side, over K steps of 64 through a ring of S
// stages in LDS, filled by LDS-DMA copies; WN x WM waves. An operand is either K-contiguous
// ("rows": its rows run along K; LDS rows of 64 elements, 16-byte chunk q of row r at
// q ^ (r / 2 % 8)) or has its rows along the other axis ("columns": LDS holds 64 rows of K,
// read with the transposing load, whose 16 lanes take four rows of K by 16 columns; the 16-byte
// chunks of row k at q ^ (4 (k % 4) + 2 (k / 8 % 2)), so that the rows that a load takes at
// once meet different banks: none of its reads conflict).
//          A side            B side             K
//   kSums  ids (W, rows)     tokens (X, rows)   hidden
//   kGrad  ids (W, rows)     tokens (X, rows)   hidden
//   kDX    hidden (W, cols)  tokens (G, rows)   ids
//   kDW    hidden (X, cols)  ids (G, cols)      tokens
// F16: H in G's place, W converted behind its LDS reads, X as vocab_half_kernel leaves it.
//
// Products are 16 x 16 x 32: with all CUs busy they are bound by power (the clock falls to 1.5 -
// 1.9 GHz, the matrix cores busy for 69% of it), and from registers alone these reach 2.06
// PFLOP/s, 32 x 32 x 16 1.87. In the kernel, of 4096 tokens of 131072 ids, 3584 wide, the sums take 5% less
// so, 5120 wide 4%, the first's gradient 2%. Register r of fragment
// (i, j): A side 16 i + 4 (lane / 16) + r, B side 16 j + lane % 16.
//
// A wave's tile in the 256 x 256 block is 64 x 128 (four by two waves; two by four spill registers, and
// four waves of 128 x 128 took 8% longer). Copies bind smaller tiles: a CU takes in about 21 - 23 bytes a
// clock, 12 bytes for 1000 operations on 256 x 128 (matrix cores 42 - 50% busy), 8 on 256 x 256. Tiles of
// 192 x 320 and 128 x 384, 8 and 10 bytes, gain 13% at best and lose elsewhere.
//
// `block` and the grid it belongs to may be a part of the launch's.
template <int MODE, int BN, int BM, int WN, int WM, int S, bool HINT, bool F16>
__device__ __forceinline__ void vocab_tile_body(const VocabTile& p, int block, uint8_t* smem) {
  constexpr bool TA = MODE == kDX || MODE == kDW, TB = MODE == kDW;
  constexpr int NW = WN * WM, KS = 64;
  constexpr int WTN = BN / WN, WTM = BM / WM, FN = WTN / 16, FM = WTM / 16;
  constexpr int IA = (BN / 8 + NW - 1) / NW * NW, IB = (BM / 8 + NW - 1) / NW * NW;
  constexpr int NA = IA / NW, NB = IB / NW, GA = (NA + 3) / 4, GB = (NB + 3) / 4, NI = NA + NB;
  constexpr int STAGE = (IA + IB) * 1024;
  constexpr int RA = BN * 2, RB = BM * 2;  // bytes of an LDS row of a "columns" operand
  static_assert(WTN % 32 == 0 && WTM % 32 == 0, "wave tile");
  static_assert(!TA || BN % 128 == 0, "columns: whole 64-byte pieces of four");
  static_assert(!TB || BM % 128 == 0, "columns: whole 64-byte pieces of four");
  static_assert(S >= 2 && (S - 1) * NI <= 63 && S * STAGE <= 160 * 1024, "ring");
  static_assert(S * STAGE == ring_bytes<BN, BM, NW, S>(), "the kernels' array");

  const int tid = threadIdx.x, lane = tid & 63;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  // A few tokens need no launch to number them: each block does, and copies from X itself.
  const bool direct = MODE == kSums && BM <= 128 && p.direct != 0;
  const int nv = direct ? vocab_number(p, wid, lane, NW, smem) : *p.nv;
  const int* const rowmap = reinterpret_cast<const int*>(smem);  // direct: token of a compact one
  const bool twice = nv <= p.twice;       // G in two parts of bf16
  const int rows = twice ? 2 * nv : nv;   // of G, and of X beside it
  const int64_t ext_b = MODE == kDW ? p.ids : (MODE == kDX ? rows : nv);
  const int64_t klen = MODE == kDW ? rows : (MODE == kDX ? p.ids : p.K);
  const int stages = (int)((klen + KS - 1) / KS);
  const bool stream = p.stream && (MODE == kDW ? rows <= 256 : ext_b <= BM);

  // An XCD takes one contiguous part of the tiles; groups of up to 8 B tiles share A tiles.
  const int tiles_b = (int)((ext_b + BM - 1) / BM);
  const int splits = MODE == kDX ? p.nv[1] : 1;
  const int tiles = p.tiles_a * tiles_b, total = tiles * splits, xcd = block & 7;
  const int end = (int)((int64_t)total * (xcd + 1) / 8);
  int cur = (int)((int64_t)total * xcd / 8) + (block >> 3);
  if (cur >= end) return;
  const int split = cur / tiles;
  cur -= split * tiles;
  int ta, tb;
  {
    const int b0 = cur / (8 * p.tiles_a) * 8, gb = tiles_b - b0 < 8 ? tiles_b - b0 : 8;
    cur -= b0 * p.tiles_a;
    tb = __builtin_amdgcn_readfirstlane(b0 + cur % gb);
    ta = __builtin_amdgcn_readfirstlane(cur / gb);
  }
  const int ks0 = __builtin_amdgcn_readfirstlane((int)((int64_t)stages * split / splits));
  const int nk = __builtin_amdgcn_readfirstlane((int)((int64_t)stages * (split + 1) / splits)) - ks0;

  const int wn = wid % WN, wm = wid / WN;
  const int lr = lane & 15, lg = lane >> 4;
  const int64_t a0 = (int64_t)ta * BN, b0 = (int64_t)tb * BM;

  // Copies. Lanes whose 16 bytes lie outside the operand take an offset past the
  // buffer: zeros.
  constexpr uint32_t kBig = 0x80000000u;
  const int ll = lane >> 3, pc = lane & 7;
  // The lane for code behind the products: what is computed from it stays there instead of
  // occupying registers during them.
  auto fresh_lane = [&]() QR_INLINE {
    int l = lane;
    asm volatile("" : "+v"(l));
    return l & 63;
  };
  // row of K (columns) or chunk of 8 elements of K (rows) that copy I of an operand takes
  auto rows_of = [&](int I, int& row, int& chunk) {
    row = I * 8 + ll;
    chunk = pc ^ ((row >> 1) & 7);
  };
  auto cols_of = [&](int I, int rowbytes, int& k, int& chunk) {
    const int cpr = rowbytes / 16;  // chunks of a row: 32 or 16
    k = I * (64 / cpr) + lane / cpr;
    chunk = (lane % cpr) ^ ((k & 3) << 2 | (k >> 3 & 1) << 1);
  };
  auto offset = [&](bool cols, int I, int rowbytes, int tile_rows, int64_t ld, int64_t left) {
    if (cols) {
      int k, c;
      cols_of(I, rowbytes, k, c);
      return c * 8 < left ? (uint32_t)(k * ld * 2 + c * 16) : kBig;
    }
    int r, c;
    rows_of(I, r, c);
    return r < tile_rows && r < left ? (uint32_t)(r * ld * 2 + c * 16) : kBig;
  };
  uint32_t oa[NA], ob[NB];
#pragma unroll
  for (int i = 0; i < NA; ++i)
    oa[i] = offset(TA, wid * NA + i, RA, BN, p.lda, p.ext_a - a0) - 1024u * (uint32_t)(i % 4);
#pragma unroll
  for (int i = 0; i < NB; ++i)
    ob[i] = offset(TB, wid * NB + i, RB, BM, p.ldb, ext_b - b0) - 1024u * (uint32_t)(i % 4);
  if constexpr (MODE == kSums) {
    if (direct) {
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        int r, c;
        rows_of(wid * NB + i, r, c);
        const uint32_t o = r < BM && r < nv - b0 ? (uint32_t)(rowmap[b0 + r] * p.ldb * 2 + c * 16) : kBig;
        ob[i] = o - 1024u * (uint32_t)(i % 4);
      }
    }
  }
  const uint16_t* const pa = (MODE == kDW && F16 ? p.Xh : p.A) + (TA ? a0 : a0 * p.lda);
  const uint16_t* const pb = p.B + (TB ? b0 : direct ? 0 : b0 * p.ldb);
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
  constexpr int NG = GA + GB;
  auto issue_group = [&](int g, int slot, int ks, bool inside) {
    const bool isA = g < GA, cols = isA ? TA : TB;
    const int i0 = (isA ? g : g - GA) * 4, n = isA ? NA : NB, cnt = n - i0 < 4 ? n - i0 : 4;
    const int I0 = wid * n + i0;
    const uint32_t lds = lds0 + (uint32_t)(slot * STAGE + ((isA ? 0 : IA) + I0) * 1024);
    const uint16_t* src = (isA ? pa : pb) + (cols ? (int64_t)ks * KS * (isA ? p.lda : p.ldb) : 0);
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc((void*)src, (short)0, 0x7ffffff0, kBufWord3);
    const int soff = cols ? 0 : ks * (KS * 2);
    uint32_t vo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + e < n ? i0 + e : 0;
      vo[e] = isA ? oa[i < NA ? i : 0] : ob[i < NB ? i : 0];
    }
    const int64_t left = klen - (int64_t)ks * KS;
    if (!inside && left < KS) {  // the last stage: K ends inside it
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        int a, c;
        if (cols) {
          cols_of(I0 + e, isA ? RA : RB, a, c);
        } else {
          rows_of(I0 + e, a, c);
          a = c * 8;
        }
        if (a >= left) vo[e] = kBig - 1024u * (uint32_t)e;
      }
    }
    if constexpr (MODE != kDW && HINT) {
      if (isA && stream) {
        if (cnt == 4) dma_group<4, true>(lds, vo, r, soff);
        else if (cnt == 3) dma_group<3, true>(lds, vo, r, soff);
        else if (cnt == 2) dma_group<2, true>(lds, vo, r, soff);
        else dma_group<1, true>(lds, vo, r, soff);
        return;
      }
    }
    if (cnt == 4) dma_group<4, false>(lds, vo, r, soff);
    else if (cnt == 3) dma_group<3, false>(lds, vo, r, soff);
    else if (cnt == 2) dma_group<2, false>(lds, vo, r, soff);
    else dma_group<1, false>(lds, vo, r, soff);
  };

  // Operand reads of K step h (32 elements): lane (lr, lg) takes row or column lr of a
  // fragment and elements 8 lg .. 8 lg + 7.
  const int tk = 8 * lg + (lr >> 2);  // columns: K row of the lane's address, and its byte's
  const int tc = 8 * (lr & 3), tx = (lr >> 2) << 6 | (lg & 1) << 5;
  auto read = [&](bool cols, const uint8_t* base, int w0, int i, int h, int rowbytes) {
    if (cols) {
      const uint8_t* s = base + (32 * h + tk) * rowbytes + (((w0 + 16 * i) * 2 + tc) ^ tx);
      typedef __attribute__((address_space(3))) v4s* lds_v4s;
      const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(s));
      const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(s + 4 * rowbytes));
      const v8s v = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
      return __builtin_bit_cast(v8b, v);
    }
    const int r = w0 + 16 * i + lr;
    return *reinterpret_cast<const v8b*>(base + r * 128 + (((4 * h + lg) ^ ((lr >> 1) & 7)) << 4));
  };
  v4f acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = v4f{};
  v8b fa[2][FN], fb[2][FM];  // operands of two K steps
  auto load_a = [&](const uint8_t* st, int h, int buf, int i) { fa[buf][i] = read(TA, st, wn * WTN, i, h, RA); };
  auto load_b = [&](const uint8_t* st, int h, int buf, int j) {
    fb[buf][j] = read(TB, st + IA * 1024, wm * WTM, j, h, RB);
  };
  auto load_ops = [&](const uint8_t* st, int h, int buf) {
#pragma unroll
    for (int i = 0; i < FN; ++i) load_a(st, h, buf, i);
#pragma unroll
    for (int j = 0; j < FM; ++j) load_b(st, h, buf, j);
  };
  // W in fp16, times its power of two: 20 instructions for a fragment (without the factor 12: 1.4% of 4096
  // tokens' gradient less). Converted a row ahead, among the products before, it takes as long.
  float half_scale = 1.0f;
  if constexpr (F16 && MODE == kDX)
    half_scale = __uint_as_float(__builtin_amdgcn_readfirstlane((int)__float_as_uint(ldexpf(1.0f, p.expo[0]))));
  auto to_half = [&](v8b x) QR_INLINE {
    const uint4 q = __builtin_bit_cast(uint4, x);
    auto pair = [&](uint32_t w) QR_INLINE {
      return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(bf16_lo(w) * half_scale, bf16_hi(w) * half_scale));
    };
    return __builtin_bit_cast(v8h, make_uint4(pair(q.x), pair(q.y), pair(q.z), pair(q.w)));
  };
  auto multiply_row = [&](int buf, int i) {
    if constexpr (F16) {
      v8h a;
      if constexpr (MODE == kDX) a = to_half(fa[buf][i]);
      else a = __builtin_bit_cast(v8h, fa[buf][i]);
#pragma unroll
      for (int j = 0; j < FM; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, __builtin_bit_cast(v8h, fb[buf][j]), acc[i][j], 0, 0, 0);
    } else {
#pragma unroll
      for (int j = 0; j < FM; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[buf][i], fb[buf][j], acc[i][j], 0, 0, 0);
    }
  };

  // Compact tokens of the lane, and where their lists enter the wave's ids.
  const int64_t id_lo = p.id0 + a0 + wn * WTN;
  const int own = (int)(p.ids - a0 - wn * WTN < WTN ? p.ids - a0 - wn * WTN : WTN);  // ids of the wave
  int tok[FM], ent[FM];  // ent: a list's one id, or its first entry that may be the wave's
  auto token = [&](int j) QR_INLINE {
    const int64_t c = b0 + wm * WTM + 16 * j + lr;
    tok[j] = c < nv ? (direct ? rowmap[c] : p.map[c]) : -1;
    ent[j] = kNone;
    if (tok[j] < 0 || own <= 0) return;
    if (p.L > 1) ent[j] = p.first[(int64_t)tok[j] * p.buckets + (id_lo >> p.shift)];
    else ent[j] = direct && p.target ? (int)p.target[tok[j]] : p.keys[tok[j]];
  };
  // before the products where registers allow
  constexpr bool EARLY = BM <= 128;
  if constexpr (EARLY && (MODE == kSums || MODE == kGrad)) {
#pragma unroll
    for (int j = 0; j < FM; ++j) token(j);
    if (direct) __syncthreads();  // the map's place is the ring's
  }
#pragma unroll
  for (int s = 0; s < S; ++s)
    if (s < nk) {
#pragma unroll
      for (int g = 0; g < NG; ++g) issue_group(g, s, ks0 + s, false);
    }

  // One stage. The next one opens when its copies have landed and no wave reads this one
  // any more (the last step's operands are in registers); its slot is refilled at once. The
  // three kinds of stage are bodies of their own: waits merged over a branch would be
  // those of the worst path.
  int cs = 0, it = 0;
  auto stage = [&](auto refill, auto last) {
    const int ns = cs + 1 == S ? 0 : cs + 1;
    const uint8_t *here = smem + cs * STAGE, *next = smem + ns * STAGE;
    // the next step's reads behind the first rows' products: RPR fragments a row
    constexpr int NF = FN + FM, RPR = (NF + (FN > 2 ? FN * 3 / 4 : FN) - 1) / (FN > 2 ? FN * 3 / 4 : FN);
    auto reads = [&](const uint8_t* st, int h, int buf, int row) QR_INLINE {
#pragma unroll
      for (int f = row * RPR; f < (row + 1) * RPR && f < NF; ++f) {
        if (f < FM) load_b(st, h, buf, f);
        else load_a(st, h, buf, f - FM);
      }
    };
#pragma unroll
    for (int i = 0; i < FN; ++i) {
      reads(here, 1, 1, i);
      multiply_row(0, i);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (!decltype(last)::value) {
      if constexpr (decltype(refill)::value != 0) wait_vm<(S - 2) * NI>();
      else wait_stages<NI, S - 2>(nk - 2 - it);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < (FN > NG ? FN : NG); ++i) {
      if (i < FN) {
        if constexpr (!decltype(last)::value) reads(next, 0, 0, i);
        multiply_row(1, i);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (decltype(refill)::value != 0) {
        if (i < NG) issue_group(i, cs, ks0 + it + S, decltype(refill)::value == 1);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    cs = ns;
  };
  if (nk > 0) {
    wait_stages<NI, S - 1>(nk - 1);
    __syncthreads();
    load_ops(smem, 0, 0);
    // refills: 1 of a whole stage, 2 of one that K may end in, 0 none
    for (; it < nk - S - 1; ++it) stage(std::integral_constant<int, 1>{}, std::false_type{});
    for (; it < nk - S; ++it) stage(std::integral_constant<int, 2>{}, std::false_type{});
    for (; it < nk - 1; ++it) stage(std::integral_constant<int, 0>{}, std::false_type{});
    stage(std::integral_constant<int, 0>{}, std::true_type{});
  }

  // Entries of the lists among the wave's ids: f(whether the lane has one, the entry, its
  // weight, its id's value among the fragment's). All lanes of the wave go along.
  auto hits = [&](int j, auto f) QR_INLINE {
    auto hit = [&](int64_t e, int key, float w) QR_INLINE {
      const int d = (int)(key - id_lo);
      const bool mine = key >= id_lo && key < id_lo + own && ((d >> 2) & 3) == lg;
      if (__any(mine)) f(mine, e, w, (d >> 4) * 4 + (d & 3));
    };
    if (p.L == 1) {
      hit(tok[j], ent[j], MODE == kGrad && p.wts && tok[j] >= 0 ? p.wts[tok[j]] : 1.0f);
      return;
    }
    const int64_t base = (int64_t)tok[j] * p.L;
    constexpr int U = 4;  // entries read at once: lists are dense where ids are frequent ones
    int e = tok[j] < 0 || own <= 0 ? p.L : ent[j];
    while (__any(e < p.L)) {
      int key[U];
      float w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool in = e + u < p.L;
        key[u] = in ? p.keys[base + e + u] : kNone;
        w[u] = MODE == kGrad && in ? p.wts[base + e + u] : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) hit(base + e + u, key[u], w[u]);
      e = key[U - 1] >= id_lo + own ? p.L : e + U;
    }
  };
  const float c2 = p.scale * kLog2e;

  // What follows takes a B fragment at a time: its values v[4 i + r], A side 16 i + 4 lg + r.
  auto values = [&](int j, float* v) QR_INLINE {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) v[4 * i + r] = acc[i][j][r];
  };
  auto beyond = [&](float* v, float to) QR_INLINE {  // ids that are not the piece's
    if (own >= WTN) return;
#pragma unroll
    for (int e = 0; e < 4 * FN; ++e) v[e] = 16 * (e >> 2) + 4 * lg + (e & 3) >= own ? to : v[e];
  };

  if constexpr (MODE == kSums) {
    // Base-2 maximum and sum of each token over the tile's ids. The logits' base-2 values are rounded
    // once, before the maximum is taken off (not by a fused multiply-add): what the sums hold and
    // what the list's ids keep in zl are the same numbers, so that the largest adds 1 exactly and no
    // log-probability comes out above 0 (with the fused form: 1.4e-6 at a logit of 100). 4096 tokens
    // of 131072 ids, 5120 wide, take as long, 257 of 100003 266 us for 264.
#pragma clang fp contract(off)
    __syncthreads();
    float2* red = reinterpret_cast<float2*>(smem);  // [WN][BM]
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      float v[4 * FN];
      values(j, v);
#pragma unroll
      for (int k = 0; k < 4 * FN; ++k) v[k] *= c2;
      if constexpr (!EARLY) token(j);
      hits(j, [&](bool mine, int64_t e, float, int reg) QR_INLINE {
        float z = 0.0f;
#pragma unroll
        for (int k = 0; k < 4 * FN; ++k) z = reg == k ? v[k] : z;
        if (mine) p.zl[e] = z;
      });
      beyond(v, -INFINITY);
      float m = -INFINITY, s = 0.0f;
#pragma unroll
      for (int k = 0; k < 4 * FN; ++k) m = fmaxf(m, v[k]);
      m = fmaxf(m, __shfl_xor(m, 16, 64));
      m = fmaxf(m, __shfl_xor(m, 32, 64));
      const float sub = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int k = 0; k < 4 * FN; ++k) s += __builtin_amdgcn_exp2f(v[k] - sub);
      s += __shfl_xor(s, 16, 64);
      s += __shfl_xor(s, 32, 64);
      if (lg == 0) red[wn * BM + wm * WTM + 16 * j + lr] = make_float2(m, s);
    }
    __syncthreads();
    for (int c = tid; c < BM; c += 64 * NW) {
      if (b0 + c >= nv) continue;
      float m = -INFINITY, s = 0.0f;
#pragma unroll
      for (int w = 0; w < WN; ++w) m = fmaxf(m, red[w * BM + c].x);
      const float sub = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int w = 0; w < WN; ++w) s += red[w * BM + c].y * __builtin_amdgcn_exp2f(red[w * BM + c].x - sub);
      p.part[(int64_t)ta * p.ldpart + b0 + c] = make_float2(m, s);
    }
  }

  if constexpr (MODE == kDX) {
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int64_t c = b0 + wm * WTM + 16 * j + lr;
      if (c >= ext_b) continue;
      float* row = p.out32 + ((int64_t)split * rows + c) * p.K;
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        const int64_t h = a0 + wn * WTN + 16 * i + 4 * lg;
        if (h >= p.K) continue;
        float4 o = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
        float4* d = reinterpret_cast<float4*>(row + h);
        if (p.add) {
          const float4 w = *d;
          o.x += w.x; o.y += w.y; o.z += w.z; o.w += w.w;
        }
        *d = o;
      }
    }
  }

  // bf16 outputs leave through the ring, each wave its own part, so that stores run along
  // the B side's rows, 16 bytes a lane.
  if constexpr (MODE == kGrad || MODE == kDW) {
    __syncthreads();
    const int l = fresh_lane();
    constexpr int LD = WTN * 2 + 16, CPR = WTN / 8;
    static_assert(NW * 16 * LD <= S * STAGE, "a fragment per wave fits");
    uint8_t* so = smem + wid * (16 * LD);
    const int64_t row0 = b0 + wm * WTM, lim = MODE == kGrad ? nv : p.ids;
    const int64_t col0 = a0 + wn * WTN, left = MODE == kGrad ? WTN : p.K - col0;
    auto rows_out = [&](int j, const float* v, uint16_t* out, auto nt, auto half) QR_INLINE {
      auto pair = [&](float x, float y) QR_INLINE {
        if constexpr (decltype(half)::value) return half_pair(x, y);
        else return bf16_pair(x, y);
      };
#pragma unroll
      for (int i = 0; i < FN; ++i)
        *reinterpret_cast<uint2*>(so + (l & 15) * LD + (16 * i + 4 * (l >> 4)) * 2) =
            make_uint2(pair(v[4 * i], v[4 * i + 1]), pair(v[4 * i + 2], v[4 * i + 3]));
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int k = 0; k < 16 * CPR / 64; ++k) {
        const int c = l + 64 * k, ml = c / CPR, nl = 8 * (c % CPR);
        const int64_t m = row0 + 16 * j + ml;
        if (m >= lim || nl >= left) continue;
        typedef uint32_t u4 __attribute__((ext_vector_type(4)));
        const u4 q = *reinterpret_cast<const u4*>(so + ml * LD + nl * 2);
        u4* dst = reinterpret_cast<u4*>(out + m * p.ldo + col0 + nl);
        if constexpr (decltype(nt)::value) __builtin_nontemporal_store(q, dst);
        else *dst = q;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };
    const int kx = MODE == kDW && F16 ? -__builtin_amdgcn_readfirstlane(p.expo[1]) : 0;
    auto all_out = [&](auto nt) QR_INLINE {
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        float v[4 * FN];
        values(j, v);
        if constexpr (MODE == kGrad) {
          // G in fp32, in two parts of bf16 (its rounding and what that left: 2^-16 of each element), or
          // H for fp16 (2^-11 of each, 2^-39 of the list's weight where that is more).
          if constexpr (!EARLY) token(j);
          float gt = 0.0f, ga = 0.0f, l2 = 0.0f, mass = 1.0f;
          if (tok[j] >= 0) {
            if (p.mass) mass = p.mass[tok[j]];
            if (twice) {
              gt = p.g[tok[j]] * p.scale * p.sign;
              ga = gt * mass;
            } else {
              ga = mass > 0.0f ? (float)(1 << kHalf) : 0.0f;
            }
            l2 = p.lse[tok[j]] * kLog2e;
          }
#pragma unroll
          for (int k = 0; k < 4 * FN; ++k) v[k] = ga * __builtin_amdgcn_exp2f(__builtin_fmaf(v[k], c2, -l2));
          beyond(v, 0.0f);
          hits(j, [&](bool mine, int64_t, float w, int reg) QR_INLINE {
            const float b = !mine ? 0.0f : twice ? gt * w : ga == 0.0f ? 0.0f : w / mass * ga;
#pragma unroll
            for (int k = 0; k < 4 * FN; ++k) v[k] -= reg == k ? b : 0.0f;
          });
          if (!twice) {
            rows_out(j, v, p.out16, nt, std::true_type{});
            continue;
          }
        }
        if constexpr (MODE == kDW && F16) {
#pragma unroll
          for (int k = 0; k < 4 * FN; ++k) v[k] = __builtin_ldexpf(v[k], kx);
        }
        rows_out(j, v, p.out16, nt, std::false_type{});
        if constexpr (MODE == kGrad) {
#pragma unroll
          for (int k = 0; k < 4 * FN; ++k) v[k] -= __uint_as_float(bf16_pair(0.0f, v[k]) & 0xffff0000u);
          rows_out(j, v, p.out16 + nv * p.ldo, nt, std::false_type{});
        }
      }
    };
    // (the branch around the loop: around the store the two are merged, without nt)
    if (MODE == kDW && stream) all_out(std::true_type{});
    else all_out(std::false_type{});
  }
}

// Copies that may carry the non-temporal hint take a branch each: tiles of 256 tokens have a body with
// it for where one holds all that count (log-probabilities of 200 tokens of 131072 ids, 3584 wide,
// 239 -> 230 us), and one without (4096 tokens: 1% faster).
template <int MODE, int BN, int BM, int WN, int WM, int S>
__device__ __forceinline__ void vocab_tile(const VocabTile& p, int block, uint8_t* smem) {
  auto body = [&](auto half) QR_INLINE {
    constexpr bool F16 = decltype(half)::value;
    if constexpr (F16 && MODE == kDX && BM == 128) {
      // one wave converts a fragment of W instead of two (gradient of 300 tokens of 131072 ids 1369 -> 1278 us)
      vocab_tile_body<MODE, BN, BM, 8, 1, S, true, F16>(p, block, smem);
    } else if constexpr (MODE == kDW || BM <= 128) {
      vocab_tile_body<MODE, BN, BM, WN, WM, S, true, F16>(p, block, smem);
    } else {
      const int nv = *p.nv, rows = MODE == kDX && nv <= p.twice ? 2 * nv : nv;
      if (p.stream && rows <= BM) vocab_tile_body<MODE, BN, BM, WN, WM, S, true, F16>(p, block, smem);
      else vocab_tile_body<MODE, BN, BM, WN, WM, S, false, F16>(p, block, smem);
    }
  };
  if constexpr (MODE == kDW || (MODE == kDX && BM > 64)) {  // (64 rows: two parts of up to 32 tokens)
    if (*p.nv > p.twice) {
      body(std::true_type{});
      return;
    }
  }
  body(std::false_type{});
}

template <int MODE, int BN, int BM, int WN, int WM, int S>
__global__ __launch_bounds__(64 * WN * WM, 1) void vocab_tile_kernel(const VocabTile p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[ring_bytes<BN, BM, WN * WM, S>()];
  vocab_tile<MODE, BN, BM, WN, WM, S>(p, blockIdx.x, smem);
}

// The logits' tiles of 256 x 256 are planned for all tokens; where few of them count, tiles of
// 256 x 128 take less time (a round of the CUs 0.6 of the other's), if the launch has blocks for them:
// log-probabilities of 200 of 2048 tokens, 32768 ids, 3584 wide, 63 us and 83 without, 120 of 250, 131072 ids,
// 162 and 225.
template <int MODE>
__global__ __launch_bounds__(512, 1) void vocab_wide_kernel(const VocabTile p) {
  constexpr int A = ring_bytes<256, 256, 8, 2>(), C = ring_bytes<256, 128, 8, 3>();
  __shared__ __attribute__((aligned(1024))) uint8_t smem[A > C ? A : C];
  const uint32_t nv = (uint32_t)*p.nv, a = (uint32_t)p.tiles_a;
  const uint32_t half = a * ((nv + 127) / 128), whole = a * ((nv + 255) / 256);
  if (half <= gridDim.x && (half + 255) / 256 * 2 < (whole + 255) / 256 * 3)
    vocab_tile<MODE, 256, 128, 4, 2, 3>(p, blockIdx.x, smem);
  else
    vocab_tile<MODE, 256, 256, 4, 2, 2>(p, blockIdx.x, smem);
}

// A piece's part of dX (the first `dx_blocks` blocks) and rows of dW in one launch: dX has
// few tiles of many stages, which seldom fill the CUs, dW many of few (gradients: 9% less time than in two
// launches at 2048 tokens of 131072 ids, 5120 wide, 20% at 64 of 5000, 1024 wide).
template <int BM, int WN, int WM, int S>
__global__ __launch_bounds__(512, 1) void vocab_grads_kernel(const VocabTile x, const VocabTile w, int dx_blocks) {
  static_assert(WN * WM == 8, "one block size");
  constexpr int A = ring_bytes<256, BM, 8, S>(), C = ring_bytes<256, 256, 8, 2>();
  __shared__ __attribute__((aligned(1024))) uint8_t smem[A > C ? A : C];
  if ((int)blockIdx.x < dx_blocks) vocab_tile<kDX, 256, BM, WN, WM, S>(x, blockIdx.x, smem);
  else vocab_tile<kDW, 256, 256, 4, 2, 2>(w, blockIdx.x - dx_blocks, smem);
}

// Sums of the tiles' parts, a wave a compact token: lse, and sum_j p (log p - (z_j - lse))
// (with wts) or z - lse. Float64, fixed order. The parts are in base 2, logits times
// c2 = fp32(scale log2 e): z = x scale / c2 takes that rounding back out. z_j - lse is formed in base
// 2, where it is at most 0: x_j is at most the maximum, and the sum at least 1.
__global__ __launch_bounds__(256) void vocab_finish_kernel(const VocabTile p, float* __restrict__ value,
                                                           float* __restrict__ lse) {
  const float2* __restrict__ const part = p.part;
  const float* __restrict__ const wts = p.wts;
  const float* __restrict__ const zl = p.zl;
  const int* __restrict__ const keys = p.keys;
  const int tiles = p.tiles_a, L = p.L, lane = threadIdx.x & 63;
  const int64_t ldpart = p.ldpart;
  int64_t c = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), t = c;
  if (p.direct) {  // a wave a token, which counts those before its own
    if (t >= p.direct) return;
    c = 0;
    bool mine = false;
    for (int i = lane; i <= t; i += 64) {
      const bool live = vocab_live(p.target, p.keys, L, p.N, i);
      c += live && i < t;
      mine |= live && i == t;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) c += __shfl_xor((int)c, o, 64);
    if (!__any(mine)) {
      if (lane == 0) value[t] = lse[t] = 0.0f;
      return;
    }
  } else {
    if (c >= *p.nv) return;
    t = p.map[c];
  }
  float m = -INFINITY;
  double s = 0.0;
  constexpr int U = 8;
  for (int i0 = lane; i0 < tiles; i0 += 64 * U) {
    float2 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      v[u] = i0 + 64 * u < tiles ? part[(int64_t)(i0 + 64 * u) * ldpart + c] : make_float2(-INFINITY, 0.0f);
    float top = m;
#pragma unroll
    for (int u = 0; u < U; ++u) top = fmaxf(top, v[u].x);
    const float sub = top == -INFINITY ? 0.0f : top;
    s *= (double)exp2f(m - sub);
#pragma unroll
    for (int u = 0; u < U; ++u) s += (double)(v[u].y * exp2f(v[u].x - sub));
    m = top;
  }
  const float top = wave_max(m);
  s *= (double)exp2f(m - (top == -INFINITY ? 0.0f : top));
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
  const double nat = (double)p.scale / (double)(p.scale * kLog2e);  // z of a base-2 logit
  const double rest = log2(s) * kLn2, total = (double)top * nat + rest;
  double v = 0.0;
  if (wts) {
    for (int j = lane; j < L; j += 64) {
      const double w = (double)wts[t * L + j];
      const double z = ((double)zl[t * L + j] - (double)top) * nat - rest;
      if (keys[t * L + j] != kNone && w != 0.0) v += w * (log(w) - z);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  } else {
    v = ((double)zl[t] - (double)top) * nat - rest;
  }
  if (lane == 0) {
    value[t] = (float)v;
    lse[t] = (float)total;
  }
}

// dX of all tokens: the splits' sums in order (a split's parts of G one after the other),
// times what fp16 products leave out, rounded once; zeros for masked tokens. A block takes 256 values of a
// token, its waves (at most kDxWaves) a run of the sums each, eight at once, which are added in order.
constexpr int kDxWaves = 8;
__global__ __launch_bounds__(64 * kDxWaves) void vocab_dx_kernel(const float* __restrict__ part, int64_t K,
                                                                 const int* __restrict__ inv,
                                                                 const int* __restrict__ nv, int twice,
                                                                 const float* __restrict__ factor,
                                                                 const int* __restrict__ expo,
                                                                 uint16_t* __restrict__ dX, int64_t lddx) {
  __shared__ float4 red[kDxWaves][64];
  const int64_t t = blockIdx.x, c = inv[t], h = 256 * (int64_t)blockIdx.y + 4 * threadIdx.x;
  const int n = nv[0], parts = n <= twice ? 2 : 1, sums = nv[1] * parts;
  const int64_t rows = (int64_t)n * parts;
  const int waves = blockDim.y, wave = threadIdx.y;
  const int run = (sums + waves - 1) / waves, end = run * (wave + 1) < sums ? run * (wave + 1) : sums;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (c >= 0 && h < K) {
    constexpr int U = 8;
    for (int s0 = run * wave; s0 < end; s0 += U) {
      float4 a[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int s = s0 + u < end ? s0 + u : end - 1;
        const int64_t row = (parts == 2 ? s >> 1 : s) * rows + c + (parts == 2 ? (s & 1) * n : 0);
        a[u] = *reinterpret_cast<const float4*>(part + row * K + h);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool in = s0 + u < end;
        v.x += in ? a[u].x : 0.0f; v.y += in ? a[u].y : 0.0f;
        v.z += in ? a[u].z : 0.0f; v.w += in ? a[u].w : 0.0f;
      }
    }
  }
  if (waves > 1) {
    red[wave][threadIdx.x] = v;
    __syncthreads();
    if (wave > 0) return;
    for (int w = 1; w < waves; ++w) {
      const float4 o = red[w][threadIdx.x];
      v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
    }
  }
  if (c >= 0 && n > twice) {  // the sums are of fp16 products
    const float f = factor[c];
    const int k = -expo[0];
    v = make_float4(ldexpf(v.x * f, k), ldexpf(v.y * f, k), ldexpf(v.z * f, k), ldexpf(v.w * f, k));
  }
  if (h < K) *reinterpret_cast<uint2*>(dX + t * lddx + h) = make_uint2(bf16_pair(v.x, v.y), bf16_pair(v.z, v.w));
}

// dW where there are no tokens at all.
__global__ __launch_bounds__(256) void vocab_zero_kernel(uint16_t* __restrict__ dW, int64_t ld, int64_t K) {
  for (int64_t i = threadIdx.x; i < K >> 3; i += 256)
    *reinterpret_cast<uint4*>(dW + blockIdx.x * ld + 8 * i) = make_uint4(0u, 0u, 0u, 0u);
}

// ---------------------------------------------------------------------------
// Plans and launches
// ---------------------------------------------------------------------------
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

constexpr int64_t kMaxBlocks = (int64_t)1 << 21;
constexpr int64_t kMall = (int64_t)256 << 20, kL2s = (int64_t)32 << 20;

int64_t grad_rows(int64_t M) { return M <= kTwice ? 2 * M : (M < 2 * kTwice ? 2 * kTwice : M); }

// Blocks of a product, a multiple of 8 (an XCD's share each). dX: its splits give 256 at most.
template <int MODE>
int64_t product_blocks(VocabTile& p, int64_t max_b, int BN, int BM) {
  p.tiles_a = (int)ceil_div(p.ext_a, BN);
  const int64_t tiles = p.tiles_a * ceil_div(max_b, BM);
  return MODE == kDX && tiles < 256 ? 256 : ceil_div(tiles, 8) * 8;
}

template <int MODE, int BN, int BM, int WN, int WM, int S>
hipError_t launch_one(VocabTile p, int64_t max_b, hipStream_t st) {
  const dim3 grid((unsigned)product_blocks<MODE>(p, max_b, BN, BM));
  hipLaunchKernelGGL((vocab_tile_kernel<MODE, BN, BM, WN, WM, S>), grid, dim3(64 * WN * WM), 0, st, p);
  return hipGetLastError();
}

// rows: of dX, or 0 for dW alone.
template <int BM, int WN, int WM, int S>
hipError_t launch_grads(VocabTile x, VocabTile w, int64_t rows, hipStream_t st) {
  const int64_t nx = rows ? product_blocks<kDX>(x, rows, 256, BM) : 0, nw = product_blocks<kDW>(w, w.ids, 256, 256);
  hipLaunchKernelGGL((vocab_grads_kernel<BM, WN, WM, S>), dim3((unsigned)(nx + nw)), dim3(512), 0, st, x, w, (int)nx);
  return hipGetLastError();
}

// Tiles of the logits' products, and what a round of them takes: us a stage and beside
// the stages, measured where the matrix cores and copies bind. Sums on every tile in turn (us, one
// card, 3584 wide; what memory bounds takes the same on every tile that holds all tokens):
//                              64 x 32   64   128   256 x 32   64   128   256
//   1 token of 131072 ids          151  146   184        145  145   154   211
//   64 tokens of 5000 ids           23   27    33         46   51    57    91
//   64 of 131072                   244  174   199        205  148   155   222
//   257 of 100003                  627  378   372        617  342   283   356
//   1024 of 32768                  543  402   341        582  320   231   192
struct LogitTile {
  int bn, bm;     // ids, tokens
  int per_round;  // tiles that the CUs hold at once
  float stage, base;
};
const LogitTile kLogitTiles[] = {
    {64, 32, 512, 0.375f, 2.0f}, {64, 64, 512, 0.44f, 3.0f},  {64, 128, 512, 0.66f, 4.0f}, {256, 32, 256, 0.66f, 3.0f},
    {256, 64, 256, 0.73f, 4.0f}, {256, 128, 256, 0.98f, 7.0f}, {256, 256, 256, 1.5f, 11.0f},
};

const LogitTile& logit_tile(int64_t M, int64_t N, int64_t K) {
  const LogitTile* best = nullptr;
  float least = 0.0f;
  for (const LogitTile& t : kLogitTiles) {
    const int64_t tiles = ceil_div(N, t.bn) * ceil_div(M, t.bm);
    const float cost = (float)ceil_div(tiles, t.per_round) * (t.stage * (float)ceil_div(K, 64) + t.base);
    if (!best || cost < least) {
      best = &t;
      least = cost;
    }
  }
  return *best;
}

template <int MODE>
hipError_t launch_logits(const VocabTile& p, const LogitTile& t, int64_t M, hipStream_t st) {
  if (t.bn == 64) {
    if (t.bm == 32) return launch_one<MODE, 64, 32, 2, 1, 6>(p, M, st);
    if (t.bm == 64) return launch_one<MODE, 64, 64, 2, 2, 5>(p, M, st);
    return launch_one<MODE, 64, 128, 2, 2, 3>(p, M, st);
  }
  switch (t.bm) {
    case 32: return launch_one<MODE, 256, 32, 8, 1, 4>(p, M, st);
    case 64: return launch_one<MODE, 256, 64, 4, 2, 3>(p, M, st);
    case 128: return launch_one<MODE, 256, 128, 4, 2, 3>(p, M, st);
    default: break;
  }
  VocabTile w = p;
  const int64_t blocks = product_blocks<MODE>(w, M, 256, 256);
  hipLaunchKernelGGL((vocab_wide_kernel<MODE>), dim3((unsigned)(blocks < 256 ? 256 : blocks)), dim3(512), 0, st, w);
  return hipGetLastError();
}

// Rows of G (twice the tokens where it is held in two parts) in a tile of dX: the fewest that hold all, up to 64
// (16 tokens of 32768 ids, 3584 wide: 86 us, on 128 rows 88; 32 rows gain nothing), else the
// cheaper by measured costs of 128 and 256 (us, dX with its logits, 3584 wide, 128 | 256; in two parts of
// bf16: 33 tokens of 32768 92 | 97, 128 of 131072 446 | 446, with dW 761 | 735; in fp16: 200 of 32768 162 | 175, 257
// of 100003 655 | 706, 512 of 131072 1101 | 1050, 600 of 32768 356 | 365, 700 378 | 379, 2048 of
// 131072, 5120 wide, 6300 | 5979).
int dx_tile(int64_t rows) {
  if (rows <= 64) return 64;
  return ceil_div(rows, 128) * 55 < ceil_div(rows, 256) * 92 ? 128 : 256;
}

hipError_t launch_dx(const VocabTile& x, int64_t rows, hipStream_t st) {
  switch (dx_tile(rows)) {
    case 64: return launch_one<kDX, 256, 64, 4, 2, 3>(x, rows, st);
    case 128: return launch_one<kDX, 256, 128, 4, 2, 3>(x, rows, st);
    default: return launch_one<kDX, 256, 256, 4, 2, 2>(x, rows, st);
  }
}

hipError_t launch_both(const VocabTile& x, const VocabTile& w, int64_t rows, hipStream_t st) {
  switch (dx_tile(rows)) {
    case 64: return launch_grads<64, 4, 2, 3>(x, w, rows, st);
    case 128: return launch_grads<128, 4, 2, 3>(x, w, rows, st);
    default: return launch_grads<256, 4, 2, 2>(x, w, rows, st);
  }
}

struct Layout {
  size_t nv, map, inv, keys, wts, mass, first, zl, xc, part, g, dx, factor, top, peaks, expo, xh, bytes;
  int buckets, shift;  // of ids, for lists
  int64_t piece;  // ids of a piece of the gradient
  DxPlan sums;
};

Layout layout(int64_t M, int64_t N, int64_t K, int64_t L, bool lists, bool grad) {
  Layout w = {};
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += align256(n);
    return o;
  };
  w.nv = take(8);
  w.map = take((size_t)M * 4);
  w.inv = take((size_t)M * 4);
  w.keys = take((size_t)(M * L) * 4);
  if (lists) {
    w.wts = take((size_t)(M * L) * 4);
    w.mass = take((size_t)M * 4);
    // buckets of 64 ids or more, four for an entry
    w.shift = 6;
    while (ceil_div(N, (int64_t)1 << w.shift) > 4 * L) ++w.shift;
    w.buckets = (int)ceil_div(N, (int64_t)1 << w.shift);
    w.first = take((size_t)(M * w.buckets) * 2);
  }
  const int64_t rows = grad ? grad_rows(M) : M;
  w.xc = take((size_t)(rows * K) * 2);
  if (!grad) {
    w.zl = take((size_t)(M * L) * 4);
    w.part = take((size_t)(ceil_div(N, logit_tile(M, N, K).bn) * M) * 8);
  } else {
    // G of a piece: 256 MiB, between 4096 ids and all of them
    const int64_t want = ((int64_t)128 << 20) / rows / 256 * 256;
    w.piece = want < 4096 ? 4096 : want;
    if (w.piece > N) w.piece = ceil_div(N, 256) * 256;
    DxPlan& d = w.sums;
    d.bm = dx_tile(rows);
    d.tiles_a = (int)ceil_div(K, 256);
    d.stages = (int)(w.piece / 64);
    d.worth = (float)d.stages * (d.bm <= 64 ? 0.4f : d.bm <= 128 ? 0.6f : 1.0f) * 5.0e5f / (float)K;
    d.cap = 0x7fffffff;
    // room for the splits of all tokens and of fewer
    int64_t cap = rows;
    for (int64_t n = d.bm < rows ? d.bm : rows;; n = 2 * n < rows ? 2 * n : rows) {
      const int64_t sums = n * d.splits(n);
      cap = sums > cap ? sums : cap;
      if (n == rows) break;
    }
    d.cap = (int)cap;
    w.g = take((size_t)(rows * w.piece) * 2);
    w.dx = take((size_t)(cap * K) * 4);
    if (M > kTwice) {  // fp16
      w.factor = take((size_t)M * 4);
      w.top = take((size_t)M * 4);
      w.peaks = take((size_t)kPeaks * 4);
      w.expo = take(8);
      w.xh = take((size_t)(M * K) * 2);
    }
  }
  w.bytes = at;
  return w;
}

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

// Lists, compact tokens and their rows.
hipError_t prepare(const VocabArgs& p, const Layout& w, void* ws, bool direct, hipStream_t st) {
  if (p.index) {
    const dim3 grid((unsigned)ceil_div(p.M, 4));
    const size_t lds = (size_t)(ceil_div(p.L, 4) * 4) * 12 * sizeof(int);
    if (p.teacher_bf16)
      hipLaunchKernelGGL((vocab_list_kernel<true>), grid, dim3(256), lds, st, p.index, p.teacher, p.teacher_lse,
                         p.M, p.N, (int)p.L, p.scale, at<int>(ws, w.keys), at<float>(ws, w.wts),
                         at<float>(ws, w.mass), at<uint16_t>(ws, w.first), w.buckets, w.shift);
    else
      hipLaunchKernelGGL((vocab_list_kernel<false>), grid, dim3(256), lds, st, p.index, p.teacher, p.teacher_lse,
                         p.M, p.N, (int)p.L, p.scale, at<int>(ws, w.keys), at<float>(ws, w.wts),
                         at<float>(ws, w.mass), at<uint16_t>(ws, w.first), w.buckets, w.shift);
  }
  if (direct) return hipGetLastError();
  VocabCompact c = {};
  c.target = p.index ? nullptr : p.target;
  c.keys = at<int>(ws, w.keys);
  c.L = (int)p.L;
  c.M = p.M; c.N = p.N; c.K = p.K; c.ldx = p.ldx;
  c.X = p.X;
  c.Xc = at<uint16_t>(ws, w.xc);
  c.twice = p.lse_out ? -1 : kTwice;
  if (!p.lse_out && p.M > kTwice) {
    c.g = p.g;
    c.mass = p.index ? at<float>(ws, w.mass) : nullptr;
    c.gscale = p.index ? p.scale : -p.scale;
    c.factor = at<float>(ws, w.factor);
    c.top = at<float>(ws, w.top);
  }
  c.dx = w.sums;
  c.nv = at<int>(ws, w.nv);
  c.map = at<int>(ws, w.map);
  c.inv = at<int>(ws, w.inv);
  c.value = p.value;
  c.lse = p.lse_out;
  if (c.factor && p.dX) {  // fp16 products, if so many tokens count
    c.W = p.W;
    c.ldw = p.ldw;
    while (c.shift < 8 && ((int64_t)1 << c.shift) < p.K >> 3) ++c.shift;  // threads of a row
    const int64_t blocks = ceil_div(p.N, 256 >> c.shift);
    c.peak_blocks = (int)(blocks < kPeaks ? blocks : kPeaks);
    c.peaks = at<float>(ws, w.peaks);
    c.stream = p.N * p.K * 2 > kMall;
  }
  const dim3 grid((unsigned)(p.M + c.peak_blocks));
  if (p.M <= kVocabCount) {
    hipLaunchKernelGGL(vocab_compact_kernel, grid, dim3(256), 0, st, c);
  } else {
    hipLaunchKernelGGL(vocab_scan_kernel, dim3(1), dim3(1024), 0, st, c);
    hipLaunchKernelGGL(vocab_gather_kernel, grid, dim3(256), 0, st, c);
  }
  if (c.factor)
    hipLaunchKernelGGL(vocab_half_kernel, dim3((unsigned)(p.M < 1024 ? p.M : 1024)), dim3(256), 0, st, c.Xc, p.K,
                       c.factor, c.top, c.peaks, c.peak_blocks, c.nv, c.twice, at<int>(ws, w.expo),
                       p.dW ? at<uint16_t>(ws, w.xh) : nullptr);
  return hipGetLastError();
}

VocabTile common(const VocabArgs& p, const Layout& w, void* ws) {
  VocabTile t = {};
  t.nv = at<int>(ws, w.nv);
  t.K = p.K;
  t.map = at<int>(ws, w.map);
  t.keys = at<int>(ws, w.keys);
  if (p.index) {
    t.wts = at<float>(ws, w.wts);
    t.mass = at<float>(ws, w.mass);
    t.first = at<uint16_t>(ws, w.first);
    t.buckets = w.buckets;
    t.shift = w.shift;
  }
  t.L = (int)p.L;
  t.scale = p.scale;
  t.twice = p.lse_out ? -1 : kTwice;
  t.expo = at<int>(ws, w.expo);
  return t;
}

}  // namespace

size_t vocab_ws_bytes(int64_t M, int64_t N, int64_t K, int64_t L, bool lists, bool grad) {
  return M == 0 ? 0 : layout(M, N, K, L, lists, grad).bytes;
}

void vocab_plan(int64_t M, int64_t N, int64_t K, int* ids, int* tokens, int* rows, int64_t* piece) {
  const Layout w = layout(M, N, K, 1, false, true);
  const LogitTile& t = logit_tile(M, N, K);
  *ids = t.bn;
  *tokens = t.bm;
  *rows = dx_tile(grad_rows(M));
  *piece = w.piece < N ? w.piece : N;
}

hipError_t launch_vocab_loss(const VocabArgs& p, void* ws, hipStream_t st) {
  const Layout w = layout(p.M, p.N, p.K, p.L, p.index != nullptr, false);
  const LogitTile& tile = logit_tile(p.M, p.N, p.K);
  const bool direct = p.M <= kVocabDirect && tile.bm <= 128;
  hipError_t e = prepare(p, w, ws, direct, st);
  if (e != hipSuccess) return e;
  VocabTile t = common(p, w, ws);
  t.lda = p.ldw;
  t.direct = direct ? (int)p.M : 0;
  t.target = p.index ? nullptr : p.target;
  t.N = p.N;
  t.B = direct ? p.X : at<uint16_t>(ws, w.xc);
  t.ldb = direct ? p.ldx : p.K;
  t.ldpart = p.M;
  t.zl = at<float>(ws, w.zl);
  t.stream = true;
  float2* const part = at<float2>(ws, w.part);
  // a launch's blocks times their threads stay in 32 bits
  const int64_t ids = kMaxBlocks / ceil_div(p.M, tile.bm) * tile.bn;
  for (int64_t id0 = 0; id0 < p.N; id0 += ids) {
    t.id0 = id0;
    t.A = p.W + id0 * p.ldw;
    t.ext_a = t.ids = p.N - id0 < ids ? p.N - id0 : ids;
    t.part = part + id0 / tile.bn * t.ldpart;
    if ((e = launch_logits<kSums>(t, tile, p.M, st)) != hipSuccess) return e;
  }
  t.part = part;
  t.tiles_a = (int)ceil_div(p.N, tile.bn);
  hipLaunchKernelGGL(vocab_finish_kernel, dim3((unsigned)ceil_div(p.M, 4)), dim3(256), 0, st, t, p.value, p.lse_out);
  return hipGetLastError();
}

hipError_t launch_vocab_grad(const VocabArgs& p, void* ws, hipStream_t st) {
  if (p.M == 0) {
    if (p.dW) hipLaunchKernelGGL(vocab_zero_kernel, dim3((unsigned)p.N), dim3(256), 0, st, p.dW, p.lddw, p.K);
    return hipGetLastError();
  }
  const Layout w = layout(p.M, p.N, p.K, p.L, p.index != nullptr, true);
  hipError_t e = prepare(p, w, ws, false, st);
  if (e != hipSuccess) return e;
  uint16_t* G = at<uint16_t>(ws, w.g);
  const int64_t rows = grad_rows(p.M);
  for (int64_t id0 = 0; id0 < p.N; id0 += w.piece) {
    const int64_t ids = p.N - id0 < w.piece ? p.N - id0 : w.piece;
    VocabTile t = common(p, w, ws);
    t.A = p.W + id0 * p.ldw;
    t.lda = p.ldw;
    t.B = at<uint16_t>(ws, w.xc);
    t.ldb = p.K;
    t.ext_a = t.ids = ids;
    t.id0 = id0;
    t.lse = p.lse;
    t.g = p.g;
    t.sign = p.index ? 1.0f : -1.0f;
    t.out16 = G;
    t.ldo = w.piece;
    const LogitTile& tile = logit_tile(p.M, ids, p.K);
    t.stream = !p.dX || ids * p.K * 2 > kMall;
    if ((e = launch_logits<kGrad>(t, tile, p.M, st)) != hipSuccess) return e;
    VocabTile x = t, y = t;  // dX, dW
    x.B = y.B = G;
    x.ldb = y.ldb = w.piece;
    x.ext_a = y.ext_a = p.K;
    x.out32 = at<float>(ws, w.dx);
    x.add = id0 > 0;
    x.stream = ids * p.K * 2 > kL2s;
    y.stream = true;
    y.A = at<uint16_t>(ws, w.xc);
    y.lda = p.K;
    y.Xh = at<uint16_t>(ws, w.xh);
    y.out16 = p.dW + (p.dW ? id0 * p.lddw : 0);
    y.ldo = p.lddw;
    if (p.dX && p.dW) e = launch_both(x, y, rows, st);
    else if (p.dX) e = launch_dx(x, rows, st);
    else e = launch_grads<64, 4, 2, 3>(x, y, 0, st);
    if (e != hipSuccess) return e;
  }
  if (p.dX) {
    // Waves for the splits where all tokens count. Where few of many do, the GPU takes more splits and a wave
    // adds up as many as 128 sums (gradient of 131072 ids, 1024 wide, 5 tokens alone 2 x 64 sums on eight
    // waves; 5 of 4096 229 us, with eight waves 215), but waves that a launch has for that case only cost more
    // than they save where all count (4096 tokens of 5000 ids, 3584 wide, 405 -> 426 us, 2048, 1024 wide,
    // 95 -> 98), and sums read 16 or 32 at once gain nothing (229 -> 226 - 232).
    const int splits = w.sums.splits(rows);
    const int waves = splits <= 4 ? 1 : splits <= 4 * kDxWaves ? (splits + 3) / 4 : kDxWaves;
    hipLaunchKernelGGL(vocab_dx_kernel, dim3((unsigned)p.M, (unsigned)ceil_div(p.K, 256)), dim3(64, (unsigned)waves),
                       0, st, at<float>(ws, w.dx), p.K, at<int>(ws, w.inv), at<int>(ws, w.nv),
                       kTwice, at<float>(ws, w.factor), at<int>(ws, w.expo), p.dX, p.lddx);
  }
  return hipGetLastError();
}

}  // namespace qr
