// C ABI of the MXFP4 operators and the block norms (declared and documented in
// include/qurl_w8a8.h). As for the other entry points, arguments are validated on
// the host before anything is enqueued, and nothing here synchronizes.
#include <cmath>
#include <cstring>

#include "qr_internal.h"
#include "qurl_w8a8.h"

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;
constexpr int64_t kMaxCodeBytes = ((int64_t)1 << 31) - ((int64_t)1 << 16);

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
bool is_mx(int fmt) { return fmt == QR_ACT_MXFP8 || fmt == QR_ACT_MXFP4; }
bool in_range(int64_t v) { return v >= 0 && v < kMaxDim; }

int done(hipError_t e, const char* fn) { return qr::hip_error(e, fn); }

// Bytes of a row of K token codes, and of the panels of `rows` rows' scales.
int64_t code_row_bytes(int64_t K, int fmt) { return fmt == QR_ACT_MXFP4 ? K / 2 : K; }
int64_t scale_bytes(int64_t rows, int64_t K) { return (K + 127) / 128 * rows * 4; }

// Shape checks of the product. Returns QR_OK or an error.
int check_product(const char* fn, int64_t M, int64_t N, int64_t K, int xfmt) {
  if (!is_mx(xfmt))
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: tokens are QR_ACT_MXFP8 or QR_ACT_MXFP4, got %d", fn, xfmt);
  if (!in_range(M) || !in_range(N) || !in_range(K))
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: bad size (M=%lld N=%lld K=%lld)", fn, (long long)M,
                         (long long)N, (long long)K);
  if (K % 128 != 0)
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: K=%lld is not a multiple of 128", fn, (long long)K);
  if (N * (K / 2) >= kMaxCodeBytes || M * code_row_bytes(K, xfmt) >= kMaxCodeBytes)
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: code matrices must stay below 2^31 - 2^16 bytes", fn);
  if (M * N >= (int64_t)1 << 38)
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: M * N must stay below 2^38", fn);
  return QR_OK;
}

int check_out(const char* fn, int64_t M, int64_t N, int64_t K, const void* Wq, const void* sw, void* Y,
              int64_t ldy) {
  if (ldy < N)
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: ldy=%lld < N=%lld", fn, (long long)ldy, (long long)N);
  if (M > 0 && N > 0 && (!Y || (K > 0 && (!Wq || !sw))))
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: null Wq, sw or Y", fn);
  if (!aligned(Wq, 16) || !aligned(sw, 16) || !aligned(Y, 16))
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: misaligned pointer (16 bytes for Wq, sw, Y)", fn);
  return QR_OK;
}

int check_ws(const char* fn, void* ws, size_t bytes, size_t need) {
  if (need == 0) return QR_OK;
  if (!ws) return qr::set_error(QR_ERR_WORKSPACE, "%s: workspace of %zu bytes required, got NULL", fn, need);
  if (!aligned(ws, 256))
    return qr::set_error(QR_ERR_WORKSPACE, "%s: workspace must be 256-byte aligned", fn);
  if (bytes < need)
    return qr::set_error(QR_ERR_WORKSPACE, "%s: workspace of %zu bytes required, got %zu", fn, need, bytes);
  return QR_OK;
}

// Whether rows of K elements (2 bytes each) at `out` (stride ldo), which a kernel
// writes, may share memory with the rows at `in` (stride ldi) that it reads: exactly
// the same rows, or rows between which the others lie.
bool may_share(const void* out, int64_t ldo, const void* in, int64_t ldi, int64_t M, int64_t K) {
  if (!in || M == 0 || K == 0) return true;
  typedef __int128 wide;  // strides are the caller's: no product here may overflow
  const wide o = (wide)(uintptr_t)out, i = (wide)(uintptr_t)in;
  const wide oe = o + ((wide)(M - 1) * ldo + K) * 2, ie = i + ((wide)(M - 1) * ldi + K) * 2;
  if (oe <= i || ie <= o) return true;
  if (M > 1 && ldo != ldi) return false;
  if (o == i) return true;
  if (M == 1) return false;
  const wide ld = (wide)ldo * 2, r = (((o - i) % ld) + ld) % ld;
  return r >= K * 2 && r <= ld - K * 2;
}

}  // namespace

namespace qr {

size_t mx4_workspace(const char* fn, int64_t M, int64_t N, int64_t K, int xfmt) {
  if (check_product("qr_workspace_size", M, N, K, xfmt) != QR_OK) return (size_t)-1;
  if (M == 0 || N == 0) return 0;
  const size_t gemm = mx4_gemm_ws_bytes(M, N, K, xfmt);
  if (std::strcmp(fn, "qr_mxfp4_gemm") == 0) return gemm;
  if (mx4_one_launch(M, K)) return 0;
  return align256(gemm) + align256((size_t)(M * code_row_bytes(K, xfmt))) +
         align256((size_t)scale_bytes(M, K));
}

}  // namespace qr

extern "C" {

int qr_mxfp4_quantize(const void* A, int64_t R, int64_t K, int64_t lda, int src_bf16, void* codes,
                      uint8_t* scales, void* stream) {
  const char* fn = "qr_mxfp4_quantize";
  if (!in_range(R) || !in_range(K))
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: bad size (R=%lld K=%lld)", fn, (long long)R, (long long)K);
  if (src_bf16 != 0 && src_bf16 != 1)
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: src_bf16 must be 0 or 1", fn);
  if (K % 32 != 0)
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: K=%lld is not a multiple of 32", fn, (long long)K);
  if (lda < K) return qr::set_error(QR_ERR_INVALID_ARG, "%s: lda=%lld < K=%lld", fn, (long long)lda, (long long)K);
  if (R > 0 && K > 0 && (!A || !codes || !scales)) return qr::set_error(QR_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (K > 0 && R > 1 && lda % (src_bf16 ? 8 : 4) != 0)
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: rows must start on 16-byte boundaries", fn);
  if (!aligned(A, 16) || !aligned(codes, 16) || !aligned(scales, 4))
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: misaligned pointer (16 bytes for A, codes; 4 for scales)", fn);
  (void)hipGetLastError();
  return done(qr::launch_mx4_quant(A, R, K, lda, src_bf16, QR_ACT_MXFP4, codes, scales,
                                   static_cast<hipStream_t>(stream)),
              fn);
}

int qr_mx_dequantize(const void* codes, const uint8_t* scales, int64_t R, int64_t K, int fmt, void* out,
                     int64_t ldo, int out_bf16, void* stream) {
  const char* fn = "qr_mx_dequantize";
  if (!is_mx(fmt)) return qr::set_error(QR_ERR_INVALID_ARG, "%s: unknown block format %d", fn, fmt);
  if (!in_range(R) || !in_range(K))
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: bad size (R=%lld K=%lld)", fn, (long long)R, (long long)K);
  if (out_bf16 != 0 && out_bf16 != 1)
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: out_bf16 must be 0 or 1", fn);
  if (K % 32 != 0)
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: K=%lld is not a multiple of 32", fn, (long long)K);
  if (ldo < K) return qr::set_error(QR_ERR_INVALID_ARG, "%s: ldo=%lld < K=%lld", fn, (long long)ldo, (long long)K);
  if (R > 0 && K > 0 && (!out || !codes || !scales))
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (K > 0 && R > 1 && ldo % (out_bf16 ? 8 : 4) != 0)
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: rows must start on 16-byte boundaries", fn);
  if (!aligned(out, 16) || !aligned(codes, 16) || !aligned(scales, 4))
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: misaligned pointer (16 bytes for codes, out; 4 for scales)", fn);
  (void)hipGetLastError();
  return done(qr::launch_mx_dequant(codes, scales, R, K, fmt, out, ldo, out_bf16,
                                    static_cast<hipStream_t>(stream)),
              fn);
}

int qr_mxfp4_gemm(const void* Xq, const uint8_t* sx, int xfmt, const void* Wq, const uint8_t* sw,
                  int64_t M, int64_t N, int64_t K, int out, void* Y, int64_t ldy, void* workspace,
                  size_t ws_bytes, void* stream) {
  const char* fn = "qr_mxfp4_gemm";
  int st = check_product(fn, M, N, K, xfmt);
  if (st != QR_OK) return st;
  if (out != QR_OUT_BF16 && out != QR_OUT_RAW)
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: unknown output mode %d", fn, out);
  st = check_out(fn, M, N, K, Wq, sw, Y, ldy);
  if (st != QR_OK) return st;
  if (M > 0 && N > 0 && K > 0 && (!Xq || !sx)) return qr::set_error(QR_ERR_INVALID_ARG, "%s: null Xq or sx", fn);
  if (!aligned(Xq, 16) || !aligned(sx, 16))
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: misaligned pointer (16 bytes for Xq, sx)", fn);
  if (M == 0 || N == 0) return done(hipSuccess, fn);
  st = check_ws(fn, workspace, ws_bytes, qr::mx4_gemm_ws_bytes(M, N, K, xfmt));
  if (st != QR_OK) return st;
  (void)hipGetLastError();
  return done(qr::launch_mx4_gemm(Xq, sx, xfmt, Wq, sw, M, N, K, out == QR_OUT_RAW, Y, ldy, workspace,
                                  static_cast<hipStream_t>(stream)),
              fn);
}

int qr_mxfp4_plan(int64_t M, int64_t N, int64_t K, int xfmt, int* tile_n, int* tile_m, int* splits,
                  int* ahead) {
  const char* fn = "qr_mxfp4_plan";
  const int st = check_product(fn, M, N, K, xfmt);
  if (st != QR_OK) return st;
  if (!tile_n || !tile_m || !splits || !ahead)
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: null output pointer", fn);
  qr::mx4_plan(M, N, K, xfmt, tile_n, tile_m, splits, ahead);
  return done(hipSuccess, fn);
}

int qr_mxfp4_linear(const void* X, int64_t ldx, int xfmt, const void* Wq, const uint8_t* sw, int64_t M,
                    int64_t N, int64_t K, void* Y, int64_t ldy, void* workspace, size_t ws_bytes,
                    void* stream) {
  const char* fn = "qr_mxfp4_linear";
  int st = check_product(fn, M, N, K, xfmt);
  if (st != QR_OK) return st;
  st = check_out(fn, M, N, K, Wq, sw, Y, ldy);
  if (st != QR_OK) return st;
  if (ldx < K) return qr::set_error(QR_ERR_INVALID_ARG, "%s: ldx=%lld < K=%lld", fn, (long long)ldx, (long long)K);
  if (M > 0 && N > 0 && K > 0 && !X) return qr::set_error(QR_ERR_INVALID_ARG, "%s: null X", fn);
  if ((M > 1 && K > 0 && ldx % 8 != 0) || !aligned(X, 16))
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: rows of X must start on 16-byte boundaries", fn);
  if (M == 0 || N == 0) return done(hipSuccess, fn);
  st = check_ws(fn, workspace, ws_bytes, qr::mx4_workspace("qr_mxfp4_linear", M, N, K, xfmt));
  if (st != QR_OK) return st;
  (void)hipGetLastError();
  return done(qr::launch_mx4_linear(X, ldx, xfmt, Wq, sw, M, N, K, Y, ldy, workspace,
                                    static_cast<hipStream_t>(stream)),
              fn);
}

int qr_block_norm_quant(const void* Y, int64_t ldy, const void* H, int64_t ldh, int64_t M, int64_t K,
                        int norm, const float* post_gamma, const float* post_beta, const void* gate,
                        int64_t ldgate, float res_scale, const float* gamma, const float* beta, float eps,
                        int fmt, void* Hout, int64_t ldo, void* codes, void* scales, void* stream) {
  const char* fn = "qr_block_norm_quant";
  if (!in_range(M) || !in_range(K))
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: bad size (M=%lld K=%lld)", fn, (long long)M, (long long)K);
  if (norm != QR_NORM_RMS && norm != QR_NORM_LAYER)
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: unknown norm kind %d", fn, norm);
  if (fmt < QR_ACT_INT8 || fmt > QR_ACT_BF16)
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: unknown output format %d", fn, fmt);
  if (!std::isfinite(eps) || eps < 0.0f)
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
  if (!std::isfinite(res_scale))
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: res_scale must be finite", fn);
  if (post_beta && !post_gamma)
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: post_beta without post_gamma", fn);
  const int unit = is_mx(fmt) ? 32 : 16;
  if (K % unit != 0)
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: K=%lld is not a multiple of %d", fn, (long long)K, unit);
  if (K > 32768) return qr::set_error(QR_ERR_UNSUPPORTED, "%s: K=%lld > 32768", fn, (long long)K);
  if (ldy < K || ldh < K || ldo < K || (gate && ldgate != 0 && ldgate < K))
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: a row stride below K=%lld", fn, (long long)K);
  if (M > 0 && K > 0 && (!Y || !H || !gamma || !Hout || !codes))
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: null Y, H, gamma, Hout or codes", fn);
  if (M > 0 && fmt != QR_ACT_BF16 && !scales) return qr::set_error(QR_ERR_INVALID_ARG, "%s: null scales", fn);
  if (M > 1 && K > 0 && (ldy % 8 != 0 || ldh % 8 != 0 || ldo % 8 != 0 || (gate && ldgate % 8 != 0)))
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: row strides must be multiples of 8", fn);
  if (!aligned(Y, 16) || !aligned(H, 16) || !aligned(post_gamma, 16) || !aligned(post_beta, 16) ||
      !aligned(gate, 16) || !aligned(gamma, 16) || !aligned(beta, 16) || !aligned(Hout, 16) ||
      !aligned(codes, 16) || !aligned(scales, 4))
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: misaligned pointer (16 bytes; 4 for scales)", fn);
  if (!may_share(Hout, ldo, H, ldh, M, K) || !may_share(Hout, ldo, Y, ldy, M, K) ||
      (gate && ldgate != 0 && !may_share(Hout, ldo, gate, ldgate, M, K)))
    return qr::set_error(QR_ERR_INVALID_ARG,
                         "%s: Hout overlaps an input's rows without being those rows", fn);
  qr::BlockNormArgs p;
  p.Y = static_cast<const uint16_t*>(Y);
  p.H = static_cast<const uint16_t*>(H);
  p.gate = gate;
  p.gate_rows = ldgate != 0;
  p.post_gamma = post_gamma;
  p.post_beta = post_beta;
  p.gamma = gamma;
  p.beta = beta;
  p.Hout = static_cast<uint16_t*>(Hout);
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = scales;
  p.ldy = ldy; p.ldh = ldh; p.ldgate = ldgate; p.ldo = ldo;
  p.M = M; p.K = K;
  p.res = res_scale;
  p.eps = eps;
  p.fmt = fmt;
  (void)hipGetLastError();
  return done(qr::launch_block_norm(p, norm, static_cast<hipStream_t>(stream)), fn);
}

int qr_silu_mul_mx(const void* G, const void* U, int64_t M, int64_t N, int64_t ldg, int64_t ldu, int fmt,
                   void* codes, uint8_t* scales, void* stream) {
  const char* fn = "qr_silu_mul_mx";
  if (!is_mx(fmt)) return qr::set_error(QR_ERR_INVALID_ARG, "%s: unknown block format %d", fn, fmt);
  if (!in_range(M) || !in_range(N))
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: bad size (M=%lld N=%lld)", fn, (long long)M, (long long)N);
  if (N % 32 != 0)
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: N=%lld is not a multiple of 32", fn, (long long)N);
  if (ldg < N || ldu < N)
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: ldg=%lld / ldu=%lld < N=%lld", fn, (long long)ldg,
                         (long long)ldu, (long long)N);
  if (M > 0 && N > 0 && (!G || !U || !codes || !scales))
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (M > 1 && N > 0 && (ldg % 8 != 0 || ldu % 8 != 0))
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: ldg and ldu must be multiples of 8", fn);
  if (!aligned(G, 16) || !aligned(U, 16) || !aligned(codes, 16) || !aligned(scales, 4))
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: misaligned pointer (16 bytes for G, U, codes; 4 for scales)", fn);
  (void)hipGetLastError();
  return done(qr::launch_silu_mx(G, U, M, N, ldg, ldu, fmt, codes, scales, static_cast<hipStream_t>(stream)),
              fn);
}

}  // extern "C"
