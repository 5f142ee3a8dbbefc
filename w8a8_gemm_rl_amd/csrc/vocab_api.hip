// C ABI of the losses over a large vocabulary (declared and documented in
// include/qurl_w8a8.h). As for the other entry points, arguments are validated on
// the host before anything is enqueued, and nothing here synchronizes.
#include <cstring>

#include "qr_internal.h"
#include "qr_vocab.h"
#include "qurl_w8a8.h"

namespace {

// Tokens and ids: what keeps the products' tile counts in 31 bits, and an id with a place in a
// list in 32. Rows: offsets inside a tile of 256 rows in 30 bits.
constexpr int64_t kMaxTokens = (int64_t)1 << 22, kMaxIds = kMaxTokens - 1;
constexpr int64_t kMaxK = (int64_t)1 << 16, kMaxLd = (int64_t)1 << 21;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int check_shape(const char* fn, int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 1 || K < 1)
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: bad size (M=%lld N=%lld K=%lld)", fn, (long long)M,
                         (long long)N, (long long)K);
  if (K % 8 != 0)
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: K=%lld is not a multiple of 8", fn, (long long)K);
  if (M > kMaxTokens || N > kMaxIds || K > kMaxK)
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: M is at most 2^22, N 2^22 - 1, K 2^16", fn);
  return QR_OK;
}

int check_list(const char* fn, int64_t L) {
  if (L < 1 || L > qr::kVocabMaxList)
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: L=%lld is not in [1, %lld]", fn, (long long)L,
                         (long long)qr::kVocabMaxList);
  return QR_OK;
}

int check_rows(const char* fn, const char* name, const void* p, int64_t rows, int64_t ld, int64_t K) {
  if (ld < K) return qr::set_error(QR_ERR_INVALID_ARG, "%s: row stride of %s below K=%lld", fn, name, (long long)K);
  if (rows > 0 && !p) return qr::set_error(QR_ERR_INVALID_ARG, "%s: null %s", fn, name);
  if ((rows > 1 && ld % 8 != 0) || !aligned(p, 16))
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: rows of %s must start on 16-byte boundaries", fn, name);
  if (rows > 1 && ld > kMaxLd)
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: row stride of %s above 2^21", fn, name);
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

// Checks that all four entry points share; fills what they share of `a`.
int check_common(const char* fn, qr::VocabArgs& a, const void* X, int64_t ldx, const void* W, int64_t ldw,
                 int64_t M, int64_t N, int64_t K, float scale) {
  int st = check_shape(fn, M, N, K);
  if (st == QR_OK) st = check_rows(fn, "X", X, M, ldx, K);
  if (st == QR_OK) st = check_rows(fn, "W", W, N, ldw, K);
  if (st != QR_OK) return st;
  // its product with log2 e is a fp32 value
  if (!(scale > 0.0f && scale <= 0x1p127f))
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: scale must be > 0 and at most 2^127", fn);
  a.X = static_cast<const uint16_t*>(X);
  a.W = static_cast<const uint16_t*>(W);
  a.ldx = ldx; a.ldw = ldw; a.M = M; a.N = N; a.K = K;
  a.scale = scale;
  return QR_OK;
}

int set_target(const char* fn, qr::VocabArgs& a, const int64_t* target) {
  if (a.M > 0 && !target) return qr::set_error(QR_ERR_INVALID_ARG, "%s: null target", fn);
  if (!aligned(target, 8)) return qr::set_error(QR_ERR_UNSUPPORTED, "%s: target must be 8-byte aligned", fn);
  a.target = target;
  return QR_OK;
}

int set_list(const char* fn, qr::VocabArgs& a, const int64_t* index, const void* teacher, int teacher_bf16,
             const float* teacher_lse, int64_t L) {
  const int st = check_list(fn, L);
  if (st != QR_OK) return st;
  if (teacher_bf16 != 0 && teacher_bf16 != 1)
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: teacher_bf16 must be 0 or 1", fn);
  if (a.M > 0 && (!index || !teacher))
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: null index or teacher", fn);
  if (!aligned(index, 8) || !aligned(teacher, teacher_bf16 ? 2 : 4) || !aligned(teacher_lse, 4))
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: misaligned index, teacher or teacher_lse", fn);
  a.index = index;
  a.teacher = teacher;
  a.teacher_bf16 = teacher_bf16 != 0;
  a.teacher_lse = teacher_lse;
  a.L = L;
  return QR_OK;
}

int run_loss(const char* fn, qr::VocabArgs& a, float* value, float* lse, void* ws, size_t ws_bytes, void* stream) {
  if (a.M > 0 && (!value || !lse)) return qr::set_error(QR_ERR_INVALID_ARG, "%s: null output", fn);
  if (!aligned(value, 4) || !aligned(lse, 4))
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: outputs must be 4-byte aligned", fn);
  if (a.M == 0) return qr::hip_error(hipSuccess, fn);
  const int st = check_ws(fn, ws, ws_bytes, qr::vocab_ws_bytes(a.M, a.N, a.K, a.L, a.index != nullptr, false));
  if (st != QR_OK) return st;
  a.value = value;
  a.lse_out = lse;
  (void)hipGetLastError();
  return qr::hip_error(qr::launch_vocab_loss(a, ws, static_cast<hipStream_t>(stream)), fn);
}

int run_grad(const char* fn, qr::VocabArgs& a, const float* lse, const float* g, void* dX, int64_t lddx, void* dW,
             int64_t lddw, void* ws, size_t ws_bytes, void* stream) {
  if (a.M > 0 && (!lse || !g)) return qr::set_error(QR_ERR_INVALID_ARG, "%s: null lse or incoming gradient", fn);
  if (!aligned(lse, 4) || !aligned(g, 4))
    return qr::set_error(QR_ERR_UNSUPPORTED, "%s: lse and the incoming gradient must be 4-byte aligned", fn);
  if (a.M > 0 && !dX && !dW) return qr::set_error(QR_ERR_INVALID_ARG, "%s: neither dX nor dW", fn);
  int st = QR_OK;
  if (dX) st = check_rows(fn, "dX", dX, a.M, lddx, a.K);
  if (st == QR_OK && dW) st = check_rows(fn, "dW", dW, a.N, lddw, a.K);
  if (st != QR_OK) return st;
  st = check_ws(fn, ws, ws_bytes, qr::vocab_ws_bytes(a.M, a.N, a.K, a.L, a.index != nullptr, true));
  if (st != QR_OK) return st;
  a.lse = lse;
  a.g = g;
  a.dX = static_cast<uint16_t*>(dX);
  a.dW = static_cast<uint16_t*>(dW);
  a.lddx = lddx;
  a.lddw = lddw;
  (void)hipGetLastError();
  return qr::hip_error(qr::launch_vocab_grad(a, ws, static_cast<hipStream_t>(stream)), fn);
}

}  // namespace

namespace qr {

size_t vocab_workspace(const char* fn, int64_t M, int64_t N, int64_t K, int64_t L) {
  const bool lists = std::strncmp(fn, "qr_vocab_distill", 16) == 0, grad = std::strstr(fn, "_grad") != nullptr;
  if (check_shape("qr_workspace_size", M, N, K) != QR_OK) return (size_t)-1;
  if (lists && check_list("qr_workspace_size", L) != QR_OK) return (size_t)-1;
  return vocab_ws_bytes(M, N, K, lists ? L : 1, lists, grad);
}

}  // namespace qr

extern "C" {

int qr_vocab_logp(const void* X, int64_t ldx, const void* W, int64_t ldw, int64_t M, int64_t N, int64_t K,
                  const int64_t* target, float scale, float* logp, float* lse, void* workspace, size_t ws_bytes,
                  void* stream) {
  const char* fn = "qr_vocab_logp";
  qr::VocabArgs a;
  int st = check_common(fn, a, X, ldx, W, ldw, M, N, K, scale);
  if (st == QR_OK) st = set_target(fn, a, target);
  return st != QR_OK ? st : run_loss(fn, a, logp, lse, workspace, ws_bytes, stream);
}

int qr_vocab_logp_grad(const void* X, int64_t ldx, const void* W, int64_t ldw, int64_t M, int64_t N, int64_t K,
                       const int64_t* target, float scale, const float* lse, const float* dlogp, void* dX,
                       int64_t lddx, void* dW, int64_t lddw, void* workspace, size_t ws_bytes, void* stream) {
  const char* fn = "qr_vocab_logp_grad";
  qr::VocabArgs a;
  int st = check_common(fn, a, X, ldx, W, ldw, M, N, K, scale);
  if (st == QR_OK) st = set_target(fn, a, target);
  return st != QR_OK ? st : run_grad(fn, a, lse, dlogp, dX, lddx, dW, lddw, workspace, ws_bytes, stream);
}

int qr_vocab_distill(const void* X, int64_t ldx, const void* W, int64_t ldw, int64_t M, int64_t N, int64_t K,
                     const int64_t* index, const void* teacher, int teacher_bf16, const float* teacher_lse,
                     int64_t L, float scale, float* loss, float* lse, void* workspace, size_t ws_bytes,
                     void* stream) {
  const char* fn = "qr_vocab_distill";
  qr::VocabArgs a;
  int st = check_common(fn, a, X, ldx, W, ldw, M, N, K, scale);
  if (st == QR_OK) st = set_list(fn, a, index, teacher, teacher_bf16, teacher_lse, L);
  return st != QR_OK ? st : run_loss(fn, a, loss, lse, workspace, ws_bytes, stream);
}

int qr_vocab_distill_grad(const void* X, int64_t ldx, const void* W, int64_t ldw, int64_t M, int64_t N, int64_t K,
                          const int64_t* index, const void* teacher, int teacher_bf16, const float* teacher_lse,
                          int64_t L, float scale, const float* lse, const float* dloss, void* dX, int64_t lddx,
                          void* dW, int64_t lddw, void* workspace, size_t ws_bytes, void* stream) {
  const char* fn = "qr_vocab_distill_grad";
  qr::VocabArgs a;
  int st = check_common(fn, a, X, ldx, W, ldw, M, N, K, scale);
  if (st == QR_OK) st = set_list(fn, a, index, teacher, teacher_bf16, teacher_lse, L);
  return st != QR_OK ? st : run_grad(fn, a, lse, dloss, dX, lddx, dW, lddw, workspace, ws_bytes, stream);
}

int qr_vocab_plan(int64_t M, int64_t N, int64_t K, int* tile_ids, int* tile_tokens, int* dx_rows, int64_t* piece) {
  const char* fn = "qr_vocab_plan";
  const int st = check_shape(fn, M, N, K);
  if (st != QR_OK) return st;
  if (M == 0) return qr::set_error(QR_ERR_INVALID_ARG, "%s: no tokens", fn);
  if (!tile_ids || !tile_tokens || !dx_rows || !piece)
    return qr::set_error(QR_ERR_INVALID_ARG, "%s: null output pointer", fn);
  qr::vocab_plan(M, N, K, tile_ids, tile_tokens, dx_rows, piece);
  return qr::hip_error(hipSuccess, fn);
}

}  // extern "C"
