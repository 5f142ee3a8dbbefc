// Losses over a large vocabulary: interface between the C-ABI layer and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qr {

constexpr int64_t kVocabMaxList = 1024;  // entries of a token's list

struct VocabArgs {
  const uint16_t *X, *W;  // [M, ldx], [N, ldw] bf16
  int64_t ldx, ldw, M, N, K;
  const int64_t* target = nullptr;  // [M], or a list:
  const int64_t* index = nullptr;   // [M, L]
  const void* teacher = nullptr;    // [M, L] fp32 or bf16
  const float* teacher_lse = nullptr;
  bool teacher_bf16 = false;
  int64_t L = 1;
  float scale = 1.0f;
  float *value = nullptr, *lse_out = nullptr;        // losses' results
  const float *lse = nullptr, *g = nullptr;          // gradients' inputs
  uint16_t *dX = nullptr, *dW = nullptr;             // and results
  int64_t lddx = 0, lddw = 0;
};

// Workspace bytes; `lists`: per-token lists with weights (else one id each).
size_t vocab_ws_bytes(int64_t M, int64_t N, int64_t K, int64_t L, bool lists, bool grad);
// Workspace of an entry point by its name; (size_t)-1 for invalid sizes.
size_t vocab_workspace(const char* fn, int64_t M, int64_t N, int64_t K, int64_t L);
void vocab_plan(int64_t M, int64_t N, int64_t K, int* ids, int* tokens, int* rows, int64_t* piece);
hipError_t launch_vocab_loss(const VocabArgs& p, void* ws, hipStream_t st);
hipError_t launch_vocab_grad(const VocabArgs& p, void* ws, hipStream_t st);

}  // namespace qr
