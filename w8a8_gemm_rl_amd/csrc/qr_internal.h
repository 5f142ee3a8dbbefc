// Internal interface between the C-ABI layer and the gfx950 kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "qr_device.h"
#include "qr_gemm.h"
#include "qr_small_m.h"

namespace qr {

hipError_t launch_act_quant(const void* X, int64_t M, int64_t K, int64_t ldx, float act_mult,
                            int qt, void* Xq, float* scale_x, hipStream_t st);
hipError_t launch_weight_quant(const float* W, int64_t N, int64_t K, int64_t ldw, float s, int qt,
                               void* Wq, float* scale_w, float* Wsc, hipStream_t st);
hipError_t launch_fold_norm(float* gamma, float* beta, int64_t K, float s, hipStream_t st);
hipError_t launch_norm_quant(const void* H, int64_t M, int64_t K, int64_t ldh, int kind,
                             const float* gamma, const float* beta, float eps, int qt, void* Xq,
                             float* scale_x, hipStream_t st);
hipError_t launch_silu_mul_quant(const void* G, const void* U, int64_t M, int64_t N, int64_t ldg,
                                 int64_t ldu, float act_mult, int qt, void* Xq, float* scale_x,
                                 hipStream_t st);
hipError_t launch_mx_quant(const void* A, int64_t R, int64_t K, int64_t lda, int bf16,
                           void* codes, uint8_t* scales, hipStream_t st);
hipError_t launch_mx_gemm(const void* Xq, const uint8_t* sx, const void* Wq, const uint8_t* sw,
                          int64_t M, int64_t N, int64_t K, int out_raw, void* Y, int64_t ldy,
                          hipStream_t st);
int64_t acr_blocks(int64_t n);
hipError_t launch_acr_tis(const float* logp, const float* lprox, const float* lbeh,
                          const float* adv, const uint8_t* mask, int64_t n, float eps, float C,
                          float* loss, float* grad, double* sums, double* part, hipStream_t st);
hipError_t launch_requant(const float* Wp, int64_t N, int64_t K, int64_t ldw, int qt, void* Wq,
                          float* scale_w, uint32_t* row_flips, hipStream_t st);

// MXFP4 operators (mxfp4_kernels.hip) and block norms (block_kernels.hip). `fmt` is
// one of the header's QR_ACT_* formats.
hipError_t launch_mx4_quant(const void* A, int64_t R, int64_t K, int64_t lda, int bf16, int fmt,
                            void* codes, uint8_t* scales, hipStream_t st);
hipError_t launch_mx_dequant(const void* codes, const uint8_t* scales, int64_t R, int64_t K, int fmt,
                             void* out, int64_t ldo, int bf16, hipStream_t st);
void mx4_plan(int64_t M, int64_t N, int64_t K, int xfmt, int* tile_n, int* tile_m, int* splits, int* ahead);
size_t mx4_gemm_ws_bytes(int64_t M, int64_t N, int64_t K, int xfmt);
hipError_t launch_mx4_gemm(const void* Xq, const uint8_t* sx, int xfmt, const void* Wq,
                           const uint8_t* sw, int64_t M, int64_t N, int64_t K, int out_raw, void* Y,
                           int64_t ldy, void* ws, hipStream_t st);
hipError_t launch_mx4_linear(const void* X, int64_t ldx, int xfmt, const void* Wq, const uint8_t* sw,
                             int64_t M, int64_t N, int64_t K, void* Y, int64_t ldy, void* ws,
                             hipStream_t st);
bool mx4_one_launch(int64_t M, int64_t K);  // qr_mxfp4_linear needs no workspace
// Workspace of qr_mxfp4_gemm / qr_mxfp4_linear; (size_t)-1 for invalid sizes.
size_t mx4_workspace(const char* fn, int64_t M, int64_t N, int64_t K, int xfmt);

struct BlockNormArgs {
  const uint16_t *Y, *H;
  const void* gate;  // NULL, fp32 [K], or (gate_rows) bf16 [M, ldgate]
  const float *post_gamma, *post_beta, *gamma, *beta;
  uint16_t* Hout;
  uint8_t* codes;
  void* scales;
  int64_t ldy, ldh, ldgate, ldo, M, K;
  int64_t row0 = 0;    // first row of the launch
  double inv_k = 0.0;  // 1 / K
  float res, eps;
  int fmt;
  bool gate_rows;
};
hipError_t launch_block_norm(const BlockNormArgs& p, int kind, hipStream_t st);
hipError_t launch_silu_mx(const void* G, const void* U, int64_t M, int64_t N, int64_t ldg, int64_t ldu,
                          int fmt, void* codes, uint8_t* scales, hipStream_t st);

// Error reporting of the C ABI (qr_last_error): set the thread-local message
// and return `code`; hip_error maps a HIP error to QR_ERR_HIP / QR_ERR_NO_DEVICE.
int set_error(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int hip_error(hipError_t e, const char* what);

unsigned read_probe_blocks();
hipError_t launch_read_probe(const void* buf, int64_t n16, uint32_t* sink, hipStream_t st);
bool copy_stream_probe_tile(int tile, int& bn, int& bm);
hipError_t launch_copy_stream_probe(int tile, const void* W, const void* X, int64_t N, int64_t M,
                                    int64_t K, int64_t ldw, int64_t ldx, int rows, int flags,
                                    uint32_t* sink, hipStream_t st);
hipError_t launch_mfma_probe(int qt, int blocks, int iters, uint32_t* sink, uint64_t* ticks,
                             hipStream_t st);

}  // namespace qr
