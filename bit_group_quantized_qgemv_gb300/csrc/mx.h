// mx.h -- argument blocks and launch entry points of the microscaled (MX)
// operators (host and device).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace qgemv {

constexpr int kMxBlock = 32;  // values along k that share a scale

// Rows of MX values: codes e2m1 (eight to a word) or e4m3 (a byte each), one scale
// byte per block.
struct MxQuantArgs {
  const __half* x;
  void* codes;
  uint8_t* scales;
  long long blocks;
};

struct MxDequantArgs {
  const void* codes;
  const uint8_t* scales;
  __half* y;
  long long blocks;
};

struct MxNormArgs {
  const __half *x, *res, *gamma;  // res null: h = x, not written
  float eps;
  int M, K;
  __half* h;
  uint8_t *codes, *scales;
};

// y[m][n] = sum_k w[n][k] x[m][k] (+ res), or with `up` the gated product
// silu(w x) (up x); x as fp16 (x16) or MXFP8 (x, xs); out as fp16 (y) and / or
// MXFP8 (yc, ys).
struct MxProductArgs {
  const uint32_t *w, *up;
  const uint8_t *ws, *us;
  const __half* x16;
  const uint8_t *x, *xs;
  const __half* res;
  __half* y;
  uint8_t *yc, *ys;
  int M, N, K;
};

cudaError_t mx_quantize_launch(const MxQuantArgs& a, int bits, int sms, cudaStream_t st);
cudaError_t mx_dequantize_launch(const MxDequantArgs& a, int bits, int sms, cudaStream_t st);
cudaError_t mx_norm_launch(const MxNormArgs& a, int sms, cudaStream_t st);
cudaError_t mx_product_launch(const MxProductArgs& a, int sms, int device, cudaStream_t st);

// Read and clear the status word of the product kernels.
cudaError_t status_mx(unsigned* out);

}  // namespace qgemv
