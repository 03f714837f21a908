// capi_mx.cu -- the extern "C" boundary of the microscaled operators (declared
// in include/qgemv.h).  Host code only: checks the arguments and enqueues the
// kernels on the caller's stream.
#include <stdint.h>

#include <cmath>

#include "mx.h"
#include "qgemv.h"

namespace qgemv {
// capi.cu
int report_launch(cudaError_t e);
int device_and_sms(int* dev, int* sms);
}  // namespace qgemv

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Rows of whole blocks, whose number a grid can count, with room above every index.
bool valid_rows(int M, int K) {
  return M >= 0 && M <= 1 << 30 && K >= 32 && K <= 1 << 30 && K % 32 == 0 &&
         static_cast<long long>(M) * K <= 1LL << 38;
}

int product(qgemv::MxProductArgs& a, void* stream) {
  if (a.M == 0) return QGEMV_OK;
  int dev, sms;
  if (int rc = qgemv::device_and_sms(&dev, &sms)) return rc;
  return qgemv::report_launch(
      qgemv::mx_product_launch(a, sms, dev, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int qgemv_mx_quantize(int bits, const uint16_t* x, int M, int K, void* codes, uint8_t* scales,
                      void* stream) {
  const bool some = M != 0;
  if (some && (!x || !codes || !scales)) return QGEMV_ENULL;
  if ((bits != 4 && bits != 8) || !valid_rows(M, K)) return QGEMV_EINVAL;
  if (!aligned(x, 16) || !aligned(codes, 16)) return QGEMV_EALIGN;
  if (!some) return QGEMV_OK;
  int dev, sms;
  if (int rc = qgemv::device_and_sms(&dev, &sms)) return rc;
  const qgemv::MxQuantArgs a{reinterpret_cast<const __half*>(x), codes, scales,
                             static_cast<long long>(M) * (K / 32)};
  return qgemv::report_launch(
      qgemv::mx_quantize_launch(a, bits, sms, static_cast<cudaStream_t>(stream)));
}

int qgemv_mx_dequantize(int bits, const void* codes, const uint8_t* scales, int M, int K,
                        uint16_t* y, void* stream) {
  const bool some = M != 0;
  if (some && (!y || !codes || !scales)) return QGEMV_ENULL;
  if ((bits != 4 && bits != 8) || !valid_rows(M, K)) return QGEMV_EINVAL;
  if (!aligned(y, 16) || !aligned(codes, 16)) return QGEMV_EALIGN;
  if (!some) return QGEMV_OK;
  int dev, sms;
  if (int rc = qgemv::device_and_sms(&dev, &sms)) return rc;
  const qgemv::MxDequantArgs a{codes, scales, reinterpret_cast<__half*>(y),
                               static_cast<long long>(M) * (K / 32)};
  return qgemv::report_launch(
      qgemv::mx_dequantize_launch(a, bits, sms, static_cast<cudaStream_t>(stream)));
}

int qgemv_residual_rmsnorm_mxfp8(const uint16_t* x, const uint16_t* residual,
                                 const uint16_t* gamma, float eps, int M, int K, uint16_t* h,
                                 uint8_t* codes, uint8_t* scales, void* stream) {
  const bool some = M != 0;
  if (!gamma || (some && (!x || !codes || !scales || (residual && !h)))) return QGEMV_ENULL;
  if (!valid_rows(M, K) || !(eps > 0.0f) || !std::isfinite(eps)) return QGEMV_EINVAL;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(gamma, 16) || !aligned(h, 16) ||
      !aligned(codes, 16))
    return QGEMV_EALIGN;
  if (!some) return QGEMV_OK;
  int dev, sms;
  if (int rc = qgemv::device_and_sms(&dev, &sms)) return rc;
  const qgemv::MxNormArgs a{reinterpret_cast<const __half*>(x),
                            reinterpret_cast<const __half*>(residual),
                            reinterpret_cast<const __half*>(gamma),
                            eps,
                            M,
                            K,
                            reinterpret_cast<__half*>(h),
                            codes,
                            scales};
  return qgemv::report_launch(qgemv::mx_norm_launch(a, sms, static_cast<cudaStream_t>(stream)));
}

int qgemv_mxfp4(const uint32_t* codes, const uint8_t* scales, const uint16_t* x, uint16_t* y,
                int M, int N, int K, const uint16_t* residual, void* stream) {
  if (!codes || !scales || !x || !y) return QGEMV_ENULL;
  if (M < 1 || M > QGEMV_MAX_M || K > QGEMV_MXFP4_MAX_K || N < 1 || !valid_rows(M, K) || !valid_rows(N, K)) return QGEMV_EINVAL;
  if (!aligned(codes, 16) || !aligned(x, 16) || !aligned(y, 2) || !aligned(residual, 2))
    return QGEMV_EALIGN;
  qgemv::MxProductArgs a{};
  a.w = codes;
  a.ws = scales;
  a.x16 = reinterpret_cast<const __half*>(x);
  a.res = reinterpret_cast<const __half*>(residual);
  a.y = reinterpret_cast<__half*>(y);
  a.M = M;
  a.N = N;
  a.K = K;
  return product(a, stream);
}

int qgemv_mx_gemm(const uint32_t* codes, const uint8_t* scales, const uint8_t* x_codes,
                  const uint8_t* x_scales, uint16_t* y, int M, int N, int K,
                  const uint16_t* residual, void* stream) {
  if (!codes || !scales || (M != 0 && (!x_codes || !x_scales || !y))) return QGEMV_ENULL;
  if (N < 1 || !valid_rows(M, K) || !valid_rows(N, K)) return QGEMV_EINVAL;
  if (!aligned(codes, 16) || !aligned(x_codes, 16) || !aligned(y, 2) || !aligned(residual, 2))
    return QGEMV_EALIGN;
  qgemv::MxProductArgs a{};
  a.w = codes;
  a.ws = scales;
  a.x = x_codes;
  a.xs = x_scales;
  a.res = reinterpret_cast<const __half*>(residual);
  a.y = reinterpret_cast<__half*>(y);
  a.M = M;
  a.N = N;
  a.K = K;
  return product(a, stream);
}

int qgemv_mx_swiglu(const uint32_t* gate_codes, const uint8_t* gate_scales,
                    const uint32_t* up_codes, const uint8_t* up_scales, const uint8_t* x_codes,
                    const uint8_t* x_scales, int M, int I, int K, uint16_t* h, uint8_t* h_codes,
                    uint8_t* h_scales, void* stream) {
  if (!gate_codes || !gate_scales || !up_codes || !up_scales) return QGEMV_ENULL;
  if (M != 0 && (!x_codes || !x_scales || (!h && !h_codes))) return QGEMV_ENULL;
  if ((h_codes == nullptr) != (h_scales == nullptr)) return QGEMV_ENULL;
  if (I < 1 || !valid_rows(M, K) || !valid_rows(I, K) || (h_codes && I % 32 != 0)) return QGEMV_EINVAL;
  if (!aligned(gate_codes, 16) || !aligned(up_codes, 16) || !aligned(x_codes, 16) ||
      !aligned(h_codes, 16) || !aligned(h, 2))
    return QGEMV_EALIGN;
  qgemv::MxProductArgs a{};
  a.w = gate_codes;
  a.ws = gate_scales;
  a.up = up_codes;
  a.us = up_scales;
  a.x = x_codes;
  a.xs = x_scales;
  a.y = reinterpret_cast<__half*>(h);
  a.yc = h_codes;
  a.ys = h_scales;
  a.M = M;
  a.N = I;
  a.K = K;
  return product(a, stream);
}

}  // extern "C"
