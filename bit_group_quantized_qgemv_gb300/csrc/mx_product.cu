// mx_product.cu -- products with MXFP4 weights: plain, with a residual, gated.
//
// A warp takes one weight row (gated: two) and eight rows of activations; a lane
// takes every 32nd word of eight codes.
#include "mx.h"
#include "mx_format.cuh"
#include "qgemv_device.cuh"

namespace qgemv {
namespace {

__device__ unsigned g_status = 0;

constexpr int kRows = 8;   // rows of activations a warp
constexpr int kWarps = 32;  // weight rows a block: a block of an MXFP8 output

// Eight codes of row m and their scale byte (fp16: the values, 127).
__device__ __forceinline__ int load8(const MxProductArgs& a, int m, int i, float* v) {
  const long long at = static_cast<long long>(m) * (a.K / 8) + i;
  if (a.x16) {
    const uint4 w = reinterpret_cast<const uint4*>(a.x16)[at];
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[k]));
      v[2 * k] = f.x + (f.x - f.x);  // an infinity becomes a NaN
      v[2 * k + 1] = f.y + (f.y - f.y);
    }
    return 127;
  }
  const uint2 c = reinterpret_cast<const uint2*>(a.x)[at];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = mx_values8((k < 2 ? c.x : c.y) >> (16 * (k & 1)));
    v[2 * k] = f.x;
    v[2 * k + 1] = f.y;
  }
  return a.xs[at >> 2];
}

// Both scales at once: one of them alone may leave fp32's range.
__device__ __forceinline__ float scaled(float dot, int ws, int xs) {
  return ws == 255 || xs == 255 ? __uint_as_float(0x7FFFFFFFu) : scalbnf(dot, ws + xs - 254);
}

template <bool GATED>
__global__ void __launch_bounds__(32 * kWarps) mx_product_kernel(const MxProductArgs a) {
  __shared__ float out[kRows][kWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = blockIdx.x * kWarps + warp, m0 = blockIdx.y * kRows;
  const int rows = min(kRows, a.M - m0), words = a.K / 8;
  float g[kRows] = {}, u[kRows] = {};
  if (n < a.N) {
    for (int i = lane; i < words; i += 32) {
      const long long at = static_cast<long long>(n) * words + i;
      float wv[2][8];
      int sw[2];
#pragma unroll
      for (int p = 0; p < (GATED ? 2 : 1); ++p) {
        const uint32_t c = (p ? a.up : a.w)[at];
        sw[p] = (p ? a.us : a.ws)[at >> 2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = mx_values4(c >> (8 * k));
          wv[p][2 * k] = f.x;
          wv[p][2 * k + 1] = f.y;
        }
      }
#pragma unroll
      for (int m = 0; m < kRows; ++m) {
        if (m >= rows) break;
        float x[8];
        const int sx = load8(a, m0 + m, i, x);
        float d[2] = {};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          d[0] = fmaf(wv[0][k], x[k], d[0]);
          if (GATED) d[1] = fmaf(wv[1][k], x[k], d[1]);
        }
        g[m] += scaled(d[0], sw[0], sx);
        if (GATED) u[m] += scaled(d[1], sw[1], sx);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < kRows; ++m) {
    for (int k = 16; k > 0; k /= 2) {
      g[m] += __shfl_xor_sync(0xFFFFFFFFu, g[m], k);
      if (GATED) u[m] += __shfl_xor_sync(0xFFFFFFFFu, u[m], k);
    }
    if (GATED) g[m] = silu_f(g[m]) * u[m];
    if (lane == 0) {
      out[m][warp] = g[m];
      if (m < rows && n < a.N) {
        const long long at = static_cast<long long>(m0 + m) * a.N + n;
        if (a.y) a.y[at] = __float2half_rn(g[m] + (a.res ? __half2float(a.res[at]) : 0.f));
      }
    }
  }
  if (a.yc == nullptr) return;
  __syncthreads();
  if (warp < rows) {
    const float v = out[warp][lane];
    uint32_t most = __float_as_uint(v) & 0x7FFFFFFFu;
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    const int byte = mx_scale_byte<8>(__uint_as_float(most));
    const long long at = static_cast<long long>(m0 + warp) * a.N + blockIdx.x * kWarps + lane;
    a.yc[at] = static_cast<uint8_t>(mx_codes8(v * mx_inverse(byte), 0.f));
    if (lane == 0) a.ys[at >> 5] = static_cast<uint8_t>(byte);
  }
}

}  // namespace

cudaError_t mx_product_launch(const MxProductArgs& a, int, int, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.N + kWarps - 1) / kWarps),
                     static_cast<unsigned>((a.M + kRows - 1) / kRows));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return a.up ? cudaLaunchKernelEx(&cfg, mx_product_kernel<true>, a)
              : cudaLaunchKernelEx(&cfg, mx_product_kernel<false>, a);
}

cudaError_t status_mx(unsigned* out) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_status, sizeof(v));
  if (e != cudaSuccess) return e;
  e = cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
  *out |= v;
  return e;
}

}  // namespace qgemv
