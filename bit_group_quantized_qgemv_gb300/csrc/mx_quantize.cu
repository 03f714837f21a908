// mx_quantize.cu -- fp16 rows to microscaled values and back, and the residual
// addition with the RMS norm whose result leaves in MXFP8.  Bound by the bytes they
// read and write, small calls by the launch.
#include "mx.h"
#include "mx_format.cuh"
#include "qgemv_device.cuh"

namespace qgemv {
namespace {

constexpr int kThreads = 256;

struct Eight {
  float v[8];
};

__device__ __forceinline__ Eight unpack(uint4 w) {
  Eight r;
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    r.v[2 * i] = f.x;
    r.v[2 * i + 1] = f.y;
  }
  return r;
}

// Largest magnitude; a NaN counts as more than an infinity (fmaxf would drop it).
__device__ __forceinline__ float magnitude(const Eight& x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x.v[i]) & 0x7FFFFFFFu);
  return __uint_as_float(m);
}

// Over the four lanes of a block.
__device__ __forceinline__ float block_magnitude(float m) {
  uint32_t u = __float_as_uint(m);
  u = max(u, __shfl_xor_sync(0xFFFFFFFFu, u, 1));
  u = max(u, __shfl_xor_sync(0xFFFFFFFFu, u, 2));
  return __uint_as_float(u);
}

__device__ __forceinline__ uint2 codes8(const Eight& x, float inv) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = mx_codes8(x.v[4 * i] * inv, x.v[4 * i + 1] * inv) |
           (mx_codes8(x.v[4 * i + 2] * inv, x.v[4 * i + 3] * inv) << 16);
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint32_t codes4(const Eight& x, float inv) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) w |= mx_codes4(x.v[2 * i] * inv, x.v[2 * i + 1] * inv) << (8 * i);
  return w;
}

// Four lanes to a block, eight values a lane: 16 bytes in, 8 (4) out.
template <int BITS>
__global__ void __launch_bounds__(kThreads) mx_quantize_kernel(const MxQuantArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const bool live = i < 4 * a.blocks;
  const Eight x = unpack(live ? reinterpret_cast<const uint4*>(a.x)[i] : make_uint4(0, 0, 0, 0));
  const int byte = mx_scale_byte<BITS>(block_magnitude(magnitude(x)));
  const float inv = mx_inverse(byte);
  if (!live) return;
  if constexpr (BITS == 8)
    static_cast<uint2*>(a.codes)[i] = codes8(x, inv);
  else
    static_cast<uint32_t*>(a.codes)[i] = codes4(x, inv);
  if ((i & 3) == 0) a.scales[i >> 2] = static_cast<uint8_t>(byte);
}

template <int BITS>
__global__ void __launch_bounds__(kThreads) mx_dequantize_kernel(const MxDequantArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= 4 * a.blocks) return;
  const float s = mx_scale(a.scales[i >> 2]);
  uint32_t w[4];
  if constexpr (BITS == 8) {
    const uint2 c = static_cast<const uint2*>(a.codes)[i];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 v = mx_values8((k < 2 ? c.x : c.y) >> (16 * (k & 1)));
      w[k] = pack_half2(__float2half_rn(v.x * s), __float2half_rn(v.y * s));
    }
  } else {
    const uint32_t c = static_cast<const uint32_t*>(a.codes)[i];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 v = mx_values4(c >> (8 * k));
      w[k] = pack_half2(__float2half_rn(v.x * s), __float2half_rn(v.y * s));
    }
  }
  reinterpret_cast<uint4*>(a.y)[i] = make_uint4(w[0], w[1], w[2], w[3]);
}

// One row a thread block: eight values a lane and step.  The row's h is read
// again (by the thread that wrote it, or x) for the second pass.
__global__ void __launch_bounds__(kThreads) mx_norm_kernel(const MxNormArgs a) {
  __shared__ float part[kThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const long long row = static_cast<long long>(blockIdx.x) * (a.K / 8);
  const uint4* x = reinterpret_cast<const uint4*>(a.x) + row;
  const uint4* r = a.res ? reinterpret_cast<const uint4*>(a.res) + row : nullptr;
  uint4* h = a.res ? reinterpret_cast<uint4*>(a.h) + row : nullptr;
  const int n = a.K / 8, whole = (n + 31) / 32 * 32;
  float sum = 0.f;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    Eight v = unpack(x[i]);
    if (r) {
      const Eight u = unpack(r[i]);
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = pack_half2(__float2half_rn(v.v[2 * k] + u.v[2 * k]),
                          __float2half_rn(v.v[2 * k + 1] + u.v[2 * k + 1]));
      h[i] = make_uint4(w[0], w[1], w[2], w[3]);
      v = unpack(make_uint4(w[0], w[1], w[2], w[3]));
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) sum = fmaf(v.v[k], v.v[k], sum);
  }
  for (int k = 16; k > 0; k /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, k);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int k = 0; k < kThreads / 32; ++k) sum += part[k];
  const float rstd = 1.0f / sqrtf(sum / static_cast<float>(a.K) + a.eps);
  for (int i = threadIdx.x; i < whole; i += kThreads) {
    const bool live = i < n;
    Eight v = unpack(live ? (r ? h[i] : x[i]) : make_uint4(0, 0, 0, 0));
    const Eight g = unpack(live ? reinterpret_cast<const uint4*>(a.gamma)[i] : make_uint4(0, 0, 0, 0));
#pragma unroll
    for (int k = 0; k < 8; ++k) v.v[k] = v.v[k] * rstd * g.v[k];
    const int byte = mx_scale_byte<8>(block_magnitude(magnitude(v)));
    if (live) {
      reinterpret_cast<uint2*>(a.codes)[row + i] = codes8(v, mx_inverse(byte));
      if ((i & 3) == 0) a.scales[(row + i) >> 2] = static_cast<uint8_t>(byte);
    }
  }
}

template <typename F, typename A>
cudaError_t launch(F* k, long long blocks, cudaStream_t st, const A& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, a);
}

}  // namespace

cudaError_t mx_quantize_launch(const MxQuantArgs& a, int bits, int, cudaStream_t st) {
  const long long blocks = (4 * a.blocks + kThreads - 1) / kThreads;
  return bits == 4 ? launch(mx_quantize_kernel<4>, blocks, st, a)
                   : launch(mx_quantize_kernel<8>, blocks, st, a);
}

cudaError_t mx_dequantize_launch(const MxDequantArgs& a, int bits, int, cudaStream_t st) {
  const long long blocks = (4 * a.blocks + kThreads - 1) / kThreads;
  return bits == 4 ? launch(mx_dequantize_kernel<4>, blocks, st, a)
                   : launch(mx_dequantize_kernel<8>, blocks, st, a);
}

cudaError_t mx_norm_launch(const MxNormArgs& a, int, cudaStream_t st) {
  return launch(mx_norm_kernel, a.M, st, a);
}

}  // namespace qgemv
