// mx_quantize.cu -- fp16 rows to microscaled values and back, and the residual
// addition with the RMS norm whose result leaves in MXFP8.
//
// A thread takes a block of 32 values: 64 bytes of fp16, 16 or 32 bytes of codes and a
// scale, in pieces of 32 bytes (a sector each) where the rows are aligned to that.  No
// lane needs another's value but for the norm's sum.  Bound by the bytes read and written;
// small calls by the launch.
#include "mx.h"
#include "mx_format.cuh"
#include "qgemv_device.cuh"

namespace qgemv {
namespace {

constexpr int kThreads = 256;

struct Block16 {
  uint32_t w[16];  // 32 fp16 values
};

__device__ __forceinline__ void load32(uint32_t* w, const void* p) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}
__device__ __forceinline__ void store32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; }

// N words (a multiple of four) from or to 16-byte aligned memory.
template <int N>
__device__ __forceinline__ void load_words(uint32_t* w, const void* p, bool wide) {
  if (N % 8 == 0 && wide) {
#pragma unroll
    for (int i = 0; i < N; i += 8) load32(w + i, static_cast<const uint32_t*>(p) + i);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint32_t*>(p) + i);
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
  }
}
template <int N>
__device__ __forceinline__ void store_words(void* p, const uint32_t* w, bool wide) {
  if (N % 8 == 0 && wide) {
#pragma unroll
    for (int i = 0; i < N; i += 8) store32(static_cast<uint32_t*>(p) + i, w + i);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<uint4*>(static_cast<uint32_t*>(p) + i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  }
}

__device__ __forceinline__ float2 unpack(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

template <int BITS>
__global__ void __launch_bounds__(kThreads) mx_quantize_kernel(const MxQuantArgs a) {
  constexpr int kWords = BITS;  // of codes
  pdl_launch_dependents();
  pdl_wait();
  const long long b = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  if (b >= a.blocks) return;
  uint32_t x[16];
  load_words<16>(x, a.x + b * 32, aligned32(a.x));
  uint32_t most = 0;  // largest magnitudes as bits; a NaN's are above an infinity's
#pragma unroll
  for (int i = 0; i < 16; ++i) most = __vmaxu2(most, x[i] & 0x7FFF7FFFu);
  const uint16_t top = static_cast<uint16_t>(max(most & 0xFFFFu, most >> 16));
  const int byte = mx_scale_byte<BITS>(__half2float(__ushort_as_half(top)));
  const float inv = mx_inverse(byte);
  uint32_t c[kWords];
  if constexpr (BITS == 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 u = unpack(x[2 * i]), v = unpack(x[2 * i + 1]);
      c[i] = mx_codes8(u.x * inv, u.y * inv) | (mx_codes8(v.x * inv, v.y * inv) << 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 u = unpack(x[4 * i + j]);
        c[i] |= mx_codes4(u.x * inv, u.y * inv) << (8 * j);
      }
    }
  }
  store_words<kWords>(static_cast<uint32_t*>(a.codes) + b * kWords, c, aligned32(a.codes));
  a.scales[b] = static_cast<uint8_t>(byte);
}

template <int BITS>
__global__ void __launch_bounds__(kThreads) mx_dequantize_kernel(const MxDequantArgs a) {
  constexpr int kWords = BITS;
  pdl_launch_dependents();
  pdl_wait();
  const long long b = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  if (b >= a.blocks) return;
  uint32_t c[kWords], y[16];
  load_words<kWords>(c, static_cast<const uint32_t*>(a.codes) + b * kWords, aligned32(a.codes));
  const float s = mx_scale(a.scales[b]);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 v = BITS == 8 ? mx_values8(c[i / 2] >> (16 * (i & 1))) : mx_values4(c[i / 4] >> (8 * (i & 3)));
    y[i] = pack_half2(__float2half_rn(v.x * s), __float2half_rn(v.y * s));
  }
  store_words<16>(a.y + b * 32, y, aligned32(a.y));
}

// T threads a row, the block's rows one behind the other; ONE: a thread has a single
// block of its row, which stays in registers; else h (or x) is read again.
template <bool ONE>
__global__ void __launch_bounds__(ONE ? kThreads : 1024) mx_norm_kernel(const MxNormArgs a, int T) {
  __shared__ float part[32];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blocks = a.K / kMxBlock, t = threadIdx.x % T, warps = T / 32;
  const long long row = static_cast<long long>(blockIdx.x) * (blockDim.x / T) + threadIdx.x / T;
  const bool live = row < a.M;
  const __half* x = a.x + row * a.K;
  const __half* r = a.res ? a.res + row * a.K : nullptr;
  __half* h = a.h + row * a.K;
  const bool wide = aligned32(a.x) && aligned32(a.res) && aligned32(a.res ? a.h : nullptr);
  float sum = 0.f;
  uint32_t v[16], g[16];
  // h of block i, which is written where there is a residual
  auto add = [&](int i) {
    load_words<16>(v, x + 32 * i, wide);
    if (r) {
      uint32_t u[16];
      load_words<16>(u, r + 32 * i, wide);
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float2 p = unpack(v[k]), q = unpack(u[k]);
        v[k] = pack_half2(__float2half_rn(p.x + q.x), __float2half_rn(p.y + q.y));
      }
      store_words<16>(h + 32 * i, v, wide);
    }
    float s[4] = {};
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float2 p = unpack(v[k]);
      s[k & 3] = fmaf(p.x, p.x, s[k & 3]);
      s[k & 3] = fmaf(p.y, p.y, s[k & 3]);
    }
    sum += (s[0] + s[1]) + (s[2] + s[3]);
  };
  auto gamma = [&](int i) { load_words<16>(g, a.gamma + 32 * i, aligned32(a.gamma)); };
  if constexpr (ONE) {
    if (live && t < blocks) {
      gamma(t);
      add(t);
    }
  } else if (live) {
    for (int i = t; i < blocks; i += T) add(i);
  }
#pragma unroll
  for (int k = 16; k > 0; k /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, k);
  if (warps > 1) {
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    sum = 0.f;
    const int from = warp / warps * warps;
    for (int k = 0; k < warps; ++k) sum += part[from + k];
  }
  const float rstd = 1.0f / sqrtf(sum / static_cast<float>(a.K) + a.eps);
  auto out = [&](int i) {
    float n[32];
    uint32_t most = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float2 p = unpack(v[k]), q = unpack(g[k]);
      n[2 * k] = p.x * rstd * q.x;
      n[2 * k + 1] = p.y * rstd * q.y;
      most = max(most, max(__float_as_uint(n[2 * k]) & 0x7FFFFFFFu, __float_as_uint(n[2 * k + 1]) & 0x7FFFFFFFu));
    }
    const int byte = mx_scale_byte<8>(__uint_as_float(most));
    const float inv = mx_inverse(byte);
    uint32_t c[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      c[k] = mx_codes8(n[4 * k] * inv, n[4 * k + 1] * inv) | (mx_codes8(n[4 * k + 2] * inv, n[4 * k + 3] * inv) << 16);
    const long long b = row * blocks + i;
    store_words<8>(a.codes + b * 32, c, aligned32(a.codes));
    a.scales[b] = static_cast<uint8_t>(byte);
  };
  if (!live) return;
  if constexpr (ONE) {
    if (t < blocks) out(t);
  } else {
    const __half* from = r ? h : x;
    for (int i = t; i < blocks; i += T) {
      load_words<16>(v, from + 32 * i, wide);
      gamma(i);
      out(i);
    }
  }
}

template <typename F, typename... A>
cudaError_t launch(F* k, long long blocks, int threads, cudaStream_t st, A... a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, a...);
}

}  // namespace

cudaError_t mx_quantize_launch(const MxQuantArgs& a, int bits, int, cudaStream_t st) {
  const long long blocks = (a.blocks + kThreads - 1) / kThreads;
  return bits == 4 ? launch(mx_quantize_kernel<4>, blocks, kThreads, st, a)
                   : launch(mx_quantize_kernel<8>, blocks, kThreads, st, a);
}

cudaError_t mx_dequantize_launch(const MxDequantArgs& a, int bits, int, cudaStream_t st) {
  const long long blocks = (a.blocks + kThreads - 1) / kThreads;
  return bits == 4 ? launch(mx_dequantize_kernel<4>, blocks, kThreads, st, a)
                   : launch(mx_dequantize_kernel<8>, blocks, kThreads, st, a);
}

cudaError_t mx_norm_launch(const MxNormArgs& a, int, cudaStream_t st) {
  // A thread a block of the row, up to 1024 of them.  Short rows share a thread block of 128
  // (with 256 or 512, 2048 rows of 4096 take 0.6 or 1.4 us more: fewer of them at a time).
  const int warps = (a.K / kMxBlock + 31) / 32, T = 32 * (warps < 32 ? warps : 32);
  if (T > kThreads) return launch(mx_norm_kernel<false>, a.M, T, st, a, T);
  const int rows = T < 128 ? 128 / T : 1;
  return launch(mx_norm_kernel<true>, (a.M + rows - 1LL) / rows, rows * T, st, a, T);
}

}  // namespace qgemv
