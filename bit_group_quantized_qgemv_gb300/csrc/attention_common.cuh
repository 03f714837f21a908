// attention_common.cuh -- what the paged-attention kernels share.
#pragma once

#include "kv_cache.cuh"

namespace qgemv {

constexpr float kLn2 = 0.69314718055994530942f;

// One row computed entry by entry in fp32, by a whole warp: taken where a
// value that the row does not see is an infinity or a NaN, which the tensor
// cores' 0 * v would carry into it.  Writes out and returns nothing else (the
// maximum and the sum are not affected by values).
template <int HD>
__device__ __noinline__ void slow_row(const AttnArgs& a, int s, int h, int t, int head, int last,
                                      int lane) {
  constexpr int D = HD / 32;
  const __half* q = a.q + static_cast<long long>(t) * a.q_stride + head * HD + lane * D;
  float qv[D], o[D], m = -INFINITY, l = 0.f;
  for (int d = 0; d < D; ++d) {
    qv[d] = __half2float(q[d]);
    o[d] = 0.f;
  }
  for (int j = 0; j <= last; ++j) {
    const int p = page_of(a.c, s, j, nullptr);
    if (p < 0) continue;
    const long long at = cache_row(a.c, p, h, j) * HD + lane * D;
    float x = 0.f;
    for (int d = 0; d < D; ++d) x = fmaf(qv[d], __half2float(a.c.k[at + d]), x);
    for (int k = 16; k > 0; k /= 2) x += __shfl_xor_sync(0xFFFFFFFFu, x, k);
    x *= a.scale_log2;
    const float mn = fmaxf(m, x), ms = mn == -INFINITY ? 0.f : mn;
    const float f = ex2(m - ms), w = ex2(x - ms);
    l = l * f + w;
    for (int d = 0; d < D; ++d) o[d] = o[d] * f + w * __half2float(a.c.v[at + d]);
    m = mn;
  }
  __half* y = a.out + static_cast<long long>(t) * a.out_stride + head * HD + lane * D;
  const float r = l > 0.f || !(l == l) ? 1.0f / l : 0.f;
  for (int d = 0; d < D; ++d) y[d] = __float2half_rn(o[d] * r);
}

// The output of one row, HD / 32 components per lane, divided by its sum and
// rounded; where the row hides entries and a component came out infinite or
// NaN, the row is computed again without the hidden values.
template <int HD>
__device__ __forceinline__ void store_row(const AttnArgs& a, int s, int h, int t, int head,
                                          int last, int len, const float* acc, float m, float l,
                                          int lane) {
  constexpr int D = HD / 32;
  const float inv = l > 0.f || !(l == l) ? 1.0f / l : 0.f;
  bool odd = false;
  __half* y = a.out + static_cast<long long>(t) * a.out_stride + head * HD + lane * D;
#pragma unroll
  for (int d = 0; d < D; ++d) {
    const float v = acc[d] * inv;
    odd |= !(fabsf(v) <= 3.0e38f);
    y[d] = __float2half_rn(v);
  }
  if (lane == 0 && a.lse != nullptr)
    a.lse[static_cast<long long>(t) * a.n_q + head] = (m + log2f(l)) * kLn2;
  if (__any_sync(0xFFFFFFFFu, odd) && last < len - 1) {
    __syncwarp();
    slow_row<HD>(a, s, h, t, head, last, lane);
  }
}

}  // namespace qgemv
