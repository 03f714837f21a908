// attention_common.cuh -- what the paged-attention kernels share.
#pragma once

#include "kv_cache.cuh"

namespace qgemv {

constexpr float kLn2 = 0.69314718055994530942f;

// Weights enter the product with v as fp16, relative to 2^base (the kernels' m): a
// base is a row's maximum at some time less kLift, in log2 units, and moves once a
// weight would pass 2^kTop.  Of an entry far below the maximum 2^-32 of the largest weight is the
// most that a rounding then takes or adds (2^-25 with the maximum as the base: one heavy
// entry in front of 3000 that are 18 nats lighter left nothing of them, or added half as much
// again).  kTop leaves a factor of 2 below the end of fp16 for what ex2 errs.  From 2^26 on,
// where floats are 8 apart, the maximum itself is the base.
constexpr float kLift = 7.0f, kTop = 15.0f;
__device__ __forceinline__ float base_of(float most) {
  return fabsf(most) < 67108864.0f ? most - kLift : most;
}

// One row computed again in fp32 by a whole warp, from the entries that it sees
// alone: taken where a value that the row does not see is an infinity or a NaN,
// which the tensor cores' 0 * v would carry into it.  Writes out only (the
// maximum and the sum are not affected by values).  32 entries at a time: a lane
// takes the score of one of them, then its HD / 32 components of all of them, so
// that the loads of a step do not wait for one another.  (In the many-rows kernel
// the block's other warps wait meanwhile: a step of 3 us puts 32 rows over 3 million
// entries at their limit, where the call ends with a status and without these rows.)
template <int HD>
__device__ __noinline__ void slow_row(const AttnArgs& a, int s, int h, int t, int head, int last,
                                      int lane) {
  constexpr int D = HD / 32;
  const uint4* q = reinterpret_cast<const uint4*>(a.q + static_cast<long long>(t) * a.q_stride +
                                                  head * HD);
  float o[D] = {}, m = -INFINITY, l = 0.f;
  for (int j0 = 0; j0 <= last; j0 += 32) {
    const int j = j0 + lane, p = j <= last ? page_of(a.c, s, j, nullptr) : -1;
    const long long at = p >= 0 ? cache_row(a.c, p, h, j) * HD : -1;
    float x = -INFINITY;
    if (at >= 0) {
      const uint4* k = reinterpret_cast<const uint4*>(a.c.k + at);
      x = 0.f;
#pragma unroll 4
      for (int i = 0; i < HD / 8; ++i) {
        const uint4 kv = k[i], qv = q[i];
        const uint32_t kw[4] = {kv.x, kv.y, kv.z, kv.w}, qw[4] = {qv.x, qv.y, qv.z, qv.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 kf = __half22float2(*reinterpret_cast<const __half2*>(&kw[e]));
          const float2 qf = __half22float2(*reinterpret_cast<const __half2*>(&qw[e]));
          x = fmaf(qf.x, kf.x, x);
          x = fmaf(qf.y, kf.y, x);
        }
      }
      x *= a.scale_log2;
    }
    float mn = x;
    for (int k = 16; k > 0; k /= 2) mn = fmaxf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, k));
    mn = fmaxf(m, mn);
    const float ms = mn == -INFINITY ? 0.f : mn, f = ex2(m - ms), w = ex2(x - ms);
    float sum = w;
    for (int k = 16; k > 0; k /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, k);
    l = l * f + sum;
    m = mn;
#pragma unroll
    for (int d = 0; d < D; ++d) o[d] *= f;
#pragma unroll 8
    for (int e = 0; e < 32; ++e) {
      const float we = __shfl_sync(0xFFFFFFFFu, w, e);
      const long long ae = __shfl_sync(0xFFFFFFFFu, at, e);
      if (ae < 0) continue;
#pragma unroll
      for (int d = 0; d < D; ++d)
        o[d] = fmaf(we, __half2float(a.c.v[ae + lane * D + d]), o[d]);
    }
  }
  __half* y = a.out + static_cast<long long>(t) * a.out_stride + head * HD + lane * D;
  const float r = l > 0.f || !(l == l) ? 1.0f / l : 0.f;
#pragma unroll
  for (int d = 0; d < D; ++d) y[d] = __float2half_rn(o[d] * r);
}

// The output of one row, HD / 32 components per lane, divided by its sum and
// rounded; where the row hides entries and a component came out infinite or
// NaN, the row is computed again without the hidden values (but not where the sum
// of the weights is a NaN, which values do not enter).
template <int HD>
__device__ __forceinline__ void store_row(const AttnArgs& a, int s, int h, int t, int head,
                                          int last, int len, const float* acc, float m, float l,
                                          int lane) {
  constexpr int D = HD / 32;
  const float inv = l > 0.f || !(l == l) ? 1.0f / l : 0.f;
  bool odd = false;
  float v[D];
#pragma unroll
  for (int d = 0; d < D; ++d) {
    v[d] = acc[d] * inv;
    odd |= !(fabsf(v[d]) <= 3.0e38f);
  }
  uint32_t* y = reinterpret_cast<uint32_t*>(a.out + static_cast<long long>(t) * a.out_stride +
                                            head * HD + lane * D);
  if constexpr (D == 4)
    *reinterpret_cast<uint2*>(y) = make_uint2(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]));
  else
    *y = pack_f16(v[0], v[1]);
  if (lane == 0 && a.lse != nullptr)
    a.lse[static_cast<long long>(t) * a.n_q + head] = (m + log2f(l)) * kLn2;
  if (__any_sync(0xFFFFFFFFu, odd) && l == l && last < len - 1) {
    __syncwarp();
    slow_row<HD>(a, s, h, t, head, last, lane);
  }
}

}  // namespace qgemv
