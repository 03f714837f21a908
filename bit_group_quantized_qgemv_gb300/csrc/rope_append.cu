// rope_append.cu -- qgemv_qk_norm_rope_append: per-head RMS norms of queries
// and keys, rotation by position and the append to the paged cache, one pass
// over the fused QKV vectors.
//
// A head is HD/8 lanes of a warp.  Lane l of a head holds two runs of four
// components, the first at 4l and the second rotary_dim/2 further on, so both
// components of every rotated pair (half-split or interleaved) lie in the
// same lane and the only exchange is the sum of squares of the norm.  The
// angle positions[t] * inv_freq[i] is reduced from its exact product (a
// float product and its rounding error, by fma), multiplied by 1/(2 pi) as a
// two-float constant: the fraction of a turn is right to about 2^-24 for any
// position, where a float angle would be off by position * 2^-24 radians.
// The sines are computed once per warp, which then walks several heads of
// its token.
#include "kv_cache.cuh"

namespace qgemv {
namespace {

constexpr int kWarps = 4;
constexpr int kUnroll = 4;  // heads of a lane group loaded before the first is processed

// 1 / (2 pi) as a sum of two floats (48 bits).
constexpr float kTurnHi = 0.15915494f;
constexpr float kTurnLo = static_cast<float>(0.15915494309189533576888 - static_cast<double>(kTurnHi));

// Turns in the angle x * f, less a whole number of them.
__device__ __forceinline__ float turns(float x, float f) {
  const float p = x * f;
  const float e = fmaf(x, f, -p);  // x * f = p + e exactly
  const float t = p * kTurnHi;
  const float te = fmaf(p, kTurnHi, -t);
  return (t - rintf(t)) + (te + fmaf(p, kTurnLo, e * kTurnHi));
}

// Sequence that token t belongs to (the last one that starts at or before it),
// -1 if none starts there; 32 starts are compared at a time.
__device__ __forceinline__ int find_seq(const int* q_start, int n_seqs, int t, int lane) {
  int lo = 0, n = n_seqs;  // candidates lo .. lo + n - 1
  while (true) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const unsigned le = __ballot_sync(0xFFFFFFFFu, i < lo + n && q_start[i] <= t);
    if (le == 0) return -1;
    const int c = 31 - __clz(le);
    const int end = lo + n;
    lo += c * step;
    n = min(step, end - lo);
    if (step == 1) return lo;
  }
}

template <int HD, bool INTER>
__global__ void __launch_bounds__(32 * kWarps) rope_append_kernel(const RopeArgs a, int per_warp,
                                                                  int groups) {
  constexpr int kLanes = HD / 8;            // lanes per head
  constexpr int kHeads = 32 / kLanes;       // heads a warp holds at once
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long task = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int l = lane % kLanes, sub = lane / kLanes;
  const int rd = a.rotary_dim, rl = rd / 8;
  const bool rot = l < rl;
  const int d0 = rot ? 4 * l : rd + 4 * (l - rl);
  const int d1 = rot ? rd / 2 + 4 * l : rd + (HD - rd) / 2 + 4 * (l - rl);
  // Weights, read before the wait for the previous kernel.
  float f[4] = {0.f, 0.f, 0.f, 0.f};
  if (rot)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      f[j] = a.inv_freq[INTER ? (j < 2 ? d0 / 2 + j : d1 / 2 + j - 2) : d0 + j];
  uint2 gq[2] = {}, gk[2] = {};
  if (a.q_norm != nullptr) {
    gq[0] = *reinterpret_cast<const uint2*>(a.q_norm + d0);
    gq[1] = *reinterpret_cast<const uint2*>(a.q_norm + d1);
    gk[0] = *reinterpret_cast<const uint2*>(a.k_norm + d0);
    gk[1] = *reinterpret_cast<const uint2*>(a.k_norm + d1);
  }
  pdl_wait();
  const int t = static_cast<int>(task / groups);
  if (t >= a.n_tokens) return;
  const int heads = a.n_q + 2 * a.c.n_kv;
  const int h0 = static_cast<int>(task % groups) * per_warp;
  const int h1 = min(h0 + per_warp, heads);

  const int pos = a.positions[t];
  const int s = find_seq(a.q_start, a.c.n_seqs, t, lane);
  if (s < 0) return;
  int first, count;
  seq_rows(a.q_start, s, a.n_tokens, a.err, &first, &count);
  if (t < first || t >= first + count) return;
  const int at = seq_len(a.c, s, a.err) - count + (t - first);
  int page = -1;
  if (at >= 0)
    page = page_of(a.c, s, at, a.err);
  else
    flag_error(a.err);

  float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
  if (rot) {
    // the position as two floats, exactly: 24 bits above, 8 below
    const float ph = static_cast<float>(pos & ~0xFF), pl = static_cast<float>(pos & 0xFF);
#pragma unroll
    for (int j = 0; j < 4; ++j) sincospif(2.0f * (turns(ph, f[j]) + turns(pl, f[j])), &sn[j], &cs[j]);
  }

  const __half* row = a.qkv + static_cast<long long>(t) * a.qkv_stride;
  for (int hb = h0; hb < h1; hb += kHeads * kUnroll) {
    uint2 x[kUnroll][2];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = hb + u * kHeads + sub;
      x[u][0] = x[u][1] = make_uint2(0u, 0u);
      if (h < h1) {
        x[u][0] = *reinterpret_cast<const uint2*>(row + h * HD + d0);
        x[u][1] = *reinterpret_cast<const uint2*>(row + h * HD + d1);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (hb + u * kHeads >= h1) break;  // the same for the whole warp
      const int h = hb + u * kHeads + sub;
      const bool is_q = h < a.n_q, is_v = h >= a.n_q + a.c.n_kv;
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w = j < 2 ? (j == 0 ? x[u][0].x : x[u][0].y) : (j == 2 ? x[u][1].x : x[u][1].y);
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w));
        v[2 * j] = p.x;
        v[2 * j + 1] = p.y;
      }
      if (a.q_norm != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o /= 2) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        const float r = 1.0f / sqrtf(ss * (1.0f / HD) + a.eps);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t wq = j < 2 ? (j == 0 ? gq[0].x : gq[0].y) : (j == 2 ? gq[1].x : gq[1].y);
          const uint32_t wk = j < 2 ? (j == 0 ? gk[0].x : gk[0].y) : (j == 2 ? gk[1].x : gk[1].y);
          const uint32_t w = is_q ? wq : wk;
          const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&w));
          v[2 * j] *= r * g.x;
          v[2 * j + 1] *= r * g.y;
        }
      }
      if (h >= h1) continue;
      uint2 y0, y1;
      if (is_v) {
        y0 = x[u][0];
        y1 = x[u][1];
      } else {
        float w[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // pair j: half-split (v[j], v[4 + j]), interleaved (v[2j], v[2j + 1])
          const int ia = INTER ? 2 * j : j, ib = INTER ? 2 * j + 1 : 4 + j;
          w[ia] = v[ia] * cs[j] - v[ib] * sn[j];
          w[ib] = v[ib] * cs[j] + v[ia] * sn[j];
        }
        if (!rot)
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = v[j];
        y0 = make_uint2(pack_f16(w[0], w[1]), pack_f16(w[2], w[3]));
        y1 = make_uint2(pack_f16(w[4], w[5]), pack_f16(w[6], w[7]));
      }
      __half* dst;
      if (is_q) {
        dst = a.q_out + static_cast<long long>(t) * a.q_stride + h * HD;
      } else {
        if (page < 0) continue;
        const int kh = h - a.n_q - (is_v ? a.c.n_kv : 0);
        dst = (is_v ? a.c.v : a.c.k) + cache_row(a.c, page, kh, at) * HD;
        if (!is_v && l == 0) {
          const long long e = (static_cast<long long>(s) * a.c.n_kv + kh) *
                                  (static_cast<long long>(a.c.max_pages) << a.c.page_shift) + at;
          if (a.entry_pos != nullptr) a.entry_pos[e] = pos;
          if (a.entry_mass != nullptr) a.entry_mass[e] = 0.f;
        }
      }
      *reinterpret_cast<uint2*>(dst + d0) = y0;
      *reinterpret_cast<uint2*>(dst + d1) = y1;
    }
  }
}

template <int HD, bool INTER>
cudaError_t launch_t(const RopeArgs& a, int sms, cudaStream_t st) {
  constexpr int kHeads = 32 * 8 / HD;
  const int heads = a.n_q + 2 * a.c.n_kv;
  const int batch = kHeads * kUnroll;  // heads of one pass of a warp's loop
  const int all = (heads + batch - 1) / batch;
  // Passes per warp: all of a token's heads once there are enough tokens to
  // fill the machine (48 warps a multiprocessor), else the heads are spread.
  long long passes = static_cast<long long>(a.n_tokens) * all / (static_cast<long long>(sms) * 48);
  if (passes > all) passes = all;
  int per_warp = static_cast<int>(passes) * batch;
  if (passes < 1) per_warp = kHeads;  // few tokens: one head per lane group
  const int groups = (heads + per_warp - 1) / per_warp;
  const long long blocks = (static_cast<long long>(a.n_tokens) * groups + kWarps - 1) / kWarps;
  if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_append_kernel<HD, INTER>, a, per_warp, groups);
}

}  // namespace

cudaError_t rope_append_launch(const RopeArgs& a, int sms, cudaStream_t st) {
  if (a.c.head_dim == 64)
    return a.interleaved ? launch_t<64, true>(a, sms, st) : launch_t<64, false>(a, sms, st);
  return a.interleaved ? launch_t<128, true>(a, sms, st) : launch_t<128, false>(a, sms, st);
}

}  // namespace qgemv
