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
// sum of floats: the fraction of a turn is right to 2^-22.8 (8.3e-7 radians, worked out
// exactly for 30000 positions up to 2^31 and frequencies up to 10^4), where a float angle
// would be off by position * 2^-24 radians.
// The sines are computed once per warp, which then walks several heads of
// its token.
#include "kv_cache.cuh"

namespace qgemv {
namespace {

constexpr int kWarps = 4;
// Blocks to a multiprocessor that the registers are cut for (measured with four
// groups of heads a pass, 7622 tokens of 48 heads: 5 blocks 38.1, 6 39.7, 7 36.2, 8
// 37.9, 10 47.2 us).  The normed forms spill 68 to 96 bytes at these 72 registers (with one
// group of heads a pass 4, for heads of 64), and are fastest all the same.
constexpr int kBlocks = 7;

// 1 / (2 pi) as a sum of floats: 48 bits, and 24 more.
constexpr float kTurnHi = 0.15915494f;
constexpr float kTurnLo = static_cast<float>(0.15915494309189533576888 - static_cast<double>(kTurnHi));
constexpr float kTurnLo2 = 7.342739e-17f;

// Turns in the angle x * f, less a whole number of them, for angles up to kFar: what
// is left of the products is then small enough not to be reduced itself.
constexpr float kFar = 1048576.0f;
__device__ __forceinline__ float turns(float x, float f) {
  const float p = x * f;
  const float e = fmaf(x, f, -p);  // x * f = p + e exactly
  const float t = p * kTurnHi;
  const float te = fmaf(p, kTurnHi, -t);
  return (t - rintf(t)) + (te + fmaf(p, kTurnLo, e * kTurnHi));
}

// The same for any angle: every product as a value, reduced, and its rounding error.
__device__ __forceinline__ float far_turns(float x, float f) {
  const float p = x * f, e = fmaf(x, f, -p);
  const float t = p * kTurnHi, te = fmaf(p, kTurnHi, -t);
  const float u = p * kTurnLo, v = e * kTurnHi;
  const float rest = fmaf(p, kTurnLo2, fmaf(p, kTurnLo, -u)) + fmaf(e, kTurnLo, fmaf(e, kTurnHi, -v));
  return (t - rintf(t)) + (((te - rintf(te)) + (u - rintf(u))) + ((v - rintf(v)) + rest));
}

// Eight fp16 values as floats.
__device__ __forceinline__ void unpack8(uint2 lo, uint2 hi, float* v) {
  const uint32_t w[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
    v[2 * j] = p.x;
    v[2 * j + 1] = p.y;
  }
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

// One pass of a warp: U groups of heads, kLanes lanes each, loaded
// together.  src, dst: this lane's head of the first group; heads: how many there are from
// the first group's first head on.
template <int HD, bool INTER, bool NORM, bool TURN, int U>
__device__ __forceinline__ void heads_pass(const __half* src, __half* dst, int src_step, int dst_step,
                                           int heads, int sub, int d0, int d1, const float* cg,
                                           bool rot, float eps) {
  constexpr int kLanes = HD / 8, kHeads = 32 / kLanes;
  uint2 x[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    x[u][0] = x[u][1] = make_uint2(0u, 0u);
    if (u * kHeads + sub < heads) {
      x[u][0] = *reinterpret_cast<const uint2*>(src + u * src_step + d0);
      x[u][1] = *reinterpret_cast<const uint2*>(src + u * src_step + d1);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (u * kHeads >= heads) break;  // the same for the whole warp
    uint2 y0 = x[u][0], y1 = x[u][1];
    if (TURN) {
      float v[8], w[8], r = 1.f;
      unpack8(y0, y1, v);
      if (NORM) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o /= 2) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        r = rsqrtf(fmaf(ss, 1.0f / HD, eps));
      }
      // cg: gamma_a cos, gamma_b sin, gamma_b cos, gamma_a sin of each pair
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // pair j: half-split (v[j], v[4 + j]), interleaved (v[2j], v[2j + 1])
        const int ia = INTER ? 2 * j : j, ib = INTER ? 2 * j + 1 : 4 + j;
        w[ia] = v[ia] * cg[4 * j] - v[ib] * cg[4 * j + 1];
        w[ib] = v[ib] * cg[4 * j + 2] + v[ia] * cg[4 * j + 3];
        if (!rot) {  // (0 times an infinity would not be nothing)
          w[ia] = v[ia] * cg[4 * j];
          w[ib] = v[ib] * cg[4 * j + 2];
        }
      }
      if (NORM)
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] *= r;
      y0 = make_uint2(pack_f16(w[0], w[1]), pack_f16(w[2], w[3]));
      y1 = make_uint2(pack_f16(w[4], w[5]), pack_f16(w[6], w[7]));
    }
    if (u * kHeads + sub < heads) {
      *reinterpret_cast<uint2*>(dst + u * dst_step + d0) = y0;
      *reinterpret_cast<uint2*>(dst + u * dst_step + d1) = y1;
    }
  }
}

// A warp's task: one token, passes p0 .. p1 of its heads.  The passes of
// a token are those of the queries, then the keys, then the values, each of
// per_pass heads of one kind.
template <int HD, bool INTER, bool NORM, int U>
__global__ void __launch_bounds__(32 * kWarps, kBlocks) rope_append_kernel(const RopeArgs a, int per_warp,
                                                                  int groups, int work) {
  constexpr int kLanes = HD / 8;       // lanes per head
  constexpr int kHeads = 32 / kLanes;  // heads a warp holds at once
  constexpr int kPerPass = kHeads * U;
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long task = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int l = lane % kLanes, sub = lane / kLanes;
  const int rd = a.rotary_dim, rl = rd / 8;
  const bool rot = l < rl;
  const int d0 = rot ? 4 * l : rd + 4 * (l - rl);
  const int d1 = rot ? rd / 2 + 4 * l : rd + (HD - rd) / 2 + 4 * (l - rl);
  pdl_wait();
  if (blockIdx.x >= work) {  // the checks of sequences that may have no token here
    const int i = static_cast<int>(blockIdx.x - work) * 32 * kWarps + threadIdx.x;
    if (i < a.c.n_seqs) check_seq(a.c, a.q_start, i, a.n_tokens, a.err);
    return;
  }
  const int t = static_cast<int>(task / groups);
  if (t >= a.n_tokens) return;
  // (frequencies and norms may be what the kernel before has just made: they are read
  // after the wait, along with the token's position and sequence)
  float f[4] = {0.f, 0.f, 0.f, 0.f};
  if (rot)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      f[j] = a.inv_freq[INTER ? (j < 2 ? d0 / 2 + j : d1 / 2 + j - 2) : d0 + j];
  uint2 g[2][2] = {};
  if (NORM) {
    g[0][0] = *reinterpret_cast<const uint2*>(a.q_norm + d0);
    g[0][1] = *reinterpret_cast<const uint2*>(a.q_norm + d1);
    g[1][0] = *reinterpret_cast<const uint2*>(a.k_norm + d0);
    g[1][1] = *reinterpret_cast<const uint2*>(a.k_norm + d1);
  }
  const int n_kv = a.c.n_kv;
  const int q_passes = (a.n_q + kPerPass - 1) / kPerPass, kv_passes = (n_kv + kPerPass - 1) / kPerPass;
  const int p0 = static_cast<int>(task % groups) * per_warp;
  const int p1 = min(p0 + per_warp, q_passes + 2 * kv_passes);

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
    float x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = turns(ph, f[j]) + turns(pl, f[j]);
    // (far angles are rare; all by that form, 7622 tokens took 36.5 us for 36.1)
    const float most = fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])));
    if ((fabsf(ph) + 256.0f) * most > kFar)
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = far_turns(ph, f[j]) + far_turns(pl, f[j]);
#pragma unroll
    for (int j = 0; j < 4; ++j) sincospif(2.0f * x[j], &sn[j], &cs[j]);
  }

  const __half* row = a.qkv + static_cast<long long>(t) * a.qkv_stride;
  const int page_size = 1 << a.c.page_shift;
  float cg[16];
  for (int p = p0; p < p1; ++p) {
    const int kind = p < q_passes ? 0 : p < q_passes + kv_passes ? 1 : 2;  // query, key, value
    const int pass = kind == 0 ? p : p - q_passes - (kind == 2 ? kv_passes : 0);
    if (kind < 2 && (p == p0 || pass == 0)) {
      float gm[8];
      unpack8(kind == 0 ? g[0][0] : g[1][0], kind == 0 ? g[0][1] : g[1][1], gm);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float ga = NORM ? gm[INTER ? 2 * j : j] : 1.f;
        const float gb = NORM ? gm[INTER ? 2 * j + 1 : 4 + j] : 1.f;
        cg[4 * j] = ga * cs[j];
        cg[4 * j + 1] = gb * sn[j];
        cg[4 * j + 2] = gb * cs[j];
        cg[4 * j + 3] = ga * sn[j];
      }
    }
    const int h = pass * kPerPass;  // first head of the pass, among its kind
    if (kind == 0) {
      heads_pass<HD, INTER, NORM, true, U>(
          row + (h + sub) * HD, a.q_out + static_cast<long long>(t) * a.q_stride + (h + sub) * HD,
          kHeads * HD, kHeads * HD, a.n_q - h, sub, d0, d1, cg, rot, a.eps);
    } else if (page >= 0) {
      const long long dst = cache_row(a.c, page, h + sub, at) * HD;
      const __half* src = row + (a.n_q + (kind == 2 ? n_kv : 0) + h + sub) * HD;
      const int step = kHeads * page_size * HD;
      if (kind == 2) {
        heads_pass<HD, INTER, NORM, false, U>(src, a.c.v + dst, kHeads * HD, step, n_kv - h, sub, d0, d1,
                                           cg, rot, a.eps);
      } else {
        heads_pass<HD, INTER, NORM, true, U>(src, a.c.k + dst, kHeads * HD, step, n_kv - h, sub, d0, d1,
                                          cg, rot, a.eps);
        const int n = min(kPerPass, n_kv - h);
        if (lane < n) {
          const long long e = (static_cast<long long>(s) * n_kv + h + lane) *
                                  (static_cast<long long>(a.c.max_pages) << a.c.page_shift) + at;
          if (a.entry_pos != nullptr) a.entry_pos[e] = pos;
          if (a.entry_mass != nullptr) a.entry_mass[e] = 0.f;
        }
      }
    }
  }
}

template <int HD, bool INTER, bool NORM, int U>
cudaError_t launch_t(const RopeArgs& a, int sms, cudaStream_t st) {
  constexpr int kPerPass = 32 * 8 / HD * U;  // heads of one pass
  const int all = (a.n_q + kPerPass - 1) / kPerPass + 2 * ((a.c.n_kv + kPerPass - 1) / kPerPass);
  // As many warps to a token as fill the machine (28 warps a multiprocessor),
  // down to one, which makes the token's sines once.
  long long split = (28LL * sms + a.n_tokens - 1) / a.n_tokens;
  if (split > all) split = all;
  const int per_warp = static_cast<int>((all + split - 1) / split);
  const int groups = (all + per_warp - 1) / per_warp;
  const long long blocks = (static_cast<long long>(a.n_tokens) * groups + kWarps - 1) / kWarps;
  // With an error flag, blocks of their own look at every sequence's start and length, so
  // that no token's warp waits for that.
  const int checks = a.err == nullptr ? 0 : (a.c.n_seqs + 32 * kWarps - 1) / (32 * kWarps);
  if (blocks + checks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks + checks));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_append_kernel<HD, INTER, NORM, U>, a, per_warp, groups,
                            static_cast<int>(blocks));
}

template <int HD, bool INTER, bool NORM>
cudaError_t launch_u(const RopeArgs& a, int sms, cudaStream_t st) {
  // One group of heads a pass while all of them together are a few warps to a
  // multiprocessor: a single token of 16/8 heads of 128 takes 2.5 us, with four
  // groups a pass 3.4; 61 tokens of 32/8 heads 3.4 and 2.7.
  constexpr int kHeads = 32 * 8 / HD;
  const long long warps =
      static_cast<long long>(a.n_tokens) * ((a.n_q + 2 * a.c.n_kv + kHeads - 1) / kHeads);
  return warps <= 4LL * sms ? launch_t<HD, INTER, NORM, 1>(a, sms, st)
                            : launch_t<HD, INTER, NORM, 4>(a, sms, st);
}

template <int HD>
cudaError_t launch_hd(const RopeArgs& a, int sms, cudaStream_t st) {
  if (a.q_norm != nullptr)
    return a.interleaved ? launch_u<HD, true, true>(a, sms, st) : launch_u<HD, false, true>(a, sms, st);
  return a.interleaved ? launch_u<HD, true, false>(a, sms, st) : launch_u<HD, false, false>(a, sms, st);
}

}  // namespace

cudaError_t rope_append_launch(const RopeArgs& a, int sms, cudaStream_t st) {
  return a.c.head_dim == 64 ? launch_hd<64>(a, sms, st) : launch_hd<128>(a, sms, st);
}

}  // namespace qgemv
