// attention_mass.cu -- qgemv_attention_mass: the attention weight every
// cached entry receives from the new tokens.
//
//   mass_out[j] = mass[j] + sum_r exp2(scale_log2 q_r . k_j - lse2_r)
// over the rows r = (token, head of the group) that see entry j.  lse is known,
// so no softmax statistics are carried, every entry is summed on its own in
// the order of the rows, and nothing has to be joined: only K is read.
//
// Few rows (decode steps): the keys stream through shared memory in tiles of
// 16 entries, a ring per warp (cp.async), S^T = K Q^T by m16n8k16 with the rows
// as columns.  Bound by HBM.
// Many rows (chunks): a block keeps 256 entries' keys in shared memory as the
// A operands of tcgen05 products and walks the query rows 128 at a time, one
// TMA box each; thread e of a softmax warpgroup owns entry e: its row of
// scores lies in its lane of tensor memory, so the sum over the rows is a sum
// over columns in one thread.  Scores are double-buffered (4 x 128 columns).
// 256 entries a block halve the query traffic, which 128 would put at the
// multiprocessor's share of the L2 bandwidth (32 KB per 512 clocks of products).
// 511 tokens over 16411 entries (32/8 heads of 128, 67.6 GFLOP) take 68 us; the
// products alone, both operands from shared memory, and the sums alone took 65 of 74.
#include <atomic>

#include "kv_tensor_map.h"
#include "mma_tile.cuh"
#include "runs.cuh"
#include "tcgen05.cuh"

namespace qgemv {
namespace {

__device__ unsigned g_status = 0;

constexpr float kLog2e = 1.4426950408889634f;

// Entries of sequence i, whose new tokens are checked too: one without entries has no
// share of the work, and nobody else would look at them.
__device__ __forceinline__ int checked_len(const MassArgs& a, int i) {
  if (a.err != nullptr) {
    int first, count;
    seq_rows(a.q_start, i, a.n_tokens, a.err, &first, &count);
    if (count > a.max_q) flag_error(a.err);
  }
  return seq_len(a.c, i, a.err);
}

// ------------------------------------------------------------- few rows
constexpr int kWarps = 4;
constexpr int kTile = 16;
// Ring depth of each warp (16 sequences of 500 to 16000 entries: two stages 30.0
// us, three 31.4, four 33.2, six 37.1; one of 30000: 12.9, 10.8, 11.9, 13.7: more
// blocks to a multiprocessor serve better than deeper rings).
constexpr int kStages = 3;
constexpr int kRowsMax = 32;  // rows of one walk over the entries

template <int HD>
__host__ __device__ constexpr int key_bytes() {
  return kTile * HD * 2;
}

// Blocks resident on a multiprocessor, by the registers of the rows.
__host__ __device__ constexpr int few_resident(int nt) { return nt > 2 ? 2 : 4; }

template <int HD, int NT>
__global__ void __launch_bounds__(32 * kWarps, few_resident(NT)) mass_few_kernel(const MassArgs a) {
  constexpr int kM = HD / 16, kChunks = HD / 8, kRows = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  // blocks of 64 entries of a sequence's units
  auto blocks_of = [&](int i) { return (checked_len(a, i) + 63) / 64; };
  int s, h, j0;
  long long per, left = run_start(a.c.n_seqs, a.c.n_kv, 2, lane, blocks_of, &per, &s, &h, &j0);
  while (left > 0) {  // segments of this block's run
    const int len = seq_len(a.c, s, nullptr);
    int first, count;
    seq_rows(a.q_start, s, a.n_tokens, nullptr, &first, &count);
    const int j1 = static_cast<int>(min(static_cast<long long>((len + 63) / 64), j0 + left));
    const int k0 = j0 * 64, k1 = min(len, j1 * 64);
    left -= j1 - j0;
    const int rows = min(count, a.max_q) * a.group, off = len - count;
    const int tiles = (k1 - k0 + kTile - 1) / kTile;
    const int mine = tiles > warp ? (tiles - warp + kWarps - 1) / kWarps : 0;
    const uint32_t ring = smem_u32(smem) + warp * (kStages * key_bytes<HD>());
    const long long entries = (static_cast<long long>(s) * a.c.n_kv + h) *
                              (static_cast<long long>(a.c.max_pages) << a.c.page_shift);

    int r0 = 0;
    do {  // one walk over the entries for every kRows rows (and one if there are none)
      const int nr = min(kRows, rows - r0);
      uint32_t qf[NT][kM][2];
      float ls[NT][2];
      int lim[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = nt * 8 + g;
        const __half* q = a.q + static_cast<long long>(first + (r0 + r) / a.group) * a.q_stride +
                          (h * a.group + (r0 + r) % a.group) * HD + 2 * tq;
#pragma unroll
        for (int k = 0; k < kM; ++k) {
          qf[nt][k][0] = r < nr ? *reinterpret_cast<const uint32_t*>(q + 16 * k) : 0u;
          qf[nt][k][1] = r < nr ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 8) : 0u;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = nt * 8 + 2 * tq + e, rr = r0 + c;
          float v = -INFINITY;
          if (c < nr)
            v = a.lse[static_cast<long long>(first + rr / a.group) * a.n_q + h * a.group + rr % a.group];
          lim[nt][e] = c < nr && v != -INFINITY ? off + rr / a.group : -1;  // a row that saw nothing
          ls[nt][e] = v * kLog2e;
        }
      }
      unsigned bad = 0;
      int next = mine > 0 ? raw_page(a.c, s, k0 + warp * kTile) : -1;
      auto issue = [&](int it) {
        if (it < mine) {
          const int e0 = k0 + (it * kWarps + warp) * kTile, st = it % kStages;
          const uint32_t kd = ring + st * key_bytes<HD>();
          const int page = good_page(a.c, next, a.err);
          const long long base = page >= 0 ? cache_row(a.c, page, h, e0) * HD : 0;
          const int end = page >= 0 ? len : 0;
          bad = page >= 0 ? bad & ~(1u << st) : bad | (1u << st);
#pragma unroll
          for (int c = 0; c < kTile * kChunks / 32; ++c) {
            const int id = c * 32 + lane, r = id / kChunks, ch = id % kChunks;
            cp_async16(kd + tile_off<HD>(r, ch), a.c.k + base + id * 8, e0 + r < end);
          }
          if (it + 1 < mine) next = raw_page(a.c, s, e0 + kWarps * kTile);
        }
        cp_commit();
      };
#pragma unroll
      for (int p = 0; p < kStages - 1; ++p) issue(p);
      const float* src = r0 == 0 ? a.mass : a.mass_out;
      const int kr = (lane & 7) + (((lane >> 3) & 1) << 3), kc = lane >> 4;
      for (int it = 0; it < mine; ++it) {
        const int e0 = k0 + (it * kWarps + warp) * kTile, st = it % kStages;
        // the entry this thread writes: tq 0 those of g, tq 1 those of g + 8
        const int j_out = e0 + g + 8 * tq;
        const bool writes = tq < 2 && j_out < len;
        float before = 0.f;
        if (writes && src != nullptr) before = src[entries + j_out];
        cp_wait<kStages - 2>();
        __syncwarp();
        issue(it + kStages - 1);
        const uint32_t kd = ring + st * key_bytes<HD>();
        float sc[NT][2][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[nt][0][e] = sc[nt][1][e] = 0.f;
#pragma unroll
        for (int k = 0; k < kM; ++k) {
          uint32_t kf[4];
          ldsm4(kf, kd + tile_off<HD>(kr, 2 * k + kc));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(sc[nt][k & 1], kf, qf[nt][k][0], qf[nt][k][1]);
        }
        const bool hidden = (bad >> st) & 1;
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float w =
                ex2(fmaf(sc[nt][0][e] + sc[nt][1][e], a.scale_log2, -ls[nt][e & 1]));
            if (!hidden && e0 + g + 8 * (e >> 1) <= lim[nt][e & 1]) sum[e >> 1] += w;
          }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], 1);
          sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], 2);
        }
        if (writes) a.mass_out[entries + j_out] = before + (tq == 0 ? sum[0] : sum[1]);
        __syncwarp();
      }
      cp_wait<0>();
      __syncwarp();
      r0 += kRows;
    } while (r0 < rows);
    j0 = 0;
    if (left > 0 && ++h == a.c.n_kv) {
      h = 0;
      s = run_next(s, a.c.n_seqs, lane, blocks_of);
      if (s >= a.c.n_seqs) return;
    }
  }
}

// ------------------------------------------------------------ many rows
constexpr int kBlock = 128;  // entries of a tile, rows of a step
constexpr int kManyThreads = 384;
constexpr int kSlots = 3;    // query tiles in flight
constexpr int kAhead = 4;    // shares found ahead

template <int HD>
struct Shape {
  static constexpr int kHalves = HD / 64;
  static constexpr int kBytes = kBlock * HD * 2;
  static constexpr int kSmem = 1024 + (4 + kSlots) * kBytes;
  static_assert(kSmem + 1536 <= 227 * 1024, "dynamic and static shared memory");
  static constexpr uint32_t kDesc = tc::idesc_f16(kBlock, kBlock, false);
};

struct Bars {
  uint64_t keys[2], k_empty[2], q_full[kSlots], q_empty[kSlots], s_full[2][2], s_empty[2][2],
      l_full[2], l_empty[2], share_full[kAhead], share_empty[kAhead], drain;
};

// A block's share: 256 entries of one head of one sequence (s -1: no more), in two
// tiles, or one of them alone.
struct Share {
  int s, h, e0, len, first, tokens, off, from, steps, tiles;
};

// Pairs of tiles of sequence i's units, and share number b of all: pairs, the
// first `whole` of them as they are, then the tiles of the rest one by one.  A whole warp.
__device__ __forceinline__ int shares_of(int len) { return (len + 2 * kBlock - 1) / (2 * kBlock); }
__device__ __forceinline__ void get_share(const MassArgs& a, long long b, long long whole,
                                          int step_tokens, int lane, Share* w) {
  int j;
  const int half = b < whole ? -1 : static_cast<int>((b - whole) & 1);
  if (half >= 0) b = whole + ((b - whole) >> 1);
  run_seek(b, a.c.n_seqs, a.c.n_kv, lane, [&](int i) { return shares_of(seq_len(a.c, i, nullptr)); }, &w->s,
           &w->h, &j);
  w->e0 = j * 2 * kBlock + max(half, 0) * kBlock;
  w->len = seq_len(a.c, w->s, nullptr);
  w->tiles = half >= 0 || w->e0 + kBlock >= w->len ? 1 : 2;
  int count;
  seq_rows(a.q_start, w->s, a.n_tokens, nullptr, &w->first, &count);
  w->tokens = min(count, a.max_q);
  w->off = w->len - count;
  // steps of step_tokens tokens, from the one whose last token sees entry e0
  w->from = max(0, w->e0 - w->off) / step_tokens;
  w->steps = w->e0 < w->len ? max(0, (w->tokens + step_tokens - 1) / step_tokens - w->from) : 0;
}

// What entry e of a share receives, computed again in fp32 by one thread, from the rows
// that count alone: taken where the sum came out a NaN, which may stem from a row whose lse
// is -inf (it adds nothing, but its score, and so its weight in the sums below, may be a NaN).
// Here because it costs nothing elsewhere: a test of every lse took 511 tokens over 16411
// entries from 69.5 to 75.5 us, a flag for each step and a loop of its own to 72.8.  (The
// other warps wait meanwhile: a row takes about a microsecond, so ten million rows are at
// their limit, where the call ends with a status and without these entries.)
template <int HD>
__device__ __noinline__ float slow_sum(const MassArgs& a, int h, int first, int tokens, int off, int e,
                                       int page) {
  const uint4* k = reinterpret_cast<const uint4*>(a.c.k + cache_row(a.c, page, h, e) * HD);
  float sum = 0.f;
  for (int t = max(0, e - off); t < tokens; ++t)
    for (int i = 0; i < a.group; ++i) {
      const int head = h * a.group + i;
      const float lse = a.lse[static_cast<long long>(first + t) * a.n_q + head];
      if (lse == -INFINITY) continue;
      const uint4* q = reinterpret_cast<const uint4*>(
          a.q + static_cast<long long>(first + t) * a.q_stride + head * HD);
      float x = 0.f;
#pragma unroll 4
      for (int c = 0; c < HD / 8; ++c) {
        const uint4 kv = k[c], qv = q[c];
        const uint32_t kw[4] = {kv.x, kv.y, kv.z, kv.w}, qw[4] = {qv.x, qv.y, qv.z, qv.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 kf = __half22float2(*reinterpret_cast<const __half2*>(&kw[j]));
          const float2 qf = __half22float2(*reinterpret_cast<const __half2*>(&qw[j]));
          x = fmaf(qf.x, kf.x, x);
          x = fmaf(qf.y, kf.y, x);
        }
      }
      sum += ex2(fmaf(x, a.scale_log2, lse * -kLog2e));
      if (!(sum == sum)) return sum;  // a row that counts has a NaN
    }
  return sum;
}

// One block per multiprocessor, each taking every gridDim.x-th share.  Warp 11
// finds them ahead of the others (lengths and starts are three loads in a row, 2 us of
// a share's 18 when every warp looked for itself), the producer is ahead of the sums
// (two buffers of keys), so that a share's start hides behind the one before it.
template <int HD>
__global__ void __launch_bounds__(kManyThreads, 1)
    mass_many_kernel(const MassArgs a, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap q_map, int step_tokens) {
  using Sh = Shape<HD>;
  extern __shared__ uint8_t raw[];
  __shared__ Bars bars;
  __shared__ uint32_t s_tmem;
  __shared__ int s_failed;  // a wait ran out
  __shared__ __align__(16) float s_lse[2][kBlock];
  __shared__ Share s_share[kAhead];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint8_t* qring = base + 4 * Sh::kBytes;
  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(smem_u32(&bars.keys[x]), 1);
      mbar_init(smem_u32(&bars.k_empty[x]), 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_u32(&bars.q_full[i]), 1);
      mbar_init(smem_u32(&bars.q_empty[i]), 1);
    }
    for (int x = 0; x < 2; ++x) {
      for (int d = 0; d < 2; ++d) {
        mbar_init(smem_u32(&bars.s_full[x][d]), 1);
        mbar_init(smem_u32(&bars.s_empty[x][d]), 4);  // one arrival per warp
      }
      mbar_init(smem_u32(&bars.l_full[x]), 1);
      mbar_init(smem_u32(&bars.l_empty[x]), 8);
    }
    for (int i = 0; i < kAhead; ++i) {
      mbar_init(smem_u32(&bars.share_full[i]), 1);
      mbar_init(smem_u32(&bars.share_empty[i]), 11);  // every warp but the finder
    }
    mbar_init(smem_u32(&bars.drain), 1);
    fence_mbar_init();
    s_failed = 0;
  }
  // Tensor memory is taken behind the kernel before and ahead of the one behind: no block
  // holds some while it waits for a block that may need it, on the same multiprocessor, to end.
  pdl_wait();
  if (warp == 8) tc::alloc(smem_u32(&s_tmem), 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = s_tmem;
  Share w;
  // Share number n of this block, as every warp but the finder reads it; false
  // behind the last.
  auto next_share = [&](int n) {
    const int i = n % kAhead;
    step_wait(smem_u32(&bars.share_full[i]), (n / kAhead) & 1, &s_failed, &g_status);
    w = s_share[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars.share_empty[i]));
    // (no shares are taken after a wait ran out)
    return __all_sync(0xFFFFFFFFu, w.s >= 0 && *static_cast<volatile int*>(&s_failed) == 0);
  };

  if (warp == 9) {
    // ---------------------------------------------------------- producer
    const int page_rows = min(1 << a.c.page_shift, kBlock), boxes = kBlock / page_rows;
    const int beyond = (a.c.n_pages * a.c.n_kv) << a.c.page_shift;
    // queries: [token][head of the group] rows of 128 bytes
    const uint32_t bytes = static_cast<uint32_t>(step_tokens * a.group * HD * 2);
    int kb = 0, g = 0;
    bool ok = true;
    for (int n = 0; ok && next_share(n); ++n) {
      if (w.steps == 0) continue;
      const int kd = kb & 1;
      if (kb > 1) ok = warp_wait(smem_u32(&bars.k_empty[kd]), (kb / 2 - 1) & 1, &g_status);
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(smem_u32(&bars.keys[kd]), w.tiles * Sh::kBytes);
      __syncwarp();
      if (lane < w.tiles * boxes) {
        const int x = lane / boxes, e = w.e0 + lane * page_rows;
        const int p = e < w.len ? page_of(a.c, w.s, e, a.err) : -1;
        const int row = p < 0 ? beyond : static_cast<int>(cache_row(a.c, p, w.h, e));
        const uint32_t dst =
            smem_u32(base + (2 * kd + x) * Sh::kBytes) + (lane % boxes) * page_rows * 128;
#pragma unroll
        for (int c = 0; c < Sh::kHalves; ++c)
          tc::tma_2d(dst + c * (kBlock * 128), &k_map, c * 64, row, smem_u32(&bars.keys[kd]));
      }
      __syncwarp();
      ++kb;
      for (int j = 0; j < w.steps; ++j) {
        const int slot = g % kSlots, use = g / kSlots;
        if (use > 0) ok = warp_wait(smem_u32(&bars.q_empty[slot]), (use - 1) & 1, &g_status);
        if (!ok) break;
        if (lane == 0) {
          const uint32_t full = smem_u32(&bars.q_full[slot]);
          mbar_arrive_expect_tx(full, bytes);
#pragma unroll
          for (int c = 0; c < Sh::kHalves; ++c)
            tc::tma_3d(smem_u32(qring + slot * Sh::kBytes) + c * (kBlock * 128), &q_map, c * 64,
                       w.h * a.group, w.first + (w.from + j) * step_tokens, full);
        }
        __syncwarp();
        ++g;
      }
    }
    // no copy may be in flight when the block ends
    for (int k = max(0, kb - 2); k < kb; ++k)
      warp_wait(smem_u32(&bars.keys[k & 1]), (k / 2) & 1, &g_status);
    for (int j = max(0, g - kSlots); j < g; ++j)
      warp_wait(smem_u32(&bars.q_full[j % kSlots]), (j / kSlots) & 1, &g_status);
  } else if (warp == 10) {
    // ------------------------------------------------- lse of each step's rows
    // (negated; a row outside the sequence, or one that saw nothing: -inf, weight 0)
    // The values of a step are loaded a step ahead.
    constexpr int kOwn = kBlock / 32;
    int row_t[kOwn], row_h[kOwn];
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      const int c = lane + 32 * k;
      row_t[k] = c < step_tokens * a.group ? c / a.group : 1 << 28;
      row_h[k] = c % a.group;
    }
    int g = 0;
    for (int n = 0; next_share(n); ++n) {
      float v[kOwn];
      auto load = [&](int j) {
        const int t0 = (w.from + j) * step_tokens;
#pragma unroll
        for (int k = 0; k < kOwn; ++k)
          v[k] = t0 + row_t[k] < w.tokens
                     ? a.lse[static_cast<long long>(w.first + t0 + row_t[k]) * a.n_q +
                             w.h * a.group + row_h[k]]
                     : -INFINITY;
      };
      if (w.steps > 0) load(0);
      for (int j = 0; j < w.steps; ++j, ++g) {
        const int d = g & 1;
        if (g > 1) step_wait(smem_u32(&bars.l_empty[d]), (g / 2 - 1) & 1, &s_failed, &g_status);
#pragma unroll
        for (int k = 0; k < kOwn; ++k)
          s_lse[d][lane + 32 * k] = v[k] != -INFINITY ? v[k] * -kLog2e : -INFINITY;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.l_full[d]));
        if (j + 1 < w.steps) load(j + 1);
      }
    }
  } else if (warp == 8) {
    // ---------------------------------------------------------- products
    const uint32_t tm = static_cast<uint32_t>(tc::uniform(static_cast<int>(tmem)));
    int kb = 0, g = 0, g1 = 0;  // buffers of keys, steps, steps of two tiles so far
    for (int n = 0; next_share(n); ++n) {
      const int n_steps = tc::uniform(w.steps), n_tiles = tc::uniform(w.tiles);
      if (n_steps == 0) continue;
      const int kd = kb & 1;
      step_wait(smem_u32(&bars.keys[kd]), (kb / 2) & 1, &s_failed, &g_status);
      ++kb;
      for (int j = 0; j < n_steps; ++j, ++g) {
        const int slot = g % kSlots;
        step_wait(smem_u32(&bars.q_full[slot]), (g / kSlots) & 1, &s_failed, &g_status);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (x >= n_tiles) break;
          const int gx = x == 0 ? g : g1, d = gx & 1;
          if (gx > 1)
            step_wait(smem_u32(&bars.s_empty[x][d]), (gx / 2 - 1) & 1, &s_failed, &g_status);
          tc::fence_after();
          if (tc::elect_one()) {
            const uint64_t k = tc::desc_k_major(smem_u32(base + (2 * kd + x) * Sh::kBytes));
            const uint64_t q = tc::desc_k_major(smem_u32(qring + slot * Sh::kBytes));
#pragma unroll
            for (int i = 0; i < HD / 16; ++i) {
              const int step = (i / 4) * (kBlock * 128) + (i % 4) * 32;
              tc::mma_ss(tm + (2 * x + d) * kBlock, k + (step >> 4), q + (step >> 4), Sh::kDesc,
                         i > 0);
            }
            tc::commit(smem_u32(&bars.s_full[x][d]));
          }
          __syncwarp();
        }
        if (tc::elect_one()) {
          tc::commit(smem_u32(&bars.q_empty[slot]));
          if (j == n_steps - 1) tc::commit(smem_u32(&bars.k_empty[kd]));
        }
        __syncwarp();
        g1 += n_tiles - 1;
      }
    }
    if (tc::elect_one()) tc::commit(smem_u32(&bars.drain));
    __syncwarp();
    warp_wait(smem_u32(&bars.drain), 0, &g_status);
  } else if (warp == 11) {
    // ------------------------------------------------------------ shares
    const long long pairs = run_total(a.c.n_seqs, a.c.n_kv, lane,
                                      [&](int i) { return shares_of(checked_len(a, i)); });
    // The pairs behind the last full round go out tile by tile where every block
    // then still gets one at most (520 pairs on 152 blocks: 68 us against 72).
    const long long rest = pairs % gridDim.x, whole = pairs - (2 * rest <= gridDim.x ? rest : 0);
    const long long shares = whole + 2 * (pairs - whole);
    int n = 0;
    for (long long b = blockIdx.x;; b += gridDim.x, ++n) {
      const int i = n % kAhead;
      if (b < shares)
        get_share(a, b, whole, step_tokens, lane, &w);
      else
        w.s = -1;
      if (n >= kAhead)
        step_wait(smem_u32(&bars.share_empty[i]), (n / kAhead - 1) & 1, &s_failed, &g_status);
      if (lane == 0) {
        s_share[i] = w;
        mbar_arrive(smem_u32(&bars.share_full[i]));
      }
      __syncwarp();
      if (b >= shares || __any_sync(0xFFFFFFFFu, *static_cast<volatile int*>(&s_failed) != 0)) break;
    }
  } else {
    // -------------------------------------------------------------- sums
    const int x = warp >> 2;
    const uint32_t lanes = tmem + ((warp & 3) << 21) + 2 * x * kBlock;
    int g = 0, gx = 0;  // steps so far, of this group's tiles
    for (int n = 0; next_share(n); ++n) {
      if (x >= w.tiles) {  // (the other group's steps: their lse passes by)
        for (int j = 0; j < w.steps; ++j, ++g) {
          step_wait(smem_u32(&bars.l_full[g & 1]), (g / 2) & 1, &s_failed, &g_status);
          if (lane == 0) mbar_arrive(smem_u32(&bars.l_empty[g & 1]));
        }
        continue;
      }
      const int e = w.e0 + x * kBlock + (warp & 3) * 32 + lane;
      const bool live = e < w.len;
      const int page = live ? raw_page(a.c, w.s, e) : 0;
      const long long at = (static_cast<long long>(w.s) * a.c.n_kv + w.h) *
                               (static_cast<long long>(a.c.max_pages) << a.c.page_shift) + e;
      const float before = live && a.mass != nullptr ? a.mass[at] : 0.f;
      uint64_t sum[2] = {0, 0};
      const uint64_t scale = pair(a.scale_log2, a.scale_log2);
      for (int j = 0; j < w.steps; ++j, ++g, ++gx) {
        const int d = gx & 1;
        step_wait(smem_u32(&bars.l_full[g & 1]), (g / 2) & 1, &s_failed, &g_status);
        step_wait(smem_u32(&bars.s_full[x][d]), (gx / 2) & 1, &s_failed, &g_status);
        tc::fence_after();
        // columns before `seen` are rows that lie before this entry, those from
        // `end` on belong to no token of the sequence (and may hold anything)
        const int t0 = (w.from + j) * step_tokens;
        const int seen = max(0, e - w.off - t0) * a.group;
        const int end = min(step_tokens, w.tokens - t0) * a.group;
        const bool all = __all_sync(0xFFFFFFFFu, seen == 0) && end == kBlock;
        uint32_t v[2][32];
        tc::ld32(v[0], lanes + d * kBlock);
        tc::wait_ld32(v[0]);
        const float* ls = s_lse[g & 1];
        if (all) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // the next 32 columns load while these are summed
            if (c < 3) tc::ld32(v[(c + 1) & 1], lanes + d * kBlock + 32 * (c + 1));
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(ls + 32 * c + k);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint64_t s = pair(__uint_as_float(v[c & 1][k + 2 * i]),
                                        __uint_as_float(v[c & 1][k + 2 * i + 1]));
                const float2 x = unpair(fma2(s, scale, i == 0 ? l.x : l.y));
                sum[i] = add2(sum[i], pair(ex2(x.x), ex2(x.y)));
              }
            }
            if (c < 3) tc::wait_ld32(v[(c + 1) & 1]);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c < 3) tc::ld32(v[(c + 1) & 1], lanes + d * kBlock + 32 * (c + 1));
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              float y[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int col = 32 * c + k + i;
                y[i] = ex2(fmaf(__uint_as_float(v[c & 1][k + i]), a.scale_log2, ls[col]));
                if (col < seen || col >= end) y[i] = 0.f;
              }
              sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], pair(y[0], y[1]));
            }
            if (c < 3) tc::wait_ld32(v[(c + 1) & 1]);
          }
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&bars.s_empty[x][d]));
          mbar_arrive(smem_u32(&bars.l_empty[g & 1]));
        }
      }
      const float2 both = unpair(add2(sum[0], sum[1]));
      if (live && *static_cast<volatile int*>(&s_failed) == 0) {
        float total = good_page(a.c, page, nullptr) >= 0 ? both.x + both.y : 0.f;
        if (!(total == total)) total = slow_sum<HD>(a, w.h, w.first, w.tokens, w.off, e, page);
        a.mass_out[at] = before + total;
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 8) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

template <typename F, typename... Args>
cudaError_t launch(F* k, std::atomic<unsigned long long>* done, long long blocks, int threads,
                   int smem, cudaStream_t st, int device, Args... args) {
  const unsigned long long bit = 1ull << (device & 63);
  if (!(done->load(std::memory_order_relaxed) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    done->fetch_or(bit, std::memory_order_relaxed);
  }
  if (blocks < 1 || blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

template <int HD, int NT>
cudaError_t launch_few(const MassArgs& a, int sms, cudaStream_t st, int device) {
  static std::atomic<unsigned long long> done{0};
  return launch(mass_few_kernel<HD, NT>, &done, static_cast<long long>(sms) * few_resident(NT),
                32 * kWarps, kWarps * kStages * key_bytes<HD>(), st, device, a);
}

template <int HD>
cudaError_t launch_many(const MassArgs& a, int sms, cudaStream_t st, int device) {
  static std::atomic<unsigned long long> done{0};
  const EncodeTiledFn fn = encode_fn();
  CUtensorMap km, qm;
  const int step_tokens = kBlock / a.group;
  const cuuint64_t dim[3] = {static_cast<cuuint64_t>(HD), static_cast<cuuint64_t>(a.n_q),
                             static_cast<cuuint64_t>(a.n_tokens)};
  const cuuint64_t stride[2] = {static_cast<cuuint64_t>(HD) * 2,
                                static_cast<cuuint64_t>(a.q_stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(a.group),
                             static_cast<cuuint32_t>(step_tokens)};
  const cuuint32_t estride[3] = {1, 1, 1};
  if (fn == nullptr || !encode_pool(&km, a.c, a.c.k) ||
      fn(&qm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half*>(a.q), dim, stride, box,
         estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  return launch(mass_many_kernel<HD>, &done, sms, kManyThreads, Shape<HD>::kSmem, st, device, a, km,
                qm, step_tokens);
}

template <int HD>
cudaError_t launch_t(const MassArgs& a, int sms, cudaStream_t st, int device) {
  const long long rows = static_cast<long long>(a.max_q) * a.group;
  // (a group of more than 128 heads has no box of whole tokens)
  if (rows > kRowsMax && a.group <= kBlock && a.n_tokens > 0) return launch_many<HD>(a, sms, st, device);
  if (rows <= 8) return launch_few<HD, 1>(a, sms, st, device);
  if (rows <= 16) return launch_few<HD, 2>(a, sms, st, device);
  return launch_few<HD, 4>(a, sms, st, device);
}

}  // namespace

cudaError_t attention_mass_launch(const MassArgs& a, int sms, cudaStream_t st, int device) {
  return a.c.head_dim == 64 ? launch_t<64>(a, sms, st, device) : launch_t<128>(a, sms, st, device);
}

cudaError_t status_mass(unsigned* out) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_status, sizeof(v));
  if (e != cudaSuccess) return e;
  e = cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
  *out |= v;
  return e;
}

}  // namespace qgemv
