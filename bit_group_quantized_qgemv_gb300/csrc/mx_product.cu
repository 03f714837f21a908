// mx_product.cu -- products with MXFP4 weights (qgemv_mxfp4, qgemv_mx_gemm,
// qgemv_mx_swiglu) on the block-scaled tensor-core instruction.
//
//   D[n][c] = sum over blocks b of 2^(sw[n][b] + sx[c][b]) sum_{k in b} w[n][k] x[c][k]
//
// A tile is 128 weight rows (the instruction's A operand, 4-bit codes as they are
// stored, spread to bytes by the copy itself) by up to 240 columns (B, e4m3): nothing
// is dequantised by arithmetic, the scales go to tensor memory and into the product.
// Columns are the MXFP8 rows of x, or for fp16 rows three columns each (B then e5m2, which has
// fp16's range): x 2^k = q1 + q2 / 2^4 + q3 / 2^8 with a k for each block.  q1 takes three
// significant bits, q2 and q3 four of what is left and its sign: the eleven of an fp16 value, down
// to fp16's last place.  All of x is held exactly but the last bit of values below 2^-13 in
// blocks whose largest is 32768 or more.  The three sums are added in fp32.  (Three columns of
// e4m3, whose range is shorter, lost entries below 2^-27 of the block's largest.)
//
// A step is 128 k: a ring of stages (codes of A and, for MXFP8 rows, of B, 128-byte
// swizzled, and their scales) between
//   two warps   codes of A and of MXFP8 rows, every other step each (one wait and issue
//               takes some 250 clocks, however large the box), by TMA or, where K or an
//               address does not allow that for A, by cp.async;
//   four warps  scales, four steps each: a row's bytes of them in one load where they are
//               aligned;
//   two warps   scales to tensor memory and four products a step: one for each weight,
//               or every other step into an accumulator of its own (a warp takes 550
//               clocks a step to wait for it and issue its products, few columns only 160
//               of the tensor core); with over 112 columns one does all;
//   eight       results, a weight row per lane; two accumulators, so that the next tile's
//               products run meanwhile.  Before the first result they turn the block's
//               share of fp16 rows into columns, which stay in shared memory for the call.
// Thread blocks stay for the whole call and take tiles one after the other.  Where
// there are few tiles, the blocks of a cluster share K: each finishes every split-th
// column, adding the others' sums, sent to its shared memory, in rank order.
#include "mx_product.cuh"

namespace qgemv {
namespace {

__device__ unsigned g_status = 0;

constexpr int kRowsW = kMxRows, kStepK = kMxStep;
constexpr int kLoaders = 4;   // warps
constexpr int kTmaWarps = 2;
constexpr int kScaleCols = 16;  // tensor memory of one step's scales

// How a launch loads its operands.
struct MxLoads {
  bool tma_w;  // weights by TMA
  int bytes;   // of a row's scales in one load: 16, 4 or 1
  bool wide;   // four values of y and the residual in one access
};

struct Bars {
  uint64_t full[kMxMaxStages], empty[kMxMaxStages];
  uint64_t rows[kMxRowSteps];  // columns of fp16 rows
  uint64_t turn[kLoaders];      // a loader may go on to its group
  uint64_t acc_full[2], acc_empty[2];
  uint64_t part_full, part_done;  // other ranks have a part in these
};

// An arrival on the mbarrier once this thread's copies so far are done; the barrier's
// count has it already.
__device__ __forceinline__ void arrive_copied(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Eight bytes, or zeros.
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, bool take) {
  const int n = take ? 8 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

// An array of bytes that starts and ends anywhere, read by aligned words: those that it only
// shares are put together from its bytes once (Ends), and loads of the others stay inside, so
// that they can all be under way together.
struct Ends {
  uint32_t head, tail;  // the words that hold its first and its last bytes, where those are not whole
};

__device__ __forceinline__ uint32_t shared_word(const uint8_t* p, const uint8_t* from, const uint8_t* to) {
  uint32_t w = 0;
  for (int i = 0; i < 4; ++i)
    if (p + i >= from && p + i < to) w |= static_cast<uint32_t>(p[i]) << (8 * i);
  return w;
}
__device__ __forceinline__ const uint8_t* first_whole(const uint8_t* from) {
  return from + (-reinterpret_cast<uintptr_t>(from) & 3);
}
__device__ __forceinline__ const uint8_t* behind_whole(const uint8_t* to) {
  return to - (reinterpret_cast<uintptr_t>(to) & 3);
}
__device__ __forceinline__ Ends ends_of(const uint8_t* from, const uint8_t* to) {
  return Ends{shared_word(first_whole(from) - 4, from, to), shared_word(behind_whole(to), from, to)};
}

// Sixteen bytes from five aligned words, the first of which starts `off` before them; those
// from the n-th on are 0.
__device__ __forceinline__ uint4 shifted(const uint32_t* raw, int off, int n) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = __funnelshift_r(raw[i], raw[i + 1], 8 * off);
    const int left = n - 4 * i;  // bytes of this word
    if (left < 4) w[i] &= left <= 0 ? 0u : (1u << (8 * left)) - 1;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Sixteen bytes at s: anywhere, with three bytes of the array before them and 20 behind.
__device__ __forceinline__ uint4 sixteen_within(const uint8_t* s, int n) {
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(s) & 3);
  const uint32_t* p = reinterpret_cast<const uint32_t*>(s - off);
  uint32_t raw[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) raw[i] = p[i];
  return shifted(raw, off, n);
}

// Sixteen bytes at s, a place in the array; those from the n-th on are 0.
__device__ __forceinline__ uint4 sixteen(const uint8_t* s, int n, const uint8_t* from, const uint8_t* to, Ends ends) {
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(s) & 3);
  const uint8_t *first = first_whole(from), *last = behind_whole(to) - 4;  // whole words, if first <= last
  uint32_t raw[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const uint8_t *p = s - off + 4 * i, *at = p < first ? first : p > last ? last : p;
    raw[i] = first <= last ? *reinterpret_cast<const uint32_t*>(at) : 0;
    raw[i] = p < first ? ends.head : p > last ? (p == last + 4 ? ends.tail : 0) : raw[i];
  }
  return shifted(raw, off, n);
}

// Place of row r's word among the scales of a step.
__device__ __forceinline__ int scale_at(int r) { return (r >> 7) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4; }

// Warps by what they do.
constexpr int kOutWarps = 8, kLoadWarp = kOutWarps, kMmaWarp = kLoadWarp + kLoaders,
              kTmaWarp = kMmaWarp + 2, kThreads = 32 * (kTmaWarp + kTmaWarps);

// 2^k, -14 <= k <= 15, in both halves.
__device__ __forceinline__ __half2 power2(int k) {
  const uint32_t h = static_cast<uint32_t>(k + 15) << 10, w = h | (h << 16);
  return *reinterpret_cast<const __half2*>(&w);
}

// Eight values of row m of x (a lane; four lanes hold a block) to three columns: their codes at
// `cols` (a step's, swizzled), the blocks' scales at `scales`.  All in fp16: x 2^k has its block's
// largest in [2^14, 2^15), so what a column leaves is at most 2^11 and 2^7, and its last bits are
// multiples of 2^-24, the last place of q3 (k = -1 halves, and rounds, fp16's last place; k = 30, for
// blocks below 2^-16, makes all of them whole numbers).  What a column leaves is a multiple of
// x's last bit and no larger than x was, so the subtractions are exact.
__device__ __forceinline__ void split_values(uint4 v, bool live, uint32_t cols, uint32_t scales, int m,
                                             int ch) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  uint32_t most = __vmaxu2(__vmaxu2(u[0] & 0x7FFF7FFFu, u[1] & 0x7FFF7FFFu),
                           __vmaxu2(u[2] & 0x7FFF7FFFu, u[3] & 0x7FFF7FFFu));
  most = __vmaxu2(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
  most = __vmaxu2(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
  const uint32_t top = max(most & 0xFFFFu, most >> 16);  // bits of the largest magnitude
  const int e = static_cast<int>(__float_as_uint(__half2float(__ushort_as_half(static_cast<uint16_t>(top)))) >> 23);
  const int k = min(max(14 + 127 - e, -1), 30);
  const __half2 k0 = power2(min(k, 15)), k1 = power2(max(k - 15, 0));
  __half2 f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __hmul2(__hmul2(*reinterpret_cast<const __half2*>(&u[i]), k0), k1);
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint16_t two;
      uint32_t got;
      asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(two) : "r"(*reinterpret_cast<const uint32_t*>(&f[i])));
      asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(got) : "h"(two));
      f[i] = __hmul2(__hsub2(f[i], *reinterpret_cast<const __half2*>(&got)), power2(4));
      w[i >> 1] = i & 1 ? w[i >> 1] | (static_cast<uint32_t>(two) << 16) : two;
    }
    const int c = 3 * m + q;
    const int sb = top >= 0x7C00u ? 255 : 127 - k - 4 * q;
    if (live) {
      asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(cols + c * 128 + (((ch >> 1) ^ (c & 7)) << 4) +
                                                           (ch & 1) * 8),
                   "r"(w[0]), "r"(w[1])
                   : "memory");
      if ((ch & 3) == 0)
        asm volatile("st.shared.u8 [%0], %1;" ::"r"(scales + scale_at(c) + (ch >> 2)), "r"(sb) : "memory");
    }
  }
}

// GATED: two weights.  SPLIT: fp16 rows.
template <bool GATED, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    mx_product_kernel(const MxProductArgs a, const MxPlan p, const MxLoads ld, const __grid_constant__ CUtensorMap w_map,
                      const __grid_constant__ CUtensorMap u_map, const __grid_constant__ CUtensorMap x_map) {
  constexpr int kW = GATED ? 2 : 1;
  extern __shared__ uint8_t raw_smem[];
  __shared__ Bars bars;
  __shared__ uint32_t s_tmem;
  __shared__ int s_failed;
  // (uniform: what the products' operands and loops depend on, see tc::elect_one)
  const int warp = tc::uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int rank = p.split > 1 ? tc::uniform(static_cast<int>(cluster_rank())) : 0;
  const uint32_t base = (smem_u32(raw_smem) + 1023) & ~1023u;
  const int b_bytes = p.cols * kStepK;
  const int c_bytes = kW * 16384 + (SPLIT ? 0 : b_bytes);        // a stage: A (, up) (, B)
  const int s_bytes = 512 * (kW + (SPLIT ? 0 : p.cols > 128 ? 2 : 1));  // and their scales
  const uint32_t x_cols = base + p.stages * c_bytes;              // columns of fp16 rows
  const uint32_t s_ring = x_cols + (SPLIT ? p.row_steps * b_bytes : 0);
  const uint32_t x_scales = s_ring + p.stages * s_bytes;
  const uint32_t part = x_scales + (SPLIT ? p.row_steps * 512 : 0);

  const int steps = (a.K + kStepK - 1) / kStepK;
  const int k0 = static_cast<int>(static_cast<long long>(steps) * rank / p.split);
  const int k1 = static_cast<int>(static_cast<long long>(steps) * (rank + 1) / p.split);
  const long long tiles = static_cast<long long>(p.row_tiles) * p.tok_tiles;
  const long long first = blockIdx.x / p.split, stride = gridDim.x / p.split;
  auto place = [&](long long tile, int* row, int* tok) {
    const int fast = p.rows_first ? p.row_tiles : p.tok_tiles;
    const int i = static_cast<int>(tile % fast), o = static_cast<int>(tile / fast);
    *row = (p.rows_first ? i : o) * kRowsW;
    *tok = (p.rows_first ? o : i) * p.tokens;
  };

  // The first tile's weights on their way to L2 while the kernel before ends.
  if (first < tiles) {
    int row, tok;
    place(first, &row, &tok);
    if (warp == kTmaWarp && lane == 0) {
      if (ld.tma_w) {
        for (int k = k0; k < k1 && k < k0 + p.stages; ++k) {
          tc::prefetch_2d(&w_map, k * kStepK, row);
          if (GATED) tc::prefetch_2d(&u_map, k * kStepK, row);
        }
      }
    } else if (warp >= kLoadWarp && warp < kMmaWarp) {
      const int n = row + threadIdx.x - kLoadWarp * 32, blocks = a.K / kMxBlock;
      const long long at = static_cast<long long>(n) * blocks + 4 * k0;
      if (n < a.N) {
        prefetch_l2(a.ws + at);
        if (GATED) prefetch_l2(a.us + at);
      }
    }
  }
  if (warp == 0) {
    if (lane < p.stages) {
      mbar_init(smem_u32(&bars.full[lane]), 1 + (ld.tma_w ? 0 : 32) + (ld.tma_w || !SPLIT ? 1 : 0));
      mbar_init(smem_u32(&bars.empty[lane]), kW);
    }
    if (lane < kLoaders) mbar_init(smem_u32(&bars.turn[lane]), 1);
    if (lane < 2) {
      mbar_init(smem_u32(&bars.acc_full[lane]), GATED || p.pair ? 2 : 1);
      mbar_init(smem_u32(&bars.acc_empty[lane]), kOutWarps);
    }
    if (lane == 0) {
      mbar_init(smem_u32(&bars.part_full), 1);
      mbar_init(smem_u32(&bars.part_done), kOutWarps * p.split);
      s_failed = 0;
    }
    if constexpr (SPLIT)
      for (int i = lane; i < k1 - k0; i += 32) mbar_init(smem_u32(&bars.rows[i]), 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (p.split > 1) cluster_arrive();
  pdl_wait();
  if (warp == kMmaWarp) tc::alloc(smem_u32(&s_tmem), 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  pdl_launch_dependents();
  if (p.split > 1) cluster_wait();  // barriers are there before a rank arrives on another's
  const uint32_t tmem = s_tmem;

  // The steps of a warp that takes every n-th of all tiles' steps, from the me-th on, and
  // their stages.
  struct Steps {
    long long t;
    int k, stage, use;
    bool moved;  // to another tile
  };
  auto start = [&](int me) { return Steps{first, k0 + me, me, 0, true}; };
  auto find = [&](Steps& s) {  // false: there are no more
    while (s.k >= k1 && s.t < tiles) s.k -= k1 - k0, s.t += stride, s.moved = true;
    while (s.stage >= p.stages) s.stage -= p.stages, ++s.use;
    return s.t < tiles;
  };
  if (warp >= kTmaWarp) {
    // ---------------------------------------------------------------- codes
    const uint32_t bytes = (ld.tma_w ? kW * 8192 : 0) + (SPLIT ? 0 : b_bytes);
    Steps s = start(warp - kTmaWarp);
    int row = 0, tok = 0;
    for (; find(s); s.k += kTmaWarps, s.stage += kTmaWarps) {
      if (s.moved) place(s.t, &row, &tok);
      s.moved = false;
      if (s.use > 0) step_wait(smem_u32(&bars.empty[s.stage]), (s.use - 1) & 1, &s_failed, &g_status);
      const uint32_t full = smem_u32(&bars.full[s.stage]), to = base + s.stage * c_bytes;
      if (lane == 0 && bytes > 0) {
        mbar_arrive_expect_tx(full, bytes);
        if (ld.tma_w) {
          tc::tma_2d(to, &w_map, s.k * kStepK, row, full);
          if (GATED) tc::tma_2d(to + 16384, &u_map, s.k * kStepK, row, full);
        }
        if (!SPLIT) tc::tma_2d(to + kW * 16384, &x_map, s.k * kStepK, tok, full);
      }
      __syncwarp();
      if (!ld.tma_w) {
        // sixteen codes a copy, eight lanes to a row
        const int r0 = lane >> 3, c = lane & 7, left = a.N - row;
        const bool inside = s.k * kStepK + c * 16 < a.K;
        const long long at = static_cast<long long>(row + r0) * (a.K / 8) + s.k * (kStepK / 8) + c * 2;
#pragma unroll
        for (int w = 0; w < kW; ++w) {
          const uint32_t* codes = w ? a.up : a.w;
#pragma unroll 8
          for (int i = 0; i < kRowsW / 4; ++i) {
            const int r = r0 + 4 * i;
            const bool has = inside && r < left;
            cp_async8(to + w * 16384 + r * 128 + ((c ^ (r & 7)) << 4),
                      codes + (has ? at + static_cast<long long>(i) * (a.K / 2) : 0), has);
          }
        }
        arrive_copied(full);
      }
    }
    cp_wait_all();
  } else if (warp >= kMmaWarp) {
    // ------------------------------------------------------------- products
    const int me = warp - kMmaWarp;
    const bool two = GATED || p.pair;
    const uint32_t tm = static_cast<uint32_t>(tc::uniform(static_cast<int>(tmem)));
    const uint32_t idesc = tc::idesc_mx(p.cols, 128, SPLIT);
    int stage = 0, use = 0, n = 0, odd = 0;  // odd: of all tiles' steps, the next one's number
    uint32_t c = base, ss = s_ring;          // of the stage
    for (long long t = first; t < tiles && (two || me == 0); t += stride, ++n) {
      const int buf = n & 1;
      if (n >= 2) step_wait(smem_u32(&bars.acc_empty[buf]), ((n >> 1) - 1) & 1, &s_failed, &g_status);
      tc::fence_after();
      const uint32_t acc = tm + (buf * (two ? 2 : 1) + me) * p.cols;
      for (int k = k0; k < k1; ++k) {
        if (GATED || !p.pair || odd == me) {
          // (with an odd number of steps a warp has the others of them in the second tile)
          if (SPLIT && n < 2) step_wait(smem_u32(&bars.rows[k - k0]), 0, &s_failed, &g_status);
          step_wait(smem_u32(&bars.full[stage]), use & 1, &s_failed, &g_status);
          if (!ld.tma_w) tc::fence_async_shared();  // codes by cp.async, for the tensor core
          tc::fence_after();
          if (tc::elect_one()) {
            const uint32_t st = tm + kMxAccCols + (two ? me : k & 1) * kScaleCols;
            tc::copy_scales(st, ss + (GATED ? me * 512 : 0));
            tc::copy_scales(st + 8, SPLIT ? x_scales + (k - k0) * 512 : ss + kW * 512);
            if (p.cols > 128) tc::copy_scales(st + 12, ss + (kW + 1) * 512);
            const uint64_t b = tc::desc_k_major(SPLIT ? x_cols + (k - k0) * b_bytes : c + kW * 16384);
            const uint64_t w = tc::desc_k_major(c + (GATED ? me * 16384 : 0));
            const int more = k > k0 + (!GATED && p.pair ? 1 : 0);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              tc::mma_mx(acc, w + 2 * j, b + 2 * j, idesc, j, st, st + 8, j > 0 || more);
            tc::commit(smem_u32(&bars.empty[stage]));
          }
          __syncwarp();
        }
        odd ^= 1;
        c += c_bytes, ss += s_bytes;
        if (++stage == p.stages) stage = 0, ++use, c = base, ss = s_ring;
      }
      if (tc::elect_one()) tc::commit(smem_u32(&bars.acc_full[buf]));
      __syncwarp();
    }
  } else if (warp >= kLoadWarp) {
    // ---------------------------------------------------------------- loads
    constexpr int kRowsX = SPLIT ? 0 : GATED ? 4 : 8;  // rows of x a lane has scales of
    const int me = warp - kLoadWarp, blocks = a.K / kMxBlock, my_steps = k1 - k0;
    const int q0 = k0 >> 2, groups = ((k1 - 1) >> 2) - q0 + 1;  // of four steps, of a tile
    const long long all = first < tiles ? ((tiles - 1 - first) / stride + 1) * groups : 0;
    Ends w_ends = {}, u_ends = {}, x_ends = {};
    if (ld.bytes == 1) {
      w_ends = ends_of(a.ws, a.ws + static_cast<long long>(a.N) * blocks);
      if (GATED) u_ends = ends_of(a.us, a.us + static_cast<long long>(a.N) * blocks);
      if (!SPLIT) x_ends = ends_of(a.xs, a.xs + static_cast<long long>(a.M) * blocks);
    }
    for (long long g = me; g < all; g += kLoaders) {
      const long long turn = g / groups;
      const int q = q0 + static_cast<int>(g % groups), from = max(k0, 4 * q), to = min(k1, 4 * q + 4);
      int row, tok;
      place(first + turn * stride, &row, &tok);
      // Scales of rows lane, lane + 32, ... of each operand: of the group's four steps.  (All
      // loads of a kind in one go, so that they are under way together.)
      uint4 vw[4], vu[GATED ? 4 : 1], vx[kRowsX ? kRowsX : 1];
      auto load_all = [&](auto load) {  // load(operand, row of the tile, 0: no row of it is there)
#pragma unroll
        for (int i = 0; i < 4; ++i) vw[i] = load(0, row + lane + 32 * i, a.N);
        if constexpr (GATED) {
#pragma unroll
          for (int i = 0; i < 4; ++i) vu[i] = load(1, row + lane + 32 * i, a.N);
        }
#pragma unroll
        for (int i = 0; i < kRowsX; ++i)  // (rows of the next tile are loaded too, and not used)
          vx[i] = load(2, tok + lane + 32 * i, 32 * i < p.tokens ? a.M : 0);
      };
      auto base_of = [&](int operand) { return operand == 0 ? a.ws : operand == 1 ? a.us : a.xs; };
      auto at = [&](int operand, int r) { return base_of(operand) + static_cast<long long>(r) * blocks + 16 * q; };
      if (ld.bytes == 16) {
        load_all([&](int operand, int r, int end) {
          return r < end ? *reinterpret_cast<const uint4*>(at(operand, r)) : make_uint4(0, 0, 0, 0);
        });
      } else if (ld.bytes == 4) {
        load_all([&](int operand, int r, int end) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w[j] = r < end && 4 * q + j >= from && 4 * q + j < to
                       ? *reinterpret_cast<const uint32_t*>(at(operand, r) + 4 * j)
                       : 0;
          return make_uint4(w[0], w[1], w[2], w[3]);
        });
      } else {
        // Tiles away from the ends of an operand's scales need no look at them.
        const int x_rows = p.tokens > 128 ? 256 : 128, n = min(16, blocks - 16 * q);
        auto inside = [&](int r, int rows, int end) {
          return r > 0 && static_cast<long long>(r) * blocks >= 3 && r + rows < end &&
                 static_cast<long long>(end - r - rows) * blocks >= 20;
        };
        if (inside(row, kRowsW, a.N) && (SPLIT || inside(tok, x_rows, a.M))) {
          load_all([&](int operand, int r, int end) { return sixteen_within(at(operand, end > 0 ? r : tok), n); });
        } else {
          load_all([&](int operand, int r, int end) {
            if (r >= end) return make_uint4(0, 0, 0, 0);
            const uint8_t* start = base_of(operand);
            return sixteen(at(operand, r), n, start,
                           start + static_cast<long long>(operand == 2 ? a.M : a.N) * blocks,
                           operand == 0 ? w_ends : operand == 1 ? u_ends : x_ends);
          });
        }
      }
      // One group after the other: a wait for a stage tells a use from the one before it,
      // not from two before.
      if (g > 0)
        step_wait(smem_u32(&bars.turn[me]), ((g / kLoaders) - (me == 0 ? 1 : 0)) & 1, &s_failed, &g_status);
      const long long done = turn * my_steps + (from - k0);  // steps before the group's
      int stage = static_cast<int>(done % p.stages);
      long long use = done / p.stages;
      int written = 0;  // steps whose scales are to be handed on
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = 4 * q + j;
        if (k < from || k >= to) continue;
        if (use > 0) step_wait(smem_u32(&bars.empty[stage]), (use - 1) & 1, &s_failed, &g_status);
        if (k == to - 1 && lane == 0) mbar_arrive(smem_u32(&bars.turn[(me + 1) % kLoaders]));
        const uint32_t ss = s_ring + stage * s_bytes + lane * 16;
        auto word = [&](const uint4& v) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; };
        store_shared(ss, word(vw[0]), word(vw[1]), word(vw[2]), word(vw[3]));
        if constexpr (GATED) store_shared(ss + 512, word(vu[0]), word(vu[1]), word(vu[2]), word(vu[3]));
        if constexpr (kRowsX > 0) {
          store_shared(ss + kW * 512, word(vx[0]), word(vx[1]), word(vx[2]), word(vx[3]));
          if constexpr (kRowsX > 4)
            if (p.cols > 128)
              store_shared(ss + (kW + 1) * 512, word(vx[4]), word(vx[5]), word(vx[6]), word(vx[7]));
        }
        if (++stage == p.stages) stage = 0, ++use;
        ++written;
        // Handed on two or four at a time: the fence takes longer than all else.
        if (k == to - 1 || j == 3 || (j == 1 && p.stages < 8)) {
          tc::fence_async_shared();
          __syncwarp();
          const int s = stage - 1 - lane;
          if (lane < written) mbar_arrive(smem_u32(&bars.full[s < 0 ? s + p.stages : s]));
          written = 0;
        }
      }
      __syncwarp();
    }
  } else {
    // -------------------------------------------------------------- results
    const int quarter = warp & 3, half = warp >> 2;  // lanes of tensor memory; which columns
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter) << 21);
    if constexpr (SPLIT) {
      // the block's share of the fp16 rows, a step a warp, two rows of x at a time
      for (int i = warp; i < k1 - k0 && first < tiles; i += kOutWarps) {
        const int ch = lane & 15, at = (k0 + i) * kStepK + ch * 8;
        uint4 v[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int m = 2 * h + (lane >> 4);
          v[h] = m < p.tokens && at < a.K
                     ? *reinterpret_cast<const uint4*>(a.x16 + static_cast<long long>(m) * a.K + at)
                     : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          if (2 * h >= p.tokens) break;
          const int m = 2 * h + (lane >> 4);
          split_values(v[h], m < p.tokens, x_cols + i * b_bytes, x_scales + i * 512, m, ch);
        }
        tc::fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.rows[i]));
      }
    }
    // Where results lie before they are written in rows of x (after a wait that ran out the
    // warps still meet at the barriers around this, and write nothing).
    const uint32_t stage_out = part + half * (kMxOut * kRowsW * 4);
    const int share = (p.tokens + p.split - 1) / p.split;  // rows of x that a rank finishes, at most
    // Where rank q's sums for this rank's j-th row lie.
    auto part_at = [&](int q, int j, int w) {
      return part + (((q * share + j) * kW + w) * kRowsW + quarter * 32 + lane) * 4;
    };
    int n_t = 0;
    for (long long t = first; t < tiles; t += stride, ++n_t) {
      int row, tok;
      place(t, &row, &tok);
      const int buf = n_t & 1, n = row + quarter * 32 + lane, count = min(p.tokens, a.M - tok);
      const bool res = !GATED && a.res != nullptr && n < a.N;
      auto residual = [&](int m) { return __half2float(a.res[static_cast<long long>(tok + m) * a.N + n]); };
      const int own = (count - rank + p.split - 1) / p.split;  // rows that this rank finishes
      step_wait(smem_u32(&bars.acc_full[buf]), (n_t >> 1) & 1, &s_failed, &g_status);
      tc::fence_after();
      const uint32_t acc = lanes + buf * (GATED || p.pair ? 2 : 1) * p.cols;
      // a tile of a single step has one of two accumulators: the step's
      const bool one = !GATED && p.pair && k1 - k0 == 1;
      const bool has0 = !one || (n_t & 1) == 0, has1 = !one || (n_t & 1) == 1;
      if (p.split > 1) {
        if (n_t > 0) step_wait<true>(smem_u32(&bars.part_done), (n_t - 1) & 1, &s_failed, &g_status);
        // (behind that wait: a rank that finishes no row, of few, ends its phase by this alone, and its
        // other warps must have seen the one before)
        if (warp == 0 && lane == 0)
          mbar_arrive_expect_tx(smem_u32(&bars.part_full), max(own, 0) * p.split * kW * kRowsW * 4);
      }
      auto give = [&](int m, float g, float u) {  // a rank's sums of one column to who finishes it
        const int q = m % p.split;
        const uint32_t to = map_rank(part_at(rank, m / p.split, 0), q), bar = map_rank(smem_u32(&bars.part_full), q);
        send(to, g, bar);
        if (GATED) send(to + kRowsW * 4, u, bar);
      };
      const bool ok = __all_sync(0xFFFFFFFFu, *static_cast<volatile int*>(&s_failed) == 0);
      if constexpr (SPLIT) {
        // four rows of x a warp: 12 columns
        const int m0 = 4 * half, c0 = 12 * half;
        if (ok && m0 < count) {
          float v[4];
          uint32_t x0[16], x1[16];
          tc::ld16(x0, acc + c0);
          tc::ld16(x1, acc + p.cols + c0);
#pragma unroll
          for (int m = 0; m < 4; ++m) v[m] = p.split == 1 && res && m0 + m < count ? residual(m0 + m) : 0.f;
          tc::wait_ld16(x0);
          tc::wait_ld16(x1);
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            float q[3];
#pragma unroll
            for (int c = 0; c < 3; ++c)
              q[c] = (has0 ? __uint_as_float(x0[3 * m + c]) : 0.f) + (has1 ? __uint_as_float(x1[3 * m + c]) : 0.f);
            v[m] += (q[2] + q[1]) + q[0];
          }
          if (p.split == 1) {
            write_results<GATED>(a, n, m0, count - m0, v, lane);
          } else {
#pragma unroll
            for (int m = 0; m < 4; ++m)
              if (m0 + m < count) give(m0 + m, v[m], 0.f);
          }
        }
      } else {
        // Some columns at a time, four warps to them (eight where there is more to do for each,
        // so that both fours have some of a tile of sixteen).
        constexpr int C = GATED ? 8 : kMxOut;
        auto sums = [&](int c0, float* g, float* u) {
          uint32_t x0[C], x1[C];
          const bool second = GATED || p.pair;
          if constexpr (C == 8) {
            tc::ld8(x0, acc + c0);
            tc::ld8(x1, acc + p.cols + c0);
            tc::wait_ld8(x0);
            tc::wait_ld8(x1);
          } else {
            tc::ld16(x0, acc + c0);
            if (second) tc::ld16(x1, acc + p.cols + c0);
            tc::wait_ld16(x0);
            if (second) tc::wait_ld16(x1);
          }
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const float s0 = __uint_as_float(x0[c]), s1 = second ? __uint_as_float(x1[c]) : 0.f;
            g[c] = GATED ? s0 : (has0 ? s0 : 0.f) + (has1 ? s1 : 0.f);
            if constexpr (GATED) u[c] = s1;
          }
        };
        for (int c0 = half * C; c0 < count; c0 += 2 * C) {
          float g[C], u[GATED ? C : 1];
          if (p.split > 1) {
            sums(c0, g, u);
#pragma unroll
            for (int c = 0; c < C; ++c)
              if (ok && c0 + c < count) give(c0 + c, g[c], GATED ? u[c] : 0.f);
            continue;
          }
          if constexpr (GATED) {
            sums(c0, g, u);
#pragma unroll
            for (int c = 0; c < C; ++c) g[c] = mx_silu(g[c]) * u[c];
            if (ok) write_results<GATED>(a, n, tok + c0, count - c0, g, lane);
          } else if (ld.wide) {
            // Through shared memory: each warp writes four rows of x, a lane four weight rows
            // of each.
            const int m0 = c0 + 4 * quarter, n4 = row + 4 * lane;
            const long long at = static_cast<long long>(tok + m0) * a.N + n4;
            const bool live = ok && n4 < a.N;
            uint2 r[4] = {};
            if (a.res != nullptr) {
              // (all four under way together: rows and columns that there are not are others again)
              const __half* from = a.res + static_cast<long long>(tok) * a.N + min(n4, a.N - 4);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                r[i] = *reinterpret_cast<const uint2*>(from + static_cast<long long>(min(m0 + i, count - 1)) * a.N);
            }
            sums(c0, g, u);
            named_bar_sync(1 + half, 128);  // the last columns' values have been read
#pragma unroll
            for (int c = 0; c < 16; ++c)
              asm volatile("st.shared.f32 [%0], %1;" ::"r"(stage_out + (c * kRowsW + quarter * 32 + lane) * 4),
                           "f"(g[c])
                           : "memory");
            named_bar_sync(1 + half, 128);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float v[4];
              asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                           : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                           : "r"(stage_out + ((4 * quarter + i) * kRowsW + 4 * lane) * 4)
                           : "memory");
              const float2 a0 = __half22float2(*reinterpret_cast<const __half2*>(&r[i].x));
              const float2 a1 = __half22float2(*reinterpret_cast<const __half2*>(&r[i].y));
              if (live && m0 + i < count)
                *reinterpret_cast<uint2*>(a.y + at + static_cast<long long>(i) * a.N) =
                    make_uint2(pack_f16(v[0] + a0.x, v[1] + a0.y), pack_f16(v[2] + a1.x, v[3] + a1.y));
            }
          } else {
            __half r[16];
            if (a.res != nullptr) {
              const __half* from = a.res + static_cast<long long>(tok) * a.N + min(n, a.N - 1);
#pragma unroll
              for (int c = 0; c < 16; ++c) r[c] = from[static_cast<long long>(min(c0 + c, count - 1)) * a.N];
            }
            sums(c0, g, u);
            if (a.res != nullptr) {
#pragma unroll
              for (int c = 0; c < 16; ++c) g[c] += __half2float(r[c]);
            }
            if (ok) write_results<GATED>(a, n, tok + c0, count - c0, g, lane);
          }
        }
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.acc_empty[buf]));
      if (p.split == 1) continue;
      step_wait<true>(smem_u32(&bars.part_full), n_t & 1, &s_failed, &g_status);
      const bool all = __all_sync(0xFFFFFFFFu, *static_cast<volatile int*>(&s_failed) == 0);
      if (all) {
        for (int j = half; j < own; j += 2) {
          const int m = rank + j * p.split;
          const float r = res ? residual(m) : 0.f;
          float g[8], u[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            g[q] = u[q] = 0.f;
            if (q < p.split) {
              asm volatile("ld.shared.f32 %0, [%1];" : "=f"(g[q]) : "r"(part_at(q, j, 0)));
              if (GATED) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(u[q]) : "r"(part_at(q, j, 1)));
            }
          }
          float v[1], w = u[0];
          v[0] = g[0];
#pragma unroll
          for (int q = 1; q < 8; ++q) v[0] += g[q], w += u[q];
          v[0] = GATED ? mx_silu(v[0]) * w : v[0] + r;
          write_results<GATED>(a, n, tok + m, 1, v, lane);
        }
      }
      __syncwarp();
      // (after the last tile nobody waits for this, and who would be told may have ended)
      if (t + stride < tiles && lane < p.split) mbar_arrive_cluster(map_rank(smem_u32(&bars.part_done), lane));
    }
  }
  tc::fence_before();
  __syncthreads();
  // Every copy and every sum of another rank has been waited for by who uses it.  After a
  // wait that ran out: time for copies in flight, and for the ranks that may still send (the
  // barrier waits for those that have not ended).
  if (s_failed != 0) {
    for (const uint64_t t0 = global_timer_ns(); global_timer_ns() - t0 < 2000000ull;) {
    }
    __syncthreads();
    if (p.split > 1) {
      cluster_arrive();
      cluster_wait();
    }
  }
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------- host

// The plans of a shape, and whether pairs of blocks are expected to be faster; a thread
// keeps those that it met last (a search takes a few microseconds, as long as all else of a
// call).
struct Plans {
  MxShape shape;
  int pairs;  // of blocks that run at a time
  MxPlan plan;
  MxPairPlan pair;
  bool by_pairs;
};

const Plans* known_plans(const MxShape& s, int pairs) {
  static thread_local Plans known[32] = {};
  const unsigned long long h = (static_cast<unsigned long long>(s.M) * 0x9E3779B97F4A7C15ull) ^
                               (static_cast<unsigned long long>(s.N) * 0xC2B2AE3D27D4EB4Full) ^
                               (static_cast<unsigned long long>(s.K) * 0x165667B19E3779F9ull);
  Plans& at = known[(h >> 40) % 32];
  if (at.shape == s && at.pairs == pairs) return &at;
  Plans p{s, pairs, {}, {}, false};
  if (!mx_plan(s, &p.plan)) return nullptr;
  double cost = 0;
  MxShape of_pairs = s;
  of_pairs.clusters[1] = pairs;
  p.by_pairs = mx_pair_plan(of_pairs, &p.pair, &cost) && cost < mx_cost(s, p.plan);
  at = p;
  return &at;
}

template <bool GATED, bool SPLIT>
cudaError_t launch(const MxProductArgs& a, int sms, int device, cudaStream_t st) {
  constexpr auto* k = mx_product_kernel<GATED, SPLIT>;
  if (const cudaError_t e = allow_smem<k>(device); e != cudaSuccess) return e;
  MxShape shape{a.M, a.N, a.K, GATED, SPLIT, {}};
  for (int i = 0; i < 4; ++i) shape.clusters[i] = clusters_at_a_time<k>(i, kThreads, sms, device);
  const int pairs = SPLIT ? 0 : mx_pair_clusters(GATED, sms, device);
  const Plans* plans = known_plans(shape, pairs);
  if (plans == nullptr) return cudaErrorInvalidValue;
  if (plans->by_pairs && mx_pair_takes(a)) return mx_pair_launch(a, plans->pair, pairs, device, st);
  const MxPlan p = plans->plan;
  auto mod = [](const void* q, uintptr_t m) { return (reinterpret_cast<uintptr_t>(q) & (m - 1)) == 0; };
  MxLoads ld;
  ld.tma_w = a.K % kStepK == 0 && mod(a.w, 32) && (!GATED || mod(a.up, 32));
  const bool all16 = mod(a.ws, 16) && mod(a.us, 16) && mod(a.xs, 16);
  const bool all4 = mod(a.ws, 4) && mod(a.us, 4) && mod(a.xs, 4);
  ld.wide = a.N % 4 == 0 && mod(a.y, 8) && mod(a.res, 8);
  ld.bytes = a.K % 512 == 0 && all16 ? 16 : a.K % kStepK == 0 && all4 ? 4 : 1;
  CUtensorMap wm{}, um{}, xm{};
  if (ld.tma_w && (!encode_codes(&wm, a.w, true, a.N, a.K, kRowsW) ||
                  (GATED && !encode_codes(&um, a.up, true, a.N, a.K, kRowsW))))
    return cudaErrorInvalidValue;
  if (!SPLIT && !encode_codes(&xm, a.x, false, a.M, a.K, p.cols)) return cudaErrorInvalidValue;
  const long long tiles = static_cast<long long>(p.row_tiles) * p.tok_tiles;
  const long long most = shape.clusters[__builtin_ctz(p.split)], clusters = tiles < most ? tiles : most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * p.split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, a, p, ld, wm, um, xm);
}

}  // namespace

cudaError_t mx_product_launch(const MxProductArgs& a, int sms, int device, cudaStream_t st) {
  if (a.x16 != nullptr) return launch<false, true>(a, sms, device, st);
  return a.up != nullptr ? launch<true, false>(a, sms, device, st) : launch<false, false>(a, sms, device, st);
}

cudaError_t status_mx(unsigned* out) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_status, sizeof(v));
  if (e != cudaSuccess) return e;
  e = cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
  *out |= v;
  return e == cudaSuccess ? status_mx_pair(out) : e;
}

}  // namespace qgemv
