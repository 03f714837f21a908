// mx_product.cu -- products with MXFP4 weights (qgemv_mxfp4, qgemv_mx_gemm,
// qgemv_mx_swiglu) on the block-scaled tensor-core instruction.
//
//   D[n][c] = sum over blocks b of 2^(sw[n][b] + sx[c][b]) sum_{k in b} w[n][k] x[c][k]
//
// A tile is 128 weight rows (the instruction's A operand, 4-bit codes as they are
// stored, spread to bytes by the copy itself) by up to 240 columns (B, e4m3): nothing
// is dequantised by arithmetic, the scales go to tensor memory and into the product.
// Columns are the MXFP8 rows of x, or for fp16 rows three columns each: x / 2^e1 = q1 +
// q2 / 2^4 + q3 / 2^9 with e4m3 q1, q2, q3 and e1 = floor(log2 of the block's largest) - 7.
// Each q takes four bits of what is left, so the eleven bits of an fp16 value are
// all held, down to 2^-26 of the block's largest value; the three sums are added in fp32.
//
// A step is 128 k: a ring of stages (codes of A and B, 128-byte swizzled, and their
// scales) between
//   warp 9     TMA: codes of A (where K and the address allow it) and of MXFP8 rows;
//   warps 4-7  scales, fp16 rows and what TMA cannot load, by cp.async, kLag steps ahead of
//              the arrival that hands them on;
//   warp 8     scales to tensor memory, four products (gated: eight) a step;
//   warps 0-3  results: a weight row per lane, a column at a time; two accumulators,
//              so that the next tile's products run meanwhile.
// Thread blocks stay for the whole call and take tiles one after the other.  Where
// there are few tiles, the blocks of a cluster share K: each leaves its sums in its
// shared memory and finishes every split-th column, adding the others' in rank order.
#include <atomic>

#include "kv_cache.cuh"
#include "mma_tile.cuh"
#include "mx.h"
#include "mx_format.cuh"
#include "tcgen05.cuh"
#include "tensor_map.h"

namespace qgemv {
namespace {

__device__ unsigned g_status = 0;

constexpr int kRowsW = 128;   // weight rows of a tile
constexpr int kStepK = 128;   // k of a stage
constexpr int kThreads = 320;
constexpr int kLoadWarp = 4, kMmaWarp = 8, kTmaWarp = 9;
constexpr int kLag = 3;       // steps between a load's start and the wait for it
constexpr int kMinStages = 4, kMaxStages = 16;
constexpr int kScaleCols = 16;                    // tensor memory of one step's scales
constexpr int kAccCols = 512 - 2 * kScaleCols;    // and of the accumulators
constexpr int kSplitTokens = 64;                  // most columns whose sums blocks share

// What a launch is made of.
struct MxPlan {
  int cols;      // columns of a tile
  int tokens;    // rows of x of a tile
  int split;     // blocks that share K (a cluster)
  int stages;
  int row_tiles, tok_tiles;
  bool rows_first;   // tiles of rows change fastest
  bool tma_w;        // weights by TMA
  bool words_w, words_u, words_x;  // scales by aligned words
};

struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t part_full, part_done;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float load_remote(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void fence_cluster() {
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int BYTES>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, bool take) {
  const int n = take ? BYTES : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n)
               : "memory");
}

// Four scale bytes of a row, from block kb on; what lies behind the row's end is 0.
__device__ __forceinline__ uint32_t scale_word(const uint8_t* row, int kb, int blocks) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (kb + i < blocks) w |= static_cast<uint32_t>(row[kb + i]) << (8 * i);
  return w;
}

// Place of row r's word among the scales of a step.
__device__ __forceinline__ int scale_at(int r) { return (r >> 7) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4; }

// GATED: two weights.  SPLIT3: fp16 rows.
template <bool GATED, bool SPLIT3>
__global__ void __launch_bounds__(kThreads, 1)
    mx_product_kernel(const MxProductArgs a, const MxPlan p, const __grid_constant__ CUtensorMap w_map,
                      const __grid_constant__ CUtensorMap u_map, const __grid_constant__ CUtensorMap x_map) {
  constexpr int kW = GATED ? 2 : 1;
  extern __shared__ uint8_t raw_smem[];
  __shared__ Bars bars;
  __shared__ uint32_t s_tmem;
  __shared__ int s_failed;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const uint32_t base = (smem_u32(raw_smem) + 1023) & ~1023u;
  const int b_bytes = p.cols * kStepK;
  const uint32_t a_ring = base, b_ring = a_ring + p.stages * kW * 16384;
  const uint32_t s_ring = b_ring + p.stages * b_bytes;            // scales: A, (up,) B
  const int s_bytes = 512 * (kW + (p.cols > 128 ? 2 : 1));
  const uint32_t x_ring = s_ring + p.stages * s_bytes;            // fp16 rows as they are
  const uint32_t part = x_ring + (SPLIT3 ? p.stages * p.tokens * 256 : 0);

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(smem_u32(&bars.full[i]), 4 + (p.tma_w || !SPLIT3 ? 1 : 0));
      mbar_init(smem_u32(&bars.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars.acc_full[i]), 1);
      mbar_init(smem_u32(&bars.acc_empty[i]), 4);
    }
    mbar_init(smem_u32(&bars.part_full), 4 * p.split);
    mbar_init(smem_u32(&bars.part_done), 4 * p.split);
    fence_mbar_init();
    s_failed = 0;
  }
  if constexpr (SPLIT3) {
    // columns that no row of x writes
    for (uint32_t i = threadIdx.x; i < static_cast<uint32_t>(p.stages * (b_bytes + s_bytes)) / 16; i += kThreads)
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(b_ring + 16 * i), "r"(0) : "memory");
    tc::fence_async_shared();
  }
  pdl_wait();
  if (warp == kMmaWarp) tc::alloc(smem_u32(&s_tmem), 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  pdl_launch_dependents();
  if (p.split > 1) cluster_sync();  // barriers are there before a rank arrives on another's
  const uint32_t tmem = s_tmem;

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

  if (warp == kTmaWarp) {
    // ------------------------------------------------------------------ TMA
    if (p.tma_w || !SPLIT3) {
      int stage = 0, use = 0;
      const uint32_t bytes = (p.tma_w ? kW * 8192 : 0) + (SPLIT3 ? 0 : b_bytes);
      for (long long t = first; t < tiles; t += stride) {
        int row, tok;
        place(t, &row, &tok);
        for (int k = k0; k < k1; ++k) {
          if (use > 0) step_wait(smem_u32(&bars.empty[stage]), (use - 1) & 1, &s_failed, &g_status);
          if (lane == 0) {
            const uint32_t full = smem_u32(&bars.full[stage]);
            mbar_arrive_expect_tx(full, bytes);
            if (p.tma_w) {
              tc::tma_2d(a_ring + stage * kW * 16384, &w_map, k * kStepK, row, full);
              if (GATED) tc::tma_2d(a_ring + (stage * kW + 1) * 16384, &u_map, k * kStepK, row, full);
            }
            if (!SPLIT3) tc::tma_2d(b_ring + stage * b_bytes, &x_map, k * kStepK, tok, full);
          }
          __syncwarp();
          if (++stage == p.stages) stage = 0, ++use;
        }
      }
      // no copy may be in flight when the block ends
      const int turn = use > 0 ? p.stages : stage;
      for (int i = 0; i < turn; ++i) {
        if (--stage < 0) stage = p.stages - 1, --use;
        warp_wait(smem_u32(&bars.full[stage]), use & 1, &g_status);
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------- products
    const uint32_t tm = static_cast<uint32_t>(tc::uniform(static_cast<int>(tmem)));
    const uint32_t idesc = tc::idesc_mx(p.cols);
    int stage = 0, use = 0, n = 0;
    for (long long t = first; t < tiles; t += stride, ++n) {
      const int buf = n & 1;
      if (n >= 2) step_wait(smem_u32(&bars.acc_empty[buf]), ((n >> 1) - 1) & 1, &s_failed, &g_status);
      tc::fence_after();
      const uint32_t acc = tm + buf * (kW * p.cols);
      for (int k = k0; k < k1; ++k) {
        step_wait(smem_u32(&bars.full[stage]), use & 1, &s_failed, &g_status);
        tc::fence_after();
        if (tc::elect_one()) {
          const uint32_t st = tm + kAccCols + (k & 1) * kScaleCols;
          const uint32_t ss = s_ring + stage * s_bytes;
          tc::copy_scales(st, ss);
          if (GATED) tc::copy_scales(st + 4, ss + 512);
          tc::copy_scales(st + 8, ss + kW * 512);
          if (p.cols > 128) tc::copy_scales(st + 12, ss + (kW + 1) * 512);
          const uint64_t b = tc::desc_k_major(b_ring + stage * b_bytes);
#pragma unroll
          for (int w = 0; w < kW; ++w) {
            const uint64_t wd = tc::desc_k_major(a_ring + (stage * kW + w) * 16384);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              tc::mma_mx(acc + w * p.cols, wd + 2 * j, b + 2 * j, idesc, j, st + 4 * w, st + 8,
                         k > k0 || j > 0);
          }
          tc::commit(smem_u32(&bars.empty[stage]));
        }
        __syncwarp();
        if (++stage == p.stages) stage = 0, ++use;
      }
      if (tc::elect_one()) tc::commit(smem_u32(&bars.acc_full[buf]));
      __syncwarp();
    }
  } else if (warp >= kLoadWarp) {
    // ---------------------------------------------------------------- loads
    const int th = threadIdx.x - kLoadWarp * 32, blocks = a.K / kMxBlock;
    int stage = 0, use = 0;      // of the step whose loads start next
    int late = 0;                // stage of the step that is handed on next
    int started = 0;             // steps under way, up to kLag
    // fp16 rows: this thread's eight values of a step (row th / 16 of the tile)
    auto convert = [&](int s) {
      const int m = th >> 4, ch = th & 15;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (m < p.tokens)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(x_ring + (s * p.tokens + m) * 256 + ch * 16));
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
      float f[8];
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
        f[2 * i] = h.x, f[2 * i + 1] = h.y;
        most = max(most, max(__float_as_uint(h.x) & 0x7FFFFFFFu, __float_as_uint(h.y) & 0x7FFFFFFFu));
      }
      most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
      most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
      if (m >= p.tokens) return;
      // 2^e1 with e1 + 127 = byte; the largest value is then below 2^8
      const int e = static_cast<int>(most >> 23), byte = max(e, 103) - 7;
      const float inv = mx_inverse(byte);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= inv;
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        const float next = q == 0 ? 16.f : 32.f;
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t two = mx_codes8(f[2 * i], f[2 * i + 1]);
          const float2 got = mx_values8(two);
          f[2 * i] = (f[2 * i] - got.x) * next;
          f[2 * i + 1] = (f[2 * i + 1] - got.y) * next;
          w[i >> 1] = i & 1 ? w[i >> 1] | (two << 16) : two;
        }
        const int c = 3 * m + q;
        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(b_ring + s * b_bytes + c * 128 +
                                                             (((ch >> 1) ^ (c & 7)) << 4) + (ch & 1) * 8),
                     "r"(w[0]), "r"(w[1])
                     : "memory");
        const int sb = e == 255 ? 255 : byte - (q == 0 ? 0 : q == 1 ? 4 : 9);
        if ((ch & 3) == 0)
          asm volatile("st.shared.u8 [%0], %1;" ::"r"(s_ring + s * s_bytes + kW * 512 + scale_at(c) + (ch >> 2)),
                       "r"(sb)
                       : "memory");
      }
    };
    auto hand_on = [&] {
      if constexpr (SPLIT3) convert(late);
      tc::fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.full[late]));
      if (++late == p.stages) late = 0;
    };
    for (long long t = first; t < tiles; t += stride) {
      int row, tok;
      place(t, &row, &tok);
      const int n = row + th, m0 = tok + th, m1 = m0 + 128;
      const bool has_n = n < a.N;
      const uint8_t* wsr = a.ws + static_cast<long long>(has_n ? n : 0) * blocks;
      const uint8_t* usr = GATED ? a.us + static_cast<long long>(has_n ? n : 0) * blocks : nullptr;
      const bool has_0 = !SPLIT3 && th < p.tokens && m0 < a.M;
      const bool has_1 = !SPLIT3 && th + 128 < p.tokens && m1 < a.M;
      const uint8_t* xs0 = has_0 ? a.xs + static_cast<long long>(m0) * blocks : nullptr;
      const uint8_t* xs1 = has_1 ? a.xs + static_cast<long long>(m1) * blocks : nullptr;
      for (int k = k0; k < k1; ++k) {
        // scales whose words are not aligned, before the wait
        uint32_t sw = 0, su = 0, sx0 = 0, sx1 = 0;
        if (!p.words_w && has_n) sw = scale_word(wsr, 4 * k, blocks);
        if (GATED && !p.words_u && has_n) su = scale_word(usr, 4 * k, blocks);
        if (!p.words_x && has_0) sx0 = scale_word(xs0, 4 * k, blocks);
        if (!p.words_x && has_1) sx1 = scale_word(xs1, 4 * k, blocks);
        if (use > 0) step_wait(smem_u32(&bars.empty[stage]), (use - 1) & 1, &s_failed, &g_status);
        const uint32_t ss = s_ring + stage * s_bytes;
        auto put = [&](uint32_t at, bool words, bool has, const uint8_t* from, uint32_t w) {
          if (words)
            cp_async_small<4>(at, has ? static_cast<const void*>(from + 4 * k) : a.w, has);
          else
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(w) : "memory");
        };
        put(ss + scale_at(th), p.words_w, has_n, wsr, sw);
        if (GATED) put(ss + 512 + scale_at(th), p.words_u, has_n, usr, su);
        if constexpr (SPLIT3) {
          const int m = th >> 4, at = k * kStepK + (th & 15) * 8;
          if (m < p.tokens) {
            const bool has = at < a.K;
            cp_async16(x_ring + (stage * p.tokens + m) * 256 + (th & 15) * 16,
                       a.x16 + (has ? static_cast<long long>(m) * a.K + at : 0), has);
          }
        } else {
          if (th < p.tokens) put(ss + kW * 512 + scale_at(th), p.words_x, has_0, xs0, sx0);
          if (th + 128 < p.tokens) put(ss + kW * 512 + scale_at(th + 128), p.words_x, has_1, xs1, sx1);
        }
        if (!p.tma_w) {
#pragma unroll
          for (int w = 0; w < kW; ++w)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int i = th + 128 * j, r = i >> 3, c = i & 7;
              const bool has = row + r < a.N && k * kStepK + c * 16 < a.K;
              const uint32_t* from = (w ? a.up : a.w) +
                  (has ? static_cast<long long>(row + r) * (a.K / 8) + k * (kStepK / 8) + c * 2 : 0);
              cp_async_small<8>(a_ring + (stage * kW + w) * 16384 + r * 128 + ((c ^ (r & 7)) << 4), from, has);
            }
        }
        cp_commit();
        if (started == kLag) {
          cp_wait<kLag>();
          hand_on();
        } else {
          ++started;
        }
        if (++stage == p.stages) stage = 0, ++use;
      }
    }
    cp_wait<0>();
    for (; started > 0; --started) hand_on();
  } else {
    // -------------------------------------------------------------- results
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp) << 21);
    // The finished value of weight row n and row m of x.
    auto finish = [&](int n, int m, float v) {
      const long long at = static_cast<long long>(m) * a.N + n;
      if (a.y != nullptr && n < a.N) a.y[at] = __float2half_rn(v);
      if (GATED && a.yc != nullptr) {
        // (N is a multiple of 32: a warp's rows are one block of the output, all there or none)
        const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v) & 0x7FFFFFFFu);
        const int byte = mx_scale_byte<8>(__uint_as_float(most));
        if (n < a.N) {
          a.yc[at] = static_cast<uint8_t>(mx_codes8(v * mx_inverse(byte), 0.f));
          if (lane == 0) a.ys[at >> 5] = static_cast<uint8_t>(byte);
        }
      }
    };
    int n_t = 0;
    for (long long t = first; t < tiles; t += stride, ++n_t) {
      int row, tok;
      place(t, &row, &tok);
      const int buf = n_t & 1, n = row + warp * 32 + lane, count = min(p.tokens, a.M - tok);
      step_wait(smem_u32(&bars.acc_full[buf]), (n_t >> 1) & 1, &s_failed, &g_status);
      tc::fence_after();
      const uint32_t acc = lanes + buf * (kW * p.cols);
      const bool res = !GATED && a.res != nullptr && n < a.N;
      if (p.split > 1 && n_t > 0) {
        step_wait(smem_u32(&bars.part_done), (n_t - 1) & 1, &s_failed, &g_status);
        fence_cluster();
      }
      auto out = [&](int m, float g, float u, float r) {  // sums of one column
        if (p.split > 1) {
          const uint32_t at = part + ((m * kW) * kRowsW + warp * 32 + lane) * 4;
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(g) : "memory");
          if (GATED) asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + kRowsW * 4), "f"(u) : "memory");
        } else {
          finish(n, tok + m, GATED ? silu_f(g) * u : g + r);
        }
      };
      const bool ok = __all_sync(0xFFFFFFFFu, *static_cast<volatile int*>(&s_failed) == 0);
      if (ok) {
        if constexpr (SPLIT3) {
          uint32_t v[32];
          if (p.cols == 32) {
            tc::ld32(v, acc);
            tc::wait_ld32(v);
          } else {
            tc::ld16(v, acc);
            tc::wait_ld16(v);
#pragma unroll
            for (int c = 16; c < 32; ++c) v[c] = 0u;
          }
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            if (m >= count) break;
            const float r = p.split == 1 && res ? __half2float(a.res[static_cast<long long>(m) * a.N + n]) : 0.f;
            out(m, (__uint_as_float(v[3 * m + 2]) + __uint_as_float(v[3 * m + 1])) + __uint_as_float(v[3 * m]), 0.f, r);
          }
        } else {
          for (int c0 = 0; c0 < count; c0 += 16) {
            uint32_t g[16], u[16];
            float r[16];
            tc::ld16(g, acc + c0);
            if (GATED) tc::ld16(u, acc + p.cols + c0);
            if (!GATED) {
#pragma unroll
              for (int c = 0; c < 16; ++c)
                r[c] = p.split == 1 && res && c0 + c < count
                           ? __half2float(a.res[static_cast<long long>(tok + c0 + c) * a.N + n])
                           : 0.f;
            }
            tc::wait_ld16(g);
            if (GATED) tc::wait_ld16(u);
#pragma unroll
            for (int c = 0; c < 16; ++c)
              if (c0 + c < count)
                out(c0 + c, __uint_as_float(g[c]), GATED ? __uint_as_float(u[c]) : 0.f, GATED ? 0.f : r[c]);
          }
        }
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.acc_empty[buf]));
      if (p.split == 1) continue;
      // sums of every rank, for the columns that are this one's to finish
      fence_cluster();
      __syncwarp();
      if (lane < p.split) arrive_remote(map_rank(smem_u32(&bars.part_full), lane));
      step_wait(smem_u32(&bars.part_full), n_t & 1, &s_failed, &g_status);
      fence_cluster();
      const bool all = __all_sync(0xFFFFFFFFu, *static_cast<volatile int*>(&s_failed) == 0);
      if (all) {
        for (int m = rank; m < count; m += p.split) {
          const uint32_t at = part + ((m * kW) * kRowsW + warp * 32 + lane) * 4;
          const float r = res ? __half2float(a.res[static_cast<long long>(tok + m) * a.N + n]) : 0.f;
          float g = 0.f, u = 0.f;
          for (int q = 0; q < p.split; ++q) {
            const uint32_t there = map_rank(at, q);
            g += load_remote(there);
            if (GATED) u += load_remote(there + kRowsW * 4);
          }
          finish(n, tok + m, GATED ? silu_f(g) * u : g + r);
        }
      }
      __syncwarp();
      if (lane < p.split) arrive_remote(map_rank(smem_u32(&bars.part_done), lane));
    }
  }
  tc::fence_before();
  __syncthreads();
  if (p.split > 1) cluster_sync();  // sums are read, and barriers arrived on, by other ranks
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------- host

constexpr int kSmemMax = 227 * 1024 - 1024;  // less the kernel's static shared memory

int stage_bytes(int w, int cols, int raw) {
  return w * 16384 + cols * kStepK + 512 * (w + (cols > 128 ? 2 : 1)) + raw;
}

int part_bytes(int w, int tokens, int split) { return split > 1 ? w * tokens * kRowsW * 4 : 0; }

bool encode_codes(CUtensorMap* m, const void* p, bool four, long long rows, int k, int box_rows) {
  const EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dim[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows)};
  const cuuint64_t stride[1] = {static_cast<cuuint64_t>(four ? k / 2 : k)};
  const cuuint32_t box[2] = {kStepK, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estride[2] = {1, 1};
  return fn(m, four ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
            const_cast<void*>(p), dim, stride, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool GATED, bool SPLIT3>
cudaError_t launch(const MxProductArgs& a, int sms, int device, cudaStream_t st) {
  constexpr int kW = GATED ? 2 : 1;
  static std::atomic<unsigned long long> done{0};
  auto* k = mx_product_kernel<GATED, SPLIT3>;
  const unsigned long long bit = 1ull << (device & 63);
  if (!(done.load(std::memory_order_relaxed) & bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_relaxed);
  }
  const int steps = (a.K + kStepK - 1) / kStepK;
  MxPlan p{};
  p.row_tiles = (a.N + kRowsW - 1) / kRowsW;
  if (SPLIT3) {
    p.tokens = a.M;
    p.cols = 3 * a.M <= 16 ? 16 : 32;
    p.tok_tiles = 1;
  } else {
    const int most = kAccCols / (2 * kW) / 16 * 16;
    p.tok_tiles = (a.M + most - 1) / most;
    p.cols = ((a.M + p.tok_tiles - 1) / p.tok_tiles + 15) / 16 * 16;
    p.tokens = p.cols;
    p.tok_tiles = (a.M + p.cols - 1) / p.cols;
  }
  p.split = 1;
  const long long tiles = static_cast<long long>(p.row_tiles) * p.tok_tiles;
  if (p.tokens <= kSplitTokens / kW)
    while (p.split < 8 && tiles * p.split * 2 <= sms && steps >= p.split * 4) p.split *= 2;
  const int raw = SPLIT3 ? p.tokens * 256 : 0;
  const int room = kSmemMax - 1024 - part_bytes(kW, p.tokens, p.split);
  p.stages = room / stage_bytes(kW, p.cols, raw);
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  if (p.stages < kMinStages) return cudaErrorInvalidValue;
  const int smem = 1024 + p.stages * stage_bytes(kW, p.cols, raw) + part_bytes(kW, p.tokens, p.split);
  auto mod = [](const void* q, uintptr_t m) { return (reinterpret_cast<uintptr_t>(q) & (m - 1)) == 0; };
  p.tma_w = a.K % kStepK == 0 && mod(a.w, 32) && (!GATED || mod(a.up, 32));
  p.words_w = a.K % kStepK == 0 && mod(a.ws, 4);
  p.words_u = a.K % kStepK == 0 && mod(a.us, 4);
  p.words_x = a.K % kStepK == 0 && mod(a.xs, 4);
  p.rows_first = static_cast<long long>(a.M) * 2 > static_cast<long long>(a.N) * kW;
  CUtensorMap wm{}, um{}, xm{};
  if (p.tma_w && (!encode_codes(&wm, a.w, true, a.N, a.K, kRowsW) ||
                  (GATED && !encode_codes(&um, a.up, true, a.N, a.K, kRowsW))))
    return cudaErrorInvalidValue;
  if (!SPLIT3 && !encode_codes(&xm, a.x, false, a.M, a.K, p.cols)) return cudaErrorInvalidValue;
  const long long clusters = tiles < sms / p.split ? tiles : sms / p.split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * p.split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
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
  return cudaLaunchKernelEx(&cfg, k, a, p, wm, um, xm);
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
  return e;
}

}  // namespace qgemv
