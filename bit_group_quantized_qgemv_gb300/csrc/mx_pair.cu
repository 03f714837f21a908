// mx_pair.cu -- products with MXFP4 weights and many MXFP8 rows (qgemv_mx_gemm,
// qgemv_mx_swiglu) by pairs of thread blocks.
//
// The same products as mx_product.cu, in tiles of 256 weight rows that the tensor cores of
// two multiprocessors work on together: each block has 128 of the rows and half of the
// columns, whose codes either tensor core reads from both.  A step of 224 columns keeps the tensor
// core busy for 448 clocks; in a tile of one block its 16 KB of weights and 28 KB of columns
// move into the product and 36 KB into shared memory, at 128 bytes a clock longer than that; in a
// pair the columns are half of it.
// Measured (us, at 2.07 GHz; those with two figures in the first milliseconds at some 1.7 GHz and
// then under the card's power cap at 1.4 to 1.7), pairs against blocks by themselves, each at its
// best width: 4096 rows of K = 14336 to 4096 131 and 151 against 156 and 168, 8192 of 8192 x 8192
// 292 and 336 against 329 and 372, 1000 rows of 4096 x 4096 16.5 against 18.6, 64 rows 7.9 against 9.3;
// gated 512 rows of 4096 to 14336 46 and 50 against 52 and 53, 2048 rows 142 and 164 against 156 and 174; but
// 64 rows of K = 14336 19.4 against 14.0 (which share K), and gated 1024 rows of 1024 to 2816
// 14.4 against 12.4, where results take longer than the steps (here they change places on the
// way).  Which of the two is expected to be faster mx_plan.h says.  By time and clock a step of 224
// columns takes 480 to 490 clocks, results of the last tile and the start included; one of up to 96
// some 280, about what the copy takes to spread 128 x 128 codes.
//
// Gated: a block's 128 rows are 64 of the gate and the same 64 of the other weight, so that
// one product has both.  Results change places between the warps of the two halves through
// shared memory, each warp finishing half of the columns of 32 rows.
//
// Warps as there: two for codes (TMA alone: other K and addresses take the other kernel); four
// for scales (each block holds its rows' and all columns'); two in the block of rank 0 that
// issue for both, every other step each into an accumulator of its own (64 columns, K = 14336:
// 284 clocks a step, 316 with one), with over 96 columns one for all; in the other block they
// hand on, to rank 0's barrier, that a stage is full there; eight for results.
#include "mx_product.cuh"

namespace qgemv {
namespace {

__device__ unsigned g_status = 0;

constexpr int kRowsW = kMxRows, kStepK = kMxStep;
constexpr int kOutWarps = 8, kLoaders = 4, kTmaWarps = 2;
constexpr int kLoadWarp = kOutWarps, kMmaWarp = kLoadWarp + kLoaders, kTmaWarp = kMmaWarp + 2,
              kThreads = 32 * (kTmaWarp + kTmaWarps);

// All but `turn` are arrived on by the other block too (by its tensor core, or as a stage that is
// full there and an accumulator that has been read): waits for them are in the cluster's scope,
// and order shared memory alone.  Places of tensor memory have fences of their own.
struct Bars {
  uint64_t full[kMxMaxStages], empty[kMxMaxStages];
  uint64_t turn[kLoaders];  // a loader may go on to its group
  uint64_t acc_full[2], acc_empty[2];
};

// TWO: every other step's products into a second accumulator, by a warp of their own.
template <bool GATED, bool TWO>
__global__ void __launch_bounds__(kThreads, 1)
    mx_pair_kernel(const MxProductArgs a, const MxPairPlan p, const bool wide16, const bool wide,
                   const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap u_map,
                   const __grid_constant__ CUtensorMap x_map) {
  constexpr int kRows = GATED ? 64 : 128;  // rows of results of a block
  extern __shared__ uint8_t raw_smem[];
  __shared__ Bars bars;
  __shared__ uint32_t s_tmem;
  __shared__ int s_failed;
  const int warp = tc::uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int rank = tc::uniform(static_cast<int>(cluster_rank()));
  const uint32_t base = (smem_u32(raw_smem) + 1023) & ~1023u;
  const int c_bytes = kRowsW * kStepK + p.cols / 2 * kStepK;  // a stage: this block's A and B
  const int s_bytes = 512 * (p.cols > 128 ? 3 : 2);           // and scales: A, all columns
  const uint32_t s_ring = base + p.stages * c_bytes;
  const uint32_t out = s_ring + p.stages * s_bytes;
  const int steps = a.K / kStepK, blocks = a.K / kMxBlock;
  const long long tiles = static_cast<long long>(p.row_tiles) * p.tok_tiles;
  const long long first = blockIdx.x / 2, stride = gridDim.x / 2;
  auto place = [&](long long tile, int* row, int* tok) {  // this block's first row, the tile's column
    const int fast = p.rows_first ? p.row_tiles : p.tok_tiles;
    const int i = static_cast<int>(tile % fast), o = static_cast<int>(tile / fast);
    *row = ((p.rows_first ? i : o) * 2 + rank) * kRows;
    *tok = (p.rows_first ? o : i) * p.cols;
  };

  // The first tile's weights on their way to L2 while the kernel before ends.
  if (first < tiles) {
    int row, tok;
    place(first, &row, &tok);
    if (warp == kTmaWarp && lane == 0) {
      for (int k = 0; k < steps && k < p.stages; ++k) {
        tc::prefetch_2d(&w_map, k * kStepK, row);
        if (GATED) tc::prefetch_2d(&u_map, k * kStepK, row);
      }
    } else if (warp >= kLoadWarp && warp < kMmaWarp) {
      const int i = threadIdx.x - kLoadWarp * 32, n = row + (i & (kRows - 1));
      if (n < a.N) prefetch_l2((GATED && i >= kRows ? a.us : a.ws) + static_cast<long long>(n) * blocks);
    }
  }
  if (warp == 0) {
    if (lane < p.stages) {
      // the block's scales and copies, and for the one that issues the other's as well
      mbar_init(smem_u32(&bars.full[lane]), rank == 0 ? 3 : 2);
      mbar_init(smem_u32(&bars.empty[lane]), 1);
    }
    if (lane < kLoaders) mbar_init(smem_u32(&bars.turn[lane]), 1);
    if (lane < 2) {
      mbar_init(smem_u32(&bars.acc_full[lane]), TWO ? 2 : 1);
      mbar_init(smem_u32(&bars.acc_empty[lane]), 2 * kOutWarps);
    }
    if (lane == 0) s_failed = 0;
    fence_mbar_init();
  }
  __syncthreads();
  cluster_arrive();
  pdl_wait();
  if (warp == kMmaWarp) tc::alloc_pair(smem_u32(&s_tmem), 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  pdl_launch_dependents();
  cluster_wait();  // barriers are there before the other block arrives on them
  const uint32_t tmem = s_tmem;

  if (warp >= kTmaWarp) {
    // ---------------------------------------------------------------- codes
    const uint32_t bytes = kRowsW * kStepK / 2 + p.cols / 2 * kStepK;
    int stage = warp - kTmaWarp, use = 0, k = stage;  // every other step of all tiles
    long long t = first;
    int row = 0, tok = 0;
    bool moved = true;
    for (;; k += kTmaWarps, stage += kTmaWarps) {
      while (k >= steps && t < tiles) k -= steps, t += stride, moved = true;
      if (t >= tiles) break;
      if (stage >= p.stages) stage -= p.stages, ++use;
      if (moved) place(t, &row, &tok);
      moved = false;
      if (use > 0) step_wait<true>(smem_u32(&bars.empty[stage]), (use - 1) & 1, &s_failed, &g_status);
      if (lane == 0) {
        const uint32_t full = smem_u32(&bars.full[stage]), to = base + stage * c_bytes;
        mbar_arrive_expect_tx(full, bytes);
        tc::tma_2d(to, &w_map, k * kStepK, row, full);
        if (GATED) tc::tma_2d(to + 64 * kStepK, &u_map, k * kStepK, row, full);
        tc::tma_2d(to + kRowsW * kStepK, &x_map, k * kStepK, tok + rank * (p.cols / 2), full);
      }
      __syncwarp();
    }
  } else if (warp >= kMmaWarp) {
    const int me = warp - kMmaWarp;
    int stage = 0, use = 0, n = 0, odd = 0;  // odd: of all tiles' steps, the next one's number
    const bool all = rank == 0 && !TWO;    // the first warp has all steps, not every other one
    auto next = [&] {
      odd ^= 1;
      if (++stage == p.stages) stage = 0, ++use;
    };
    if (rank == 0) {
      // ----------------------------------------------------------- products
      const uint32_t tm = static_cast<uint32_t>(tc::uniform(static_cast<int>(tmem)));
      const uint32_t idesc = tc::idesc_mx(p.cols, 256);
      uint32_t c = base, ss = s_ring;  // of the stage
      for (long long t = first; t < tiles && (TWO || me == 0); t += stride, ++n) {
        const int buf = n & 1;
        if (n >= 2) step_wait<true>(smem_u32(&bars.acc_empty[buf]), ((n >> 1) - 1) & 1, &s_failed, &g_status);
        tc::fence_after();
        const uint32_t acc = tm + (buf * (TWO ? 2 : 1) + me) * p.cols;
        for (int k = 0; k < steps; ++k) {
          if (all || odd == me) {
            step_wait<true>(smem_u32(&bars.full[stage]), use & 1, &s_failed, &g_status);
            tc::fence_after();
            if (tc::elect_one()) {
              const uint32_t st = tm + kMxAccCols + (TWO ? me : k & 1) * 16;
              tc::copy_scales_pair(st, ss);
              tc::copy_scales_pair(st + 8, ss + 512);
              if (p.cols > 128) tc::copy_scales_pair(st + 12, ss + 1024);
              const uint64_t w = tc::desc_k_major(c), b = tc::desc_k_major(c + kRowsW * kStepK);
              const int more = k > (TWO ? 1 : 0);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                tc::mma_mx_pair(acc, w + 2 * j, b + 2 * j, idesc, j, st, st + 8, j > 0 || more);
              tc::commit_pair(smem_u32(&bars.empty[stage]));
            }
            __syncwarp();
          }
          next();
          c = stage == 0 ? base : c + c_bytes, ss = stage == 0 ? s_ring : ss + s_bytes;
        }
        if (tc::elect_one()) tc::commit_pair(smem_u32(&bars.acc_full[buf]));
        __syncwarp();
      }
    } else {
      // a stage that is full here, told to the block that issues
      const uint32_t there = map_rank(smem_u32(&bars.full[0]), 0);
      for (long long t = first; t < tiles; t += stride)
        for (int k = 0; k < steps; ++k, next())
          if (odd == me) {
            step_wait<true>(smem_u32(&bars.full[stage]), use & 1, &s_failed, &g_status);
            if (lane == 0) mbar_arrive_cluster(there + stage * 8);
            __syncwarp();
          }
    }
    // A block that ends has been told of every use of its stages: no arrival is under way.
    for (int i = 0; i < p.stages; ++i) {
      if (stage == 0) stage = p.stages, --use;
      --stage, odd ^= 1;
      if (use < 0) break;
      if (all ? me == 0 : odd == me) step_wait<true>(smem_u32(&bars.empty[stage]), use & 1, &s_failed, &g_status);
    }
  } else if (warp >= kLoadWarp) {
    // --------------------------------------------------------------- scales
    const int me = warp - kLoadWarp, groups = (steps + 3) / 4;  // of four steps, of a tile
    const long long all = first < tiles ? ((tiles - 1 - first) / stride + 1) * groups : 0;
    for (long long g = me; g < all; g += kLoaders) {
      const long long turn = g / groups;
      const int q = static_cast<int>(g % groups), to = min(steps, 4 * q + 4);
      int row, tok;
      place(first + turn * stride, &row, &tok);
      // Scales of rows lane, lane + 32, ... of an operand: of the group's four steps.
      uint4 vw[4], vx[8];
      auto load_all = [&](auto load) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          vw[i] = GATED && i >= 2 ? load(a.us, row + lane + 32 * (i - 2), a.N) : load(a.ws, row + lane + 32 * i, a.N);
#pragma unroll
        for (int i = 0; i < 8; ++i)  // (rows of the next tile are loaded too, and not used)
          vx[i] = load(a.xs, tok + lane + 32 * i, 32 * i < p.cols ? a.M : 0);
      };
      if (wide16) {
        load_all([&](const uint8_t* scales, int r, int end) {
          return r < end ? *reinterpret_cast<const uint4*>(scales + static_cast<long long>(r) * blocks + 16 * q)
                         : make_uint4(0, 0, 0, 0);
        });
      } else {
        load_all([&](const uint8_t* scales, int r, int end) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w[j] = r < end && 4 * q + j < to
                       ? *reinterpret_cast<const uint32_t*>(scales + static_cast<long long>(r) * blocks + 16 * q + 4 * j)
                       : 0;
          return make_uint4(w[0], w[1], w[2], w[3]);
        });
      }
      // One group after the other: a wait for a stage tells a use from the one before it,
      // not from two before.
      if (g > 0)
        step_wait(smem_u32(&bars.turn[me]), ((g / kLoaders) - (me == 0 ? 1 : 0)) & 1, &s_failed, &g_status);
      const long long done = turn * steps + 4 * q;  // steps before the group's
      int stage = static_cast<int>(done % p.stages);
      long long use = done / p.stages;
      int written = 0;  // steps whose scales are to be handed on
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = 4 * q + j;
        if (k >= to) continue;
        if (use > 0) step_wait<true>(smem_u32(&bars.empty[stage]), (use - 1) & 1, &s_failed, &g_status);
        if (k == to - 1 && lane == 0) mbar_arrive(smem_u32(&bars.turn[(me + 1) % kLoaders]));
        const uint32_t ss = s_ring + stage * s_bytes + lane * 16;
        auto word = [&](const uint4& v) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; };
        store_shared(ss, word(vw[0]), word(vw[1]), word(vw[2]), word(vw[3]));
        store_shared(ss + 512, word(vx[0]), word(vx[1]), word(vx[2]), word(vx[3]));
        if (p.cols > 128) store_shared(ss + 1024, word(vx[4]), word(vx[5]), word(vx[6]), word(vx[7]));
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
    // (After a wait that ran out the warps still meet at the barriers, and write nothing.)
    const int quarter = warp & 3, half = warp >> 2;  // lanes of tensor memory; which columns
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter) << 21);
    const uint32_t stage_out = out + half * (kMxOut * kRowsW * 4);
    int n_t = 0, chunk = 0;
    for (long long t = first; t < tiles; t += stride, ++n_t) {
      int row, tok;
      place(t, &row, &tok);
      const int buf = n_t & 1, count = min(p.cols, a.M - tok);
      step_wait<true>(smem_u32(&bars.acc_full[buf]), (n_t >> 1) & 1, &s_failed, &g_status);
      tc::fence_after();
      const uint32_t acc = lanes + buf * (TWO ? 2 : 1) * p.cols;
      // (a tile of a single step has one of two accumulators: the step's)
      const bool has0 = !TWO || steps > 1 || (n_t & 1) == 0, has1 = TWO && (steps > 1 || (n_t & 1) == 1);
      auto sums = [&](int c0, float (&v)[16]) {
        uint32_t x[16], x1[16];
        tc::ld16(x, acc + c0);
        if (TWO) tc::ld16(x1, acc + p.cols + c0);
        tc::wait_ld16(x);
        if (TWO) tc::wait_ld16(x1);
#pragma unroll
        for (int c = 0; c < 16; ++c)
          v[c] = !TWO ? __uint_as_float(x[c]) : (has0 ? __uint_as_float(x[c]) : 0.f) + (has1 ? __uint_as_float(x1[c]) : 0.f);
      };
      const bool ok = __all_sync(0xFFFFFFFFu, *static_cast<volatile int*>(&s_failed) == 0);
      for (int c0 = half * kMxOut; c0 < count; c0 += 2 * kMxOut) {
        float v[16];
        if constexpr (GATED) {
          sums(c0, v);
          // The warps with the gate's rows finish the first eight columns, those with the other
          // weight's the last: each gives its values of the others to its partner.  (Two places in
          // turn: one is written again after everyone has been past the barrier behind its reads.)
          const int part = quarter >> 1, n = row + (quarter & 1) * 32 + lane;
          const uint32_t place_ = stage_out + (chunk & 1) * (kMxOut * 64 * 4);
          auto at = [&](int c) { return place_ + (c * 64 + (quarter & 1) * 32 + lane) * 4; };
          ++chunk;
#pragma unroll
          for (int c = 0; c < 8; ++c)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at(part == 0 ? 8 + c : c)),
                         "r"(__float_as_uint(part == 0 ? v[8 + c] : v[c]))
                         : "memory");
          named_bar_sync(1 + half, 128);
          float h[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            float other;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(other) : "r"(at(part == 0 ? c : 8 + c)) : "memory");
            const float mine = part == 0 ? v[c] : v[8 + c];
            h[c] = mx_silu(part == 0 ? mine : other) * (part == 0 ? other : mine);
          }
          const int m = c0 + 8 * part;
          if (ok) write_results<GATED>(a, n, tok + m, count - m, h, lane);
        } else {
          const int m0 = c0 + 4 * quarter, n4 = row + 4 * lane, n = row + quarter * 32 + lane;
          if (wide) {
            // Through shared memory: each warp writes four rows of x, a lane four weight rows
            // of each.
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
            sums(c0, v);
            named_bar_sync(1 + half, 128);  // the last columns' values have been read
#pragma unroll
            for (int c = 0; c < 16; ++c)
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(stage_out + (c * kRowsW + quarter * 32 + lane) * 4), "r"(__float_as_uint(v[c]))
                           : "memory");
            named_bar_sync(1 + half, 128);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float o[4];
              asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                           : "=f"(o[0]), "=f"(o[1]), "=f"(o[2]), "=f"(o[3])
                           : "r"(stage_out + ((4 * quarter + i) * kRowsW + 4 * lane) * 4)
                           : "memory");
              const float2 a0 = __half22float2(*reinterpret_cast<const __half2*>(&r[i].x));
              const float2 a1 = __half22float2(*reinterpret_cast<const __half2*>(&r[i].y));
              if (live && m0 + i < count)
                *reinterpret_cast<uint2*>(a.y + at + static_cast<long long>(i) * a.N) =
                    make_uint2(pack_f16(o[0] + a0.x, o[1] + a0.y), pack_f16(o[2] + a1.x, o[3] + a1.y));
            }
          } else {
            __half r[16];
            if (a.res != nullptr) {
              const __half* from = a.res + static_cast<long long>(tok) * a.N + min(n, a.N - 1);
#pragma unroll
              for (int c = 0; c < 16; ++c) r[c] = from[static_cast<long long>(min(c0 + c, count - 1)) * a.N];
            }
            sums(c0, v);
#pragma unroll
            for (int c = 0; c < 16; ++c) v[c] += a.res != nullptr ? __half2float(r[c]) : 0.f;
            if (ok) write_results<GATED>(a, n, tok + c0, count - c0, v, lane);
          }
        }
      }
      tc::fence_before();
      __syncwarp();
      // (of the last two tiles nobody waits for this)
      if (lane == 0 && t + 2 * stride < tiles) mbar_arrive_cluster(map_rank(smem_u32(&bars.acc_empty[buf]), 0));
    }
  }
  tc::fence_before();
  __syncthreads();
  // Every copy has been waited for by who uses it; after a wait that ran out, time for those
  // in flight.
  if (s_failed != 0)
    for (const uint64_t t0 = global_timer_ns(); global_timer_ns() - t0 < 2000000ull;) {
    }
  cluster_arrive();  // neither block ends, or frees, before the other has its results
  cluster_wait();
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::dealloc_pair(tmem, 512);
  }
}

template <bool GATED, bool TWO>
cudaError_t launch(const MxProductArgs& a, const MxPairPlan& p, int clusters, int device, cudaStream_t st) {
  constexpr auto* k = mx_pair_kernel<GATED, TWO>;
  if (const cudaError_t e = allow_smem<k>(device); e != cudaSuccess) return e;
  auto mod = [](const void* q, uintptr_t m) { return (reinterpret_cast<uintptr_t>(q) & (m - 1)) == 0; };
  const bool wide16 = a.K % 512 == 0 && mod(a.ws, 16) && mod(a.us, 16) && mod(a.xs, 16);
  const bool wide = a.N % 4 == 0 && mod(a.y, 8) && mod(a.res, 8);
  CUtensorMap wm{}, um{}, xm{};
  if (!encode_codes(&wm, a.w, true, a.N, a.K, GATED ? 64 : kRowsW) ||
      (GATED && !encode_codes(&um, a.up, true, a.N, a.K, 64)) || !encode_codes(&xm, a.x, false, a.M, a.K, p.cols / 2))
    return cudaErrorInvalidValue;
  const long long tiles = static_cast<long long>(p.row_tiles) * p.tok_tiles;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (tiles < clusters ? tiles : clusters)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k, a, p, wide16, wide, wm, um, xm);
}

}  // namespace

// (as many as each of the two kernels has: which one a plan takes follows from it)
int mx_pair_clusters(bool gated, int sms, int device) {
  const int one = gated ? clusters_at_a_time<mx_pair_kernel<true, false>>(1, kThreads, sms, device)
                        : clusters_at_a_time<mx_pair_kernel<false, false>>(1, kThreads, sms, device);
  const int two = gated ? clusters_at_a_time<mx_pair_kernel<true, true>>(1, kThreads, sms, device)
                        : clusters_at_a_time<mx_pair_kernel<false, true>>(1, kThreads, sms, device);
  return one < two ? one : two;
}

bool mx_pair_takes(const MxProductArgs& a) {
  auto mod = [](const void* q, uintptr_t m) { return (reinterpret_cast<uintptr_t>(q) & (m - 1)) == 0; };
  return a.x16 == nullptr && a.K % kMxStep == 0 && mod(a.w, 32) && mod(a.up, 32) && mod(a.ws, 4) && mod(a.us, 4) &&
         mod(a.xs, 4);
}

cudaError_t mx_pair_launch(const MxProductArgs& a, const MxPairPlan& p, int clusters, int device, cudaStream_t st) {
  if (a.up != nullptr)
    return p.two ? launch<true, true>(a, p, clusters, device, st) : launch<true, false>(a, p, clusters, device, st);
  return p.two ? launch<false, true>(a, p, clusters, device, st) : launch<false, false>(a, p, clusters, device, st);
}

cudaError_t status_mx_pair(unsigned* out) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_status, sizeof(v));
  if (e != cudaSuccess) return e;
  e = cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
  *out |= v;
  return e;
}

}  // namespace qgemv
