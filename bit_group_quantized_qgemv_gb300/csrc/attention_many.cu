// attention_many.cu -- qgemv_paged_attention for many query rows per
// key/value head (prompts, chunks of prompts): tcgen05 products, TMA loads.
//
// The work is a list of units: 256 query rows (two tiles of 128, A and B) of one
// (sequence, key/value head) against the tiles of 128 entries that they see.
// One thread block per multiprocessor stays for the whole call and takes
// segments (units, or parts of units, see Scheduler):
//   warp 10     scheduler: finds the block's segments from the lengths on the
//               device and hands them to the others through a ring;
//   warp 9      producer: K and V tiles by TMA, page by page, into a ring of
//               128-byte-swizzled slots (keys and values alternate);
//   warp 8      issues the products: S = Q K^T (operands in shared memory) and
//               O += P V (P in tensor memory, V as the transposed operand);
//   warps 0-3   softmax of tile A, warps 4-7 of tile B: one row per thread,
//               read from tensor memory, weights written back as fp16 over the
//               scores they came from; the queries of the next segment are
//               loaded while the last weights of this one are computed.
// While one tile's weights are computed the tensor core works on the other's
// products.  Tensor memory: S/P of A and B (128 columns each), O of A and B
// (HD each).
//
// The base that weights are relative to is lazy: an older maximum less kLift, until a
// weight would pass 2^kTop, so O is rescaled (a round trip through tensor memory) a few
// times per row instead of at every tile.  Weights are then rounded to 11 bits down
// to 2^-21 of the maximum.
//
// 2048 tokens over 30759 entries (32/8 heads of 128) take 660 us in a few replays of a
// graph, 1.51 PFLOP/s or 79 % of a library product; in calls one after the other, where the
// power limit lowers the clocks, 740 to 770 us, 1.30 to 1.35 PFLOP/s.  What bounds it: Q K^T reads both operands from shared
// memory, which at 128 columns takes its 128 bytes a clock; P V (P in tensor memory)
// does not.  The softmax, in pairs of floats, just hides behind the products: as single
// floats it took 685 us, with an eighth of the exponentials by polynomial 2 % more.
//
// Entries behind the sequence or on bad pages are loaded as zeros (a TMA box
// outside the tensor); the rows of the last page behind the sequence's end,
// which may hold anything, are zeroed in the V tile before the product.
#include <atomic>

#include "attention_common.cuh"
#include "attention_units.cuh"
#include "mma_tile.cuh"
#include "tcgen05.cuh"
#include "kv_tensor_map.h"

namespace qgemv {
namespace {

__device__ unsigned g_status = 0;

// Three warpgroups; the launch gives 168 registers a thread (64,512), of which
// the third group passes on what the two of the softmax need: 256 x 192 + 128 x
// 120 = 64,512.
constexpr int kThreads = 384;
constexpr int kMmaWarp = 8, kTmaWarp = 9;

template <int HD>
struct Shape {
  static constexpr int kHalves = HD / 64;                 // 128-byte columns of a row
  static constexpr int kSlotBytes = kTile * HD * 2;
  static constexpr int kSlots = HD == 128 ? 5 : 10;
  static constexpr int kSmem = 1024 + (2 + kSlots) * kSlotBytes;
  static_assert(kSmem + 2048 <= 227 * 1024, "dynamic and static shared memory");
  static constexpr uint32_t kDescS = tc::idesc_f16(kTile, kTile, false);
  static constexpr uint32_t kDescO = tc::idesc_f16(kTile, HD, true);
};

constexpr int kSegs = 4;        // segments the scheduler may be ahead

struct Bars {
  uint64_t full[10], empty[10];
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2], drain;
  uint64_t seg_full[kSegs], seg_empty[kSegs];
};

// A block's piece of work: tiles j0 .. j1 of a unit.
struct Seg {
  int s, h, r0;              // sequence (-1: no more), head, first row
  int first, rows, off, len; // first token, rows and entries of the sequence
  int j0, j1, slot;          // slot: where a part's result goes, -1: the output
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 32 bytes, in one store where they are aligned to it: a row per thread, every
// store touches 32 lines of the cache.
__device__ __forceinline__ void store32(void* p, const uint32_t* v, bool wide) {
  if (wide)
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  else {
    static_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    static_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    attention_many_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap k_map,
                          const __grid_constant__ CUtensorMap v_map) {
  using Sh = Shape<HD>;
  extern __shared__ uint8_t raw[];
  __shared__ Bars bars;
  __shared__ uint32_t s_tmem;
  __shared__ int s_failed;  // a wait ran out
  __shared__ Seg segs[kSegs];
  __shared__ int s_span[kMaxBlocks], s_load[kMaxBlocks];  // the scheduler's
  __shared__ uint8_t s_order[kMaxBlocks];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint8_t* ring = base + 2 * Sh::kSlotBytes;

  if (threadIdx.x == 0) {
    for (int i = 0; i < Sh::kSlots; ++i) {
      mbar_init(smem_u32(&bars.full[i]), 1);
      mbar_init(smem_u32(&bars.empty[i]), 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(smem_u32(&bars.q_full[x]), 4);  // one arrival per warp
      mbar_init(smem_u32(&bars.s_full[x]), 1);
      mbar_init(smem_u32(&bars.p_full[x]), 4);
      mbar_init(smem_u32(&bars.o_full[x]), 1);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(smem_u32(&bars.seg_full[i]), 1);
      mbar_init(smem_u32(&bars.seg_empty[i]), 10);  // softmax, products and producer warps
    }
    mbar_init(smem_u32(&bars.drain), 1);
    fence_mbar_init();
    s_failed = 0;
  }
  // Tensor memory is taken behind the kernel before and ahead of the one behind: no block
  // holds some while it waits for a block that may need it, on the same multiprocessor, to end.
  pdl_wait();
  if (warp == kMmaWarp) tc::alloc(smem_u32(&s_tmem), 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = s_tmem;

  // Segment number n, as every warp but the scheduler reads it; the last look
  // (next_seg) gives its place in the ring back.
  auto look_seg = [&](int n) {
    const int i = n % kSegs;
    step_wait(smem_u32(&bars.seg_full[i]), (n / kSegs) & 1, &s_failed, &g_status);
    Seg g = segs[i];
    // (no segments are read after a wait ran out)
    if (*static_cast<volatile int*>(&s_failed) != 0) g.s = -1;
    g.s = __shfl_sync(0xFFFFFFFFu, g.s, 0);
    return g;
  };
  auto next_seg = [&](int n) {
    const Seg g = look_seg(n);
    if (lane == 0) mbar_arrive(smem_u32(&bars.seg_empty[n % kSegs]));
    return g;
  };
  // Tiles of tile x (0: A, 1: B) of a segment, from its j0 on.
  auto tiles_in = [&](const Seg& g, int x) {
    const int last = min(g.rows, g.r0 + (x + 1) * kTile) - 1;
    if (last < g.r0 + x * kTile) return 0;
    const int see = min(g.len, g.off + div_group(a, last) + 1);
    return max(0, min(g.j1, (see + kTile - 1) / kTile) - g.j0);
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
    if (warp == 10) {
      // -------------------------------------------------------- scheduler
      Scheduler sc(a, lane);
      int n = 0;
      auto emit = [&](bool end, int j0, int j1, int slot) {
        const int i = n % kSegs;
        if (n >= kSegs)
          step_wait(smem_u32(&bars.seg_empty[i]), (n / kSegs - 1) & 1, &s_failed, &g_status);
        if (lane == 0) {
          segs[i] = Seg{end ? -1 : sc.s, sc.h, sc.rt * kUnitRows, sc.first, sc.rows,
                        sc.len - sc.count, sc.len, j0, j1, slot};
          mbar_arrive(smem_u32(&bars.seg_full[i]));
        }
        __syncwarp();
        ++n;
      };
      const AttnUnit split = hand_out(a, sc, lane, s_span, s_load, s_order, emit);
      emit(true, 0, 0, -1);
      if (a.splits != nullptr && lane == 0) a.splits[blockIdx.x] = split;
    } else if (warp == kTmaWarp) {
      // --------------------------------------------------------- producer
      const int page_rows = min(1 << a.c.page_shift, kTile);
      const int boxes = kTile / page_rows;  // per tile, at most 8
      const int beyond = (a.c.n_pages * a.c.n_kv) << a.c.page_shift;  // a row outside the tensor
      int issued = 0;
      bool ok = true;
      for (int ns = 0; ok; ++ns) {
        const Seg g = next_seg(ns);
        if (g.s < 0) break;
        const int tiles = max(tiles_in(g, 0), tiles_in(g, 1));
        auto page_at = [&](int j) {  // this lane's box of tile j
          const int e = (g.j0 + j) * kTile + lane * page_rows;
          return lane < boxes && e < g.len ? raw_page(a.c, g.s, e) : 0;
        };
        int next = tiles > 0 ? page_at(0) : 0;
        for (int j = 0; j < tiles && ok; ++j) {
          const int e = (g.j0 + j) * kTile + lane * page_rows, p = good_page(a.c, next, a.err);
          const int row = p < 0 || e >= g.len ? beyond : static_cast<int>(cache_row(a.c, p, g.h, e));
          if (j + 1 < tiles) next = page_at(j + 1);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int slot = issued % Sh::kSlots, use = issued / Sh::kSlots;
            if (use > 0 && ok) ok = warp_wait(smem_u32(&bars.empty[slot]), (use - 1) & 1, &g_status);
            if (!ok) break;
            const uint32_t full = smem_u32(&bars.full[slot]);
            if (lane == 0) mbar_arrive_expect_tx(full, Sh::kSlotBytes);
            __syncwarp();
            ++issued;
            if (lane < boxes) {
              const uint32_t dst = smem_u32(ring + slot * Sh::kSlotBytes) + lane * page_rows * 128;
#pragma unroll
              for (int c = 0; c < Sh::kHalves; ++c)
                tc::tma_2d(dst + c * (kTile * 128), w == 0 ? &k_map : &v_map, c * 64, row, full);
            }
            __syncwarp();
          }
        }
      }
      // no copy may be in flight when the block ends
      for (int n = max(0, issued - Sh::kSlots); n < issued; ++n)
        warp_wait(smem_u32(&bars.full[n % Sh::kSlots]), (n / Sh::kSlots) & 1, &g_status);
    } else if (warp == kMmaWarp) {
      // --------------------------------------------------------- products
      const uint32_t tm = static_cast<uint32_t>(tc::uniform(static_cast<int>(tmem)));
      int item = 0;              // slots of the ring taken so far
      int n_p[2] = {0, 0};       // tiles of weights awaited so far
      int n_q[2] = {0, 0};       // queries awaited so far
      auto slot_of = [&](int n) { return smem_u32(ring + (n % Sh::kSlots) * Sh::kSlotBytes); };
      auto wait_full = [&](int n) {
        step_wait(smem_u32(&bars.full[n % Sh::kSlots]), (n / Sh::kSlots) & 1, &s_failed, &g_status);
      };
      auto release = [&](int n) { tc::commit(smem_u32(&bars.empty[n % Sh::kSlots])); };
      auto scores = [&](int x, int n) {  // with the keys in item n
        if (tc::elect_one()) {
          const uint64_t q = tc::desc_k_major(smem_u32(base + x * Sh::kSlotBytes));
          const uint64_t k = tc::desc_k_major(slot_of(n));
#pragma unroll
          for (int i = 0; i < HD / 16; ++i) {
            const int step = (i / 4) * (kTile * 128) + (i % 4) * 32;
            tc::mma_ss(tm + x * kTile, q + (step >> 4), k + (step >> 4), Sh::kDescS, i > 0);
          }
          tc::commit(smem_u32(&bars.s_full[x]));
        }
        __syncwarp();
      };
      for (int ns = 0;; ++ns) {
        const Seg g = next_seg(ns);
        if (g.s < 0) break;
        const int n_of[2] = {tc::uniform(tiles_in(g, 0)), tc::uniform(tiles_in(g, 1))};
        const int n_tiles = max(n_of[0], n_of[1]);
        const int tail = tc::uniform(g.len - g.j0 * kTile);  // entries from the segment's start on
        for (int x = 0; x < 2; ++x)
          if (n_of[x] > 0) {
            step_wait(smem_u32(&bars.q_full[x]), n_q[x] & 1, &s_failed, &g_status);
            ++n_q[x];
          }
        tc::fence_after();
        if (n_tiles > 0) {
          wait_full(item);
          if (n_of[0] > 0) scores(0, item);
          if (n_of[1] > 0) scores(1, item);
          if (tc::elect_one()) release(item);
          __syncwarp();
        }
        for (int j = 0; j < n_tiles; ++j, item += 2) {
          wait_full(item + 1);
          if (tail < (j + 1) * kTile) {
            // the rest of the last page may hold anything
            const int ps = 1 << a.c.page_shift;
            const int from = tail - j * kTile, to = min(kTile, (from + ps - 1) / ps * ps);
            uint8_t* v = ring + ((item + 1) % Sh::kSlots) * Sh::kSlotBytes;
            for (int c = lane; c < (to - from) * 8 * Sh::kHalves; c += 32) {
              const int r = from + c / (8 * Sh::kHalves), ch = c % (8 * Sh::kHalves);
              *reinterpret_cast<uint4*>(v + (ch >> 3) * (kTile * 128) + r * 128 + (ch & 7) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
            }
            tc::fence_async_shared();
            __syncwarp();
          }
          if (j + 1 < n_tiles) wait_full(item + 2);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (j < n_of[x]) {
              step_wait(smem_u32(&bars.p_full[x]), n_p[x] & 1, &s_failed, &g_status);
              ++n_p[x];
              tc::fence_after();
              if (tc::elect_one()) {
                const uint64_t v = tc::desc_mn_major(slot_of(item + 1), kTile * 128);
#pragma unroll
                for (int i = 0; i < kTile / 16; ++i)
                  tc::mma_ts(tm + 2 * kTile + x * HD, tm + x * kTile + i * 8, v + (i * 2048 >> 4),
                             Sh::kDescO, j > 0 || i > 0);
                if (j == n_of[x] - 1) tc::commit(smem_u32(&bars.o_full[x]));
              }
              __syncwarp();
            }
            if (x == 1 && tc::elect_one()) release(item + 1);
            __syncwarp();
            if (j + 1 < n_of[x]) scores(x, item + 2);
          }
          if (j + 1 < n_tiles && tc::elect_one()) release(item + 2);
          __syncwarp();
        }
      }
      // every product is done before tensor memory goes back
      if (tc::elect_one()) tc::commit(smem_u32(&bars.drain));
      __syncwarp();
      warp_wait(smem_u32(&bars.drain), 0, &g_status);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    // ----------------------------------------------------------- softmax
    const int x = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + ((warp & 3) << 21);  // 32 lanes per warp, lane in bits 16..
    const uint32_t st = lanes + x * kTile, ot = lanes + 2 * kTile + x * HD;
    // Queries of a segment into the swizzled operand layout: [column of 128
    // bytes][row][128 B], asynchronously (once every product with the ones before is
    // done: the last tile's scores are there).  A segment in which this tile sees
    // nothing has none: nothing would hold its arrival back until the one before has
    // been seen.
    auto wants_q = [&](const Seg& g) { return g.s >= 0 && tiles_in(g, x) > 0; };
    auto load_q = [&](const Seg& g) {
      const uint32_t qs = smem_u32(base + x * Sh::kSlotBytes);
#pragma unroll 4
      for (int k = 0; k < kTile * (HD / 8) / 128; ++k) {
        const int c = k * 128 + (threadIdx.x & 127);
        const int row = c / (HD / 8), ch = c % (HD / 8), rr = g.r0 + x * kTile + row;
        const bool take = rr < g.rows;
        const int i = take ? div_group(a, rr) : 0;
        cp_async16(qs + (ch >> 3) * (kTile * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4),
                   a.q + static_cast<long long>(g.first + i) * a.q_stride +
                       (g.h * a.group + (take ? rr - i * a.group : 0)) * HD + ch * 8,
                   take);
      }
      cp_commit();
    };
    auto q_loaded = [&] {
      cp_wait<0>();
      tc::fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.q_full[x]));
    };
    int n_s = 0, n_o = 0;  // tiles of scores, outputs awaited so far
    Seg g = next_seg(0);
    if (wants_q(g)) {
      load_q(g);
      q_loaded();
    }
    for (int ns = 1; g.s >= 0; ++ns) {
      const int rr = g.r0 + x * kTile + r;
      const bool live = rr < g.rows;
      const int i = live ? div_group(a, rr) : 0;
      const int lim = live ? g.off + i : -1;
      const int tiles = tiles_in(g, x);
      auto page_at = [&](int j) {  // lane b: page of entries 16b.. of tile j
        const int e = (g.j0 + j) * kTile + lane * 16;
        return lane < kTile / 16 && e < g.len ? raw_page(a.c, g.s, e) : 0;
      };
      float m = -INFINITY, l = 0.f;
      int page_next = tiles > 0 ? page_at(0) : 0;
      for (int j = 0; j < tiles; ++j, ++n_s) {
        const unsigned bad = __ballot_sync(0xFFFFFFFFu, good_page(a.c, page_next, nullptr) < 0);
        if (j + 1 < tiles) page_next = page_at(j + 1);
        step_wait(smem_u32(&bars.s_full[x]), n_s & 1, &s_failed, &g_status);
        tc::fence_after();
        if (j == tiles - 1) {
          const Seg after = look_seg(ns);
          if (wants_q(after)) load_q(after);
        }
        uint32_t v[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::ld32(v + 32 * c, st + 32 * c);
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::wait_ld32(v + 32 * c);
        const int hide = lim - (g.j0 + j) * kTile;  // entries above this one are hidden
        if (__any_sync(0xFFFFFFFFu, hide < kTile - 1)) {
#pragma unroll
          for (int k = 0; k < 128; ++k)
            if (k > hide) v[k] = 0xFF800000u;
        }
        if (bad != 0) {
#pragma unroll
          for (int k = 0; k < 128; ++k)
            if ((bad >> (k / 16)) & 1) v[k] = 0xFF800000u;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 128; k += 2)
          mx[(k / 2) & 3] = max3(mx[(k / 2) & 3], __uint_as_float(v[k]), __uint_as_float(v[k + 1]));
        const float most = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        // a row that grows past the top (or from nothing, -inf) is rescaled
        if (__any_sync(0xFFFFFFFFu, fmaf(most, a.scale_log2, -m) > kTop)) {
          const float mn = fmaxf(m, base_of(most * a.scale_log2));
          const float f = mn == m ? 1.f : ex2(m - mn);
          m = mn;
          l *= f;
          if (j > 0) {
#pragma unroll
            for (int c = 0; c < HD; c += 16) {
              uint32_t o[16];
              tc::ld16(o, ot + c);
              tc::wait_ld16(o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tc::st16(ot + c, o);
            }
          }
        }
        const float b = m == -INFINITY ? 0.f : m;
        uint64_t sum[2] = {0, 0};
        const uint64_t scale = pair(a.scale_log2, a.scale_log2), less = pair(-b, -b);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t p[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int n = 32 * c + 2 * k;
            const float2 x = unpair(fma2(pair(__uint_as_float(v[n]), __uint_as_float(v[n + 1])), scale, less));
            const float y0 = ex2(x.x), y1 = ex2(x.y);
            sum[k & 1] = add2(sum[k & 1], pair(y0, y1));
            p[k] = pack_f16(y0, y1);
          }
          tc::st16(st + 16 * c, p);
        }
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.p_full[x]));
        const float2 s2 = unpair(add2(sum[0], sum[1]));
        l += s2.x + s2.y;
      }
      const Seg after = next_seg(ns);
      if (wants_q(after)) {
        if (tiles == 0) load_q(after);
        q_loaded();
      }

      if (tiles > 0) {
        step_wait(smem_u32(&bars.o_full[x]), n_o & 1, &s_failed, &g_status);
        ++n_o;
      }
      tc::fence_after();
      const bool ok = __all_sync(0xFFFFFFFFu, *static_cast<volatile int*>(&s_failed) == 0);
      const int t = g.first + i, head = g.h * a.group + (live ? rr - i * a.group : 0);
      if (ok && g.slot >= 0) {
        const long long at = static_cast<long long>(g.slot) * kUnitRows + x * kTile + r;
        const bool wide = (reinterpret_cast<uintptr_t>(a.part_o) & 31) == 0;
#pragma unroll
        for (int c = 0; c < HD; c += 32) {
          uint32_t o[32];
          if (tiles > 0) {
            tc::ld32(o, ot + c);
            tc::wait_ld32(o);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0u;
          }
          if (live)
#pragma unroll
            for (int k = 0; k < 32; k += 8) store32(a.part_o + at * HD + c + k, o + k, wide);
        }
        if (live) a.part_ml[at] = make_float2(m, l);
      } else if (ok) {
        const float inv = l > 0.f || !(l == l) ? 1.0f / l : 0.f;
        bool odd = false;
        __half* y = a.out + static_cast<long long>(t) * a.out_stride + head * HD;
        const bool wide = (reinterpret_cast<uintptr_t>(y) & 31) == 0;
#pragma unroll
        for (int c = 0; c < HD; c += 32) {
          uint32_t o[32];
          if (tiles > 0) {
            tc::ld32(o, ot + c);
            tc::wait_ld32(o);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0u;
          }
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float u = __uint_as_float(o[2 * k]) * inv, v = __uint_as_float(o[2 * k + 1]) * inv;
            odd |= !(fabsf(u) <= 3.0e38f) || !(fabsf(v) <= 3.0e38f);
            w[k] = pack_f16(u, v);
          }
          if (live) {
            store32(y + c, w, wide);
            store32(y + c + 16, w + 8, wide);
          }
        }
        if (live && a.lse != nullptr)
          a.lse[static_cast<long long>(t) * a.n_q + head] = (m + log2f(l)) * kLn2;
        // rows that hide entries and came out infinite or NaN: again, without them
        unsigned again = __ballot_sync(0xFFFFFFFFu, live && odd && l == l && lim < g.len - 1);
        while (again != 0) {
          const int src = __ffs(again) - 1;
          again &= again - 1;
          const int tt = __shfl_sync(0xFFFFFFFFu, t, src), hh = __shfl_sync(0xFFFFFFFFu, head, src);
          const int ll = __shfl_sync(0xFFFFFFFFu, lim, src);
          __syncwarp();
          slow_row<HD>(a, g.s, g.h, tt, hh, ll, lane);
        }
      }
      // (the next segment's first product into O waits for weights that these
      // warps have yet to write)
      tc::fence_before();
      g = after;
    }
    cp_wait<0>();  // (nothing is in flight here unless a wait ran out)
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

// Join the parts of split units: block c of the kernel above has the first part
// of at most one (in its slot 1), the blocks behind it the others (in their
// slots 0).  A warp per row.  Bound by the way to the parts and back: 64 tokens over
// 30000 entries (8 units in 19 parts) take 38 us without it, 70 with 4 blocks to a
// unit, 55 with 8 and 16-byte loads; where no unit is cut (92 us for prompts) 8 blocks
// cost 1 us more than 4.
constexpr int kJoinRows = 16, kJoinBlocks = 8;  // rows at a time, blocks per unit

template <int HD>
__global__ void __launch_bounds__(32 * kJoinRows) attention_join_units_kernel(const AttnArgs a) {
  constexpr int D = HD / 32, kU = 4;
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x / kJoinBlocks, lane = threadIdx.x & 31;
  const AttnUnit u = a.splits[c];
  if (u.parts == 0) return;
  for (int r = blockIdx.x % kJoinBlocks * kJoinRows + (threadIdx.x >> 5); r < kUnitRows;
       r += kJoinBlocks * kJoinRows) {
    const int rr = u.r0 + r;
    if (rr >= u.rows) return;
    float m = -INFINITY, l = 0.f, acc[D] = {};
    for (int p0 = 0; p0 < u.parts; p0 += kU) {
      float2 ml[kU];
      float o[kU][D];
#pragma unroll
      for (int k = 0; k < kU; ++k) {
        const int p = p0 + k;
        ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int d = 0; d < D; ++d) o[k][d] = 0.f;
        if (p < u.parts) {
          const long long at = static_cast<long long>(p == 0 ? 2 * c + 1 : 2 * (c + p)) * kUnitRows + r;
          ml[k] = a.part_ml[at];
          const float* src = a.part_o + at * HD + lane * D;
          if constexpr (D == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            o[k][0] = v.x, o[k][1] = v.y, o[k][2] = v.z, o[k][3] = v.w;
          } else {
            const float2 v = *reinterpret_cast<const float2*>(src);
            o[k][0] = v.x, o[k][1] = v.y;
          }
        }
      }
      float mn = m;
#pragma unroll
      for (int k = 0; k < kU; ++k) mn = fmaxf(mn, ml[k].x);
      const float base = mn == -INFINITY ? 0.f : mn, f0 = ex2(m - base);
      l *= f0;
#pragma unroll
      for (int d = 0; d < D; ++d) acc[d] *= f0;
#pragma unroll
      for (int k = 0; k < kU; ++k) {
        const float f = ex2(ml[k].x - base);
        l += ml[k].y * f;
#pragma unroll
        for (int d = 0; d < D; ++d) acc[d] += o[k][d] * f;
      }
      m = mn;
    }
    const int i = rr / a.group;
    store_row<HD>(a, u.s, u.h, u.first + i, u.h * a.group + rr % a.group, min(u.off + i, u.len - 1),
                  u.len, acc, m, l, lane);
  }
}

template <typename F, typename... Args>
cudaError_t launch(F* k, long long blocks, int threads, int smem, cudaStream_t st, Args... args) {
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

template <int HD>
cudaError_t launch_many(AttnArgs a, int sms, cudaStream_t st, int device, void* workspace,
                        size_t bytes) {
  static std::atomic<unsigned long long> done{0};
  auto* k = attention_many_kernel<HD>;
  const unsigned long long bit = 1ull << (device & 63);
  if (!(done.load(std::memory_order_relaxed) & bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<HD>::kSmem);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_relaxed);
  }
  CUtensorMap km, vm;
  if (!encode_pool(&km, a.c, a.c.k) || !encode_pool(&vm, a.c, a.c.v)) return cudaErrorInvalidValue;
  a.splits = nullptr;
  if (bytes >= attention_many_bytes(HD, sms)) {  // outputs, {max, sum}, what the join needs
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + 2LL * sms * kUnitRows * HD);
    a.splits = reinterpret_cast<AttnUnit*>(a.part_ml + 2LL * sms * kUnitRows);
  }
  const cudaError_t e = launch(k, sms, kThreads, Shape<HD>::kSmem, st, a, km, vm);
  if (e != cudaSuccess || a.splits == nullptr) return e;
  return launch(attention_join_units_kernel<HD>, static_cast<long long>(sms) * kJoinBlocks,
                32 * kJoinRows, 0, st, a);
}

}  // namespace

size_t attention_many_bytes(int head_dim, int sms) {
  if (sms > kMaxBlocks) sms = kMaxBlocks;
  return static_cast<size_t>(sms) * (2 * kUnitRows * (static_cast<size_t>(head_dim) * 4 + 8) +
                                     sizeof(AttnUnit));
}

cudaError_t attention_many_launch(const AttnArgs& a, int sms, cudaStream_t st, int device,
                                  void* workspace, size_t bytes) {
  if (sms > kMaxBlocks) sms = kMaxBlocks;
  return a.c.head_dim == 64 ? launch_many<64>(a, sms, st, device, workspace, bytes)
                            : launch_many<128>(a, sms, st, device, workspace, bytes);
}

cudaError_t status_attention(unsigned* out) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_status, sizeof(v));
  if (e != cudaSuccess) return e;
  e = cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
  *out |= v;
  return e;
}

}  // namespace qgemv
