// attention_many.cu -- qgemv_paged_attention for many query rows per
// key/value head (prompts, chunks of prompts): tcgen05 products, TMA loads.
//
// A thread block takes 256 rows (two tiles of 128, A and B) of one (sequence,
// key/value head) and walks the cache in tiles of 128 entries:
//   warp 9      producer: K and V tiles by TMA, page by page, into a ring of
//               128-byte-swizzled slots (keys and values alternate);
//   warp 8      issues the products: S = Q K^T (operands in shared memory) and
//               O += P V (P in tensor memory, V as the transposed operand);
//   warps 0-3   softmax of tile A, warps 4-7 of tile B: one row per thread,
//               read from tensor memory, weights written back as fp16 over the
//               scores they came from.
// While one tile's weights are computed the tensor core works on the other's
// products.  Tensor memory: S/P of A and B (128 columns each), O of A and B
// (HD each).
//
// The running maximum is lazy: the weights are taken relative to an older
// maximum until the new one exceeds it by 2^kSlack, so O is rescaled (a round
// trip through tensor memory) a few times per row instead of at every tile.
// Weights are then at most 2^kSlack, far inside fp16; their relative rounding is
// the same as below 1.
//
// Entries behind the sequence or on bad pages are loaded as zeros (a TMA box
// outside the tensor); the rows of the last page behind the sequence's end,
// which may hold anything, are zeroed in the V tile before the product.
#include <atomic>

#include "attention_common.cuh"
#include "tcgen05.cuh"
#include "kv_tensor_map.h"

namespace qgemv {
namespace {

__device__ unsigned g_status = 0;

constexpr int kTile = 128;           // rows of a tile, entries of a step
// Three warpgroups; the launch gives 168 registers a thread (64,512), of which
// the third group passes on what the two of the softmax need: 256 x 200 + 128 x
// 104 = 64,512.
constexpr int kThreads = 384;
constexpr int kMmaWarp = 8, kTmaWarp = 9;
constexpr float kSlack = 8.0f;       // log2 of the growth that makes O be rescaled

template <int HD>
struct Shape {
  static constexpr int kHalves = HD / 64;                 // 128-byte columns of a row
  static constexpr int kSlotBytes = kTile * HD * 2;
  static constexpr int kSlots = HD == 128 ? 5 : 10;
  static constexpr int kSmem = 1024 + (2 + kSlots) * kSlotBytes;
  static_assert(kSmem + 1024 <= 227 * 1024, "dynamic and static shared memory");
  static constexpr uint32_t kDescS = tc::idesc_f16(kTile, kTile, false);
  static constexpr uint32_t kDescO = tc::idesc_f16(kTile, HD, true);
};

struct Bars {
  uint64_t full[10], empty[10];
  uint64_t s_full[2], p_full[2], o_full[2], drain;
};

// (sequence, row tile) of block unit u: sequences in order, each with
// ceil(rows / 256) units, the last (longest) first.  s = -1 behind the end.
__device__ __forceinline__ void find_unit(const AttnArgs& a, int u, int lane, int* s_out, int* rt) {
  *s_out = -1;
  *rt = 0;
  for (int s0 = 0; s0 < a.c.n_seqs; s0 += 32) {
    const int s = s0 + lane;
    int first = 0, count = 0;
    if (s < a.c.n_seqs) seq_rows(a.q_start, s, a.n_tokens, a.err, &first, &count);
    if (count > a.max_q) flag_error(a.err);
    const int mine = (min(count, a.max_q) * a.group + 2 * kTile - 1) / (2 * kTile);
    int incl = mine;
#pragma unroll
    for (int k = 1; k < 32; k *= 2) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, incl, k);
      if (lane >= k) incl += v;
    }
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, u < incl);
    if (hit != 0) {
      const int l = __ffs(hit) - 1;
      const int end = __shfl_sync(0xFFFFFFFFu, incl, l);
      *s_out = s0 + l;
      *rt = end - 1 - u;
      return;
    }
    u -= __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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
  __shared__ int s_unit[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint8_t* ring = base + 2 * Sh::kSlotBytes;

  pdl_launch_dependents();
  if (warp == kMmaWarp) {
    if (lane == 0) {
      for (int i = 0; i < Sh::kSlots; ++i) {
        mbar_init(smem_u32(&bars.full[i]), 1);
        mbar_init(smem_u32(&bars.empty[i]), 1);
      }
      for (int x = 0; x < 2; ++x) {
        mbar_init(smem_u32(&bars.s_full[x]), 1);
        mbar_init(smem_u32(&bars.p_full[x]), 4);  // one arrival per warp
        mbar_init(smem_u32(&bars.o_full[x]), 1);
      }
      mbar_init(smem_u32(&bars.drain), 1);
      fence_mbar_init();
      s_failed = 0;
    }
    __syncwarp();
  }
  pdl_wait();
  if (warp == kTmaWarp) {
    int s, rt;
    find_unit(a, static_cast<int>(blockIdx.x / (a.n_parts * a.c.n_kv)), lane, &s, &rt);
    if (lane == 0) {
      s_unit[0] = s;
      s_unit[1] = rt;
    }
  }
  __syncthreads();
  const int s = s_unit[0];
  if (s < 0) return;
  const int sp = blockIdx.x % a.n_parts, h = blockIdx.x / a.n_parts % a.c.n_kv;
  int first, count;
  seq_rows(a.q_start, s, a.n_tokens, nullptr, &first, &count);
  const int rows = min(count, a.max_q) * a.group;
  const int r0 = s_unit[1] * 2 * kTile;
  const int len = seq_len(a.c, s, a.err);
  const int off = len - count;
  const int k0 = sp * a.part;
  if (sp > 0 && k0 >= len) return;
  // tiles of entries that tile x sees (its last row sees the most)
  int nt[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int last = min(rows, r0 + (x + 1) * kTile) - 1;
    const int see = last >= r0 + x * kTile ? min(min(len, off + last / a.group + 1), k0 + a.part) : 0;
    nt[x] = see > k0 ? (see - k0 + kTile - 1) / kTile : 0;
  }
  const int tiles = max(nt[0], nt[1]);
  const bool has_b = r0 + kTile < rows;

  if (warp == kMmaWarp) {
    tc::alloc(smem_u32(&s_tmem), 512);
  } else if (warp < 8 && tiles > 0) {
    // Queries into the swizzled operand layout: [column of 128 bytes][row][128 B].
    const int x = warp >> 2;
    uint8_t* qs = base + x * Sh::kSlotBytes;
    if (x == 0 || has_b)
      for (int c = threadIdx.x & 127; c < kTile * (HD / 8); c += 128) {
        const int r = c / (HD / 8), ch = c % (HD / 8), rr = r0 + x * kTile + r;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (rr < rows)
          v = *reinterpret_cast<const uint4*>(
              a.q + static_cast<long long>(first + rr / a.group) * a.q_stride +
              (h * a.group + rr % a.group) * HD + ch * 8);
        *reinterpret_cast<uint4*>(qs + (ch >> 3) * (kTile * 128) + r * 128 +
                                  (((ch & 7) ^ (r & 7)) << 4)) = v;
      }
    tc::fence_async_shared();
  }
  // (the producer starts at once)
  tc::fence_before();
  if (warp <= kMmaWarp) named_bar_sync(1, 32 * (kMmaWarp + 1));
  tc::fence_after();
  const uint32_t tmem = s_tmem;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
  if (warp == kTmaWarp) {
    // ---------------------------------------------------------- producer
    const int page_rows = min(1 << a.c.page_shift, kTile);
    const int boxes = kTile / page_rows;  // per tile, at most 8
    const int beyond = (a.c.n_pages * a.c.n_kv) << a.c.page_shift;  // a row outside the tensor
    auto page_at = [&](int j) {  // this lane's box of tile j
      const int e = k0 + j * kTile + lane * page_rows;
      return lane < boxes && e < len ? raw_page(a.c, s, e) : 0;
    };
    int next = tiles > 0 ? page_at(0) : 0, issued = 0;
    for (int j = 0; j < tiles; ++j) {
      const int e = k0 + j * kTile + lane * page_rows, p = good_page(a.c, next, a.err);
      const int row = p < 0 || e >= len ? beyond : static_cast<int>(cache_row(a.c, p, h, e));
      if (j + 1 < tiles) next = page_at(j + 1);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int n = 2 * j + w, slot = n % Sh::kSlots, use = n / Sh::kSlots;
        if (use > 0 && !warp_wait(smem_u32(&bars.empty[slot]), (use - 1) & 1, &g_status)) {
          j = tiles;  // no more copies
          break;
        }
        const uint32_t full = smem_u32(&bars.full[slot]);
        if (lane == 0) mbar_arrive_expect_tx(full, Sh::kSlotBytes);
        __syncwarp();
        issued = n + 1;
        if (lane < boxes) {
          const uint32_t dst = smem_u32(ring + slot * Sh::kSlotBytes) + lane * page_rows * 128;
#pragma unroll
          for (int c = 0; c < Sh::kHalves; ++c)
            tc::tma_2d(dst + c * (kTile * 128), w == 0 ? &k_map : &v_map, c * 64, row, full);
        }
        __syncwarp();
      }
    }
    // no copy may be in flight when the block ends
    for (int n = max(0, issued - Sh::kSlots); n < issued; ++n)
      warp_wait(smem_u32(&bars.full[n % Sh::kSlots]), (n / Sh::kSlots) & 1, &g_status);
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------- products
    const uint32_t tm = static_cast<uint32_t>(tc::uniform(static_cast<int>(tmem)));
    const int n_tiles = tc::uniform(tiles), n_of[2] = {tc::uniform(nt[0]), tc::uniform(nt[1])};
    const int tail = tc::uniform(len - k0);
    auto slot_of = [&](int n) { return smem_u32(ring + (n % Sh::kSlots) * Sh::kSlotBytes); };
    auto wait_full = [&](int n) {
      step_wait(smem_u32(&bars.full[n % Sh::kSlots]), (n / Sh::kSlots) & 1, &s_failed, &g_status);
    };
    auto release = [&](int n) { tc::commit(smem_u32(&bars.empty[n % Sh::kSlots])); };
    auto scores = [&](int x, int j) {
      if (tc::elect_one()) {
        const uint64_t q = tc::desc_k_major(smem_u32(base + x * Sh::kSlotBytes));
        const uint64_t k = tc::desc_k_major(slot_of(2 * j));
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) {
          const int step = (i / 4) * (kTile * 128) + (i % 4) * 32;
          tc::mma_ss(tm + x * kTile, q + (step >> 4), k + (step >> 4), Sh::kDescS, i > 0);
        }
        tc::commit(smem_u32(&bars.s_full[x]));
      }
      __syncwarp();
    };
    if (n_tiles > 0) {
      wait_full(0);
      if (n_of[0] > 0) scores(0, 0);
      if (n_of[1] > 0) scores(1, 0);
      if (tc::elect_one()) release(0);
    }
    for (int j = 0; j < n_tiles; ++j) {
      wait_full(2 * j + 1);
      if (tail < (j + 1) * kTile) {
        // the rest of the last page may hold anything
        const int ps = 1 << a.c.page_shift;
        const int from = tail - j * kTile, to = min(kTile, (from + ps - 1) / ps * ps);
        uint8_t* v = ring + ((2 * j + 1) % Sh::kSlots) * Sh::kSlotBytes;
        for (int c = lane; c < (to - from) * 8 * Sh::kHalves; c += 32) {
          const int r = from + c / (8 * Sh::kHalves), ch = c % (8 * Sh::kHalves);
          *reinterpret_cast<uint4*>(v + (ch >> 3) * (kTile * 128) + r * 128 + (ch & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        }
        tc::fence_async_shared();
        __syncwarp();
      }
      if (j + 1 < n_tiles) wait_full(2 * j + 2);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (j < n_of[x]) {
          step_wait(smem_u32(&bars.p_full[x]), j & 1, &s_failed, &g_status);
          tc::fence_after();
          if (tc::elect_one()) {
            const uint64_t v = tc::desc_mn_major(slot_of(2 * j + 1), kTile * 128);
#pragma unroll
            for (int i = 0; i < kTile / 16; ++i)
              tc::mma_ts(tm + 2 * kTile + x * HD, tm + x * kTile + i * 8, v + (i * 2048 >> 4),
                         Sh::kDescO, j > 0 || i > 0);
            if (j == n_of[x] - 1) tc::commit(smem_u32(&bars.o_full[x]));
          }
          __syncwarp();
        }
        if (x == 1 && tc::elect_one()) release(2 * j + 1);
        __syncwarp();
        if (j + 1 < n_of[x]) scores(x, j + 1);
      }
      if (j + 1 < n_tiles && tc::elect_one()) release(2 * j + 2);
      __syncwarp();
    }
    // every product is done before tensor memory goes back
    if (tc::elect_one()) tc::commit(smem_u32(&bars.drain));
    __syncwarp();
    warp_wait(smem_u32(&bars.drain), 0, &g_status);
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ----------------------------------------------------------- softmax
    const int x = warp >> 2, r = (warp & 3) * 32 + lane, rr = r0 + x * kTile + r;
    const bool live = rr < rows;
    const int i = live ? rr / a.group : 0;
    const int lim = live ? off + i : -1;
    const uint32_t lanes = tmem + ((warp & 3) << 21);  // 32 lanes per warp, lane in bits 16..
    const uint32_t st = lanes + x * kTile, ot = lanes + 2 * kTile + x * HD;
    auto page_at = [&](int j) {  // lane b: page of entries 16b.. of tile j
      const int e = k0 + j * kTile + lane * 16;
      return lane < kTile / 16 && e < len ? raw_page(a.c, s, e) : 0;
    };
    float m = -INFINITY, l = 0.f;
    int page_next = nt[x] > 0 ? page_at(0) : 0;
    for (int j = 0; j < nt[x]; ++j) {
      const unsigned bad = __ballot_sync(0xFFFFFFFFu, good_page(a.c, page_next, nullptr) < 0);
      if (j + 1 < nt[x]) page_next = page_at(j + 1);
      step_wait(smem_u32(&bars.s_full[x]), j & 1, &s_failed, &g_status);
      tc::fence_after();
      uint32_t v[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::ld32(v + 32 * c, st + 32 * c);
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::wait_ld32(v + 32 * c);
      const int hide = lim - (k0 + j * kTile);  // entries above this one are hidden
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
      const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
      // a row that grows past the slack (or from nothing) is rescaled
      if (__any_sync(0xFFFFFFFFu, mt > m + kSlack)) {
        const float mn = fmaxf(m, mt);
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
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t p[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int n = 32 * c + 2 * k;
          const float x0 = ex2(fmaf(__uint_as_float(v[n]), a.scale_log2, -b));
          const float x1 = ex2(fmaf(__uint_as_float(v[n + 1]), a.scale_log2, -b));
          sum[n & 3] += x0;
          sum[(n + 1) & 3] += x1;
          p[k] = pack_f16(x0, x1);
        }
        tc::st16(st + 16 * c, p);
      }
      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.p_full[x]));
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    }
    if (nt[x] > 0) step_wait(smem_u32(&bars.o_full[x]), 0, &s_failed, &g_status);
    const bool ok = __all_sync(0xFFFFFFFFu, *static_cast<volatile int*>(&s_failed) == 0);
    tc::fence_after();
    const int t = first + i, head = h * a.group + (live ? rr % a.group : 0);
    const long long at = static_cast<long long>(t) * a.n_q + head;
    if (ok && a.n_parts > 1) {
      float* po = a.part_o + (static_cast<long long>(sp) * a.n_tokens * a.n_q + at) * HD;
#pragma unroll
      for (int c = 0; c < HD; c += 32) {
        uint32_t o[32];
        if (nt[x] > 0) {
          tc::ld32(o, ot + c);
          tc::wait_ld32(o);
        }
        if (live)
#pragma unroll
          for (int k = 0; k < 32; k += 4)
            *reinterpret_cast<uint4*>(po + c + k) =
                nt[x] > 0 ? make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]) : make_uint4(0, 0, 0, 0);
      }
      if (live) a.part_ml[static_cast<long long>(sp) * a.n_tokens * a.n_q + at] = make_float2(m, l);
    } else if (ok) {
      const float inv = l > 0.f || !(l == l) ? 1.0f / l : 0.f;
      bool odd = false;
      __half* y = a.out + static_cast<long long>(t) * a.out_stride + head * HD;
#pragma unroll
      for (int c = 0; c < HD; c += 32) {
        uint32_t o[32];
        if (nt[x] > 0) {
          tc::ld32(o, ot + c);
          tc::wait_ld32(o);
        }
#pragma unroll
        for (int k = 0; k < 32; k += 8) {
          float w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            w[e] = nt[x] > 0 ? __uint_as_float(o[k + e]) * inv : 0.f;
            odd |= !(fabsf(w[e]) <= 3.0e38f);
          }
          if (live)
            *reinterpret_cast<uint4*>(y + c + k) =
                make_uint4(pack_f16(w[0], w[1]), pack_f16(w[2], w[3]), pack_f16(w[4], w[5]),
                           pack_f16(w[6], w[7]));
        }
      }
      if (live && a.lse != nullptr) a.lse[at] = (m + log2f(l)) * kLn2;
      // rows that hide entries and came out infinite or NaN: again, without them
      unsigned again = __ballot_sync(0xFFFFFFFFu, live && odd && lim < len - 1);
      while (again != 0) {
        const int src = __ffs(again) - 1;
        again &= again - 1;
        const int tt = __shfl_sync(0xFFFFFFFFu, t, src), hh = __shfl_sync(0xFFFFFFFFu, head, src);
        const int ll = __shfl_sync(0xFFFFFFFFu, lim, src);
        __syncwarp();
        slow_row<HD>(a, s, h, tt, hh, ll, lane);
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

template <int HD>
cudaError_t launch_many(const AttnArgs& a, cudaStream_t st, int device) {
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
  const long long blocks =
      attention_many_units(a.c.n_seqs, a.n_tokens, a.group, a.max_q) * a.c.n_kv * a.n_parts;
  if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Shape<HD>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, a, km, vm);
}

}  // namespace

// Upper bound of the row tiles (256 rows) of all sequences: a sequence adds
// at most one that is not full.
long long attention_many_units(int n_seqs, int n_tokens, int group, int max_q) {
  const long long each = (static_cast<long long>(max_q) * group + 2 * kTile - 1) / (2 * kTile);
  const long long full = static_cast<long long>(n_tokens) * group / (2 * kTile);
  const long long part = n_seqs < n_tokens ? n_seqs : n_tokens;
  const long long bound = full + part;
  return each * n_seqs < bound ? each * n_seqs : bound;
}

// Parts of the cache: as many as fill the machine once (a block takes a whole
// multiprocessor), each of 512 entries at least.
AttnSplit attention_many_split(long long units, int n_kv, long long capacity, int sms) {
  const long long want = sms / (units * n_kv);
  if (want <= 1) return {1, static_cast<int>(capacity), 1};
  long long part = ((capacity + want - 1) / want + kTile - 1) / kTile * kTile;
  if (part < 512) part = 512;
  return {static_cast<int>((capacity + part - 1) / part), static_cast<int>(part), 1};
}

cudaError_t attention_many_launch(const AttnArgs& a, cudaStream_t st, int device) {
  return a.c.head_dim == 64 ? launch_many<64>(a, st, device) : launch_many<128>(a, st, device);
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
