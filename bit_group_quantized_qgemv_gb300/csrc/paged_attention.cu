// paged_attention.cu -- qgemv_paged_attention for few query rows per
// key/value head (decode steps, drafts): split over the cache, mma.sync.
//
// The rows of a (sequence, key/value head) are its new tokens times the query
// heads that share the head, row r = token r / group, head r % group.  A
// thread block takes MT * 16 of them and one part of the cache; its four
// warps take every fourth tile of 16 entries, each through a ring of its own
// (cp.async, no block-wide barrier until the end), so the loop is a stream of
// K and V through shared memory.  Per tile: S = Q K^T by m16n8k16, the
// running maximum and sum of the softmax in fp32 registers, P V with P
// straight from the accumulator registers as the next A operand.  The warps'
// (max, sum, O) are joined in shared memory, the parts of a split cache by a
// second kernel.
//
// P is split into fp16 high and low parts (two products with V), which
// keeps the weights at 22 bits; the tensor cores have the time, the kernel
// is bound by HBM.
#include <atomic>

#include "attention_common.cuh"

namespace qgemv {
namespace {

constexpr int kWarps = 4;
constexpr int kTile = 16;    // entries per warp and step
constexpr int kStages = 3;   // ring depth of each warp

template <int HD>
__host__ __device__ constexpr int stage_bytes() {
  return 2 * kTile * HD * 2;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
  const int n = take ? 16 : 0;  // 0: the 16 bytes are filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// Byte offset of 16-byte chunk ch of row r in a tile of HD-wide rows; the
// swizzle spreads 8 rows over the banks.
template <int HD>
__device__ __forceinline__ int tile_off(int r, int ch) {
  return r * (HD * 2) + ((ch ^ (r & 7)) << 4);
}

template <int HD, int MT>
__global__ void __launch_bounds__(32 * kWarps) attention_few_kernel(const AttnArgs a) {
  constexpr int kN = HD / 8;    // n-tiles of the output
  constexpr int kK = HD / 16;   // k-steps of the scores
  constexpr int kRows = 16 * MT;
  constexpr int kChunks = HD / 8;  // 16-byte chunks per row
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float sm_m[kWarps][kRows], sm_l[kWarps][kRows];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tq = lane & 3;

  long long b = blockIdx.x;
  const int sp = static_cast<int>(b % a.n_splits);
  b /= a.n_splits;
  const int h = static_cast<int>(b % a.c.n_kv);
  b /= a.c.n_kv;
  const int rt = static_cast<int>(b % a.row_tiles);
  const int s = static_cast<int>(b / a.row_tiles);

  int first, count;
  seq_rows(a.q_start, s, a.n_tokens, a.err, &first, &count);
  if (count > a.max_q) flag_error(a.err);
  const int rows = min(count, a.max_q) * a.group;
  const int r0 = rt * kRows;
  if (r0 >= rows) return;
  const int nr = min(kRows, rows - r0);
  const int len = seq_len(a.c, s, a.err);
  const int off = len - count;  // token i sees entries up to off + i
  const int per = part_len(len, a.n_splits, a.part_unit);
  const int k0 = sp * per;
  if (sp > 0 && k0 >= len) return;  // the join knows
  // entries that some row of this block sees
  const int see = min(len, off + (r0 + nr - 1) / a.group + 1);
  const int k1 = min(see, k0 + per);

  // Queries as A fragments.
  uint32_t qf[MT][kK][4];
  int lim[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = mt * 16 + g + 8 * e;
      const int i = (r0 + r) / a.group, head = h * a.group + (r0 + r) % a.group;
      lim[mt][e] = r < nr ? off + i : -1;
      const __half* q = a.q + static_cast<long long>(first + i) * a.q_stride + head * HD + 2 * tq;
#pragma unroll
      for (int k = 0; k < kK; ++k) {
        qf[mt][k][e] = r < nr ? *reinterpret_cast<const uint32_t*>(q + 16 * k) : 0u;
        qf[mt][k][2 + e] = r < nr ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 8) : 0u;
      }
    }

  float o[MT][kN][4], m[MT][2], l[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.f;
    m[mt][0] = m[mt][1] = -INFINITY;
    l[mt][0] = l[mt][1] = 0.f;
  }

  const uint32_t ring = smem_u32(smem) + warp * (kStages * stage_bytes<HD>());
  const int tiles = k1 > k0 ? (k1 - k0 + kTile - 1) / kTile : 0;
  const int mine = tiles > warp ? (tiles - warp + kWarps - 1) / kWarps : 0;
  unsigned bad = 0;  // bit st: the tile in stage st lies on a bad page
  int page = mine > 0 ? page_of(a.c, s, k0 + warp * kTile, a.err) : -1;

  auto issue = [&](int it) {
    if (it < mine) {
      const int e0 = k0 + (it * kWarps + warp) * kTile;
      const int st = it % kStages;
      const uint32_t kd = ring + st * stage_bytes<HD>(), vd = kd + stage_bytes<HD>() / 2;
      const long long base = page >= 0 ? cache_row(a.c, page, h, e0) * HD : 0;
      bad = page >= 0 ? bad & ~(1u << st) : bad | (1u << st);
#pragma unroll
      for (int c = 0; c < kTile * kChunks / 32; ++c) {
        const int id = c * 32 + lane, r = id / kChunks, ch = id % kChunks;
        const bool take = page >= 0 && e0 + r < len;
        const long long src = take ? base + r * HD + ch * 8 : 0;
        cp_async16(kd + tile_off<HD>(r, ch), a.c.k + src, take);
        cp_async16(vd + tile_off<HD>(r, ch), a.c.v + src, take);
      }
      // the next tile's page, a step ahead of its use
      if (it + 1 < mine) page = page_of(a.c, s, e0 + kWarps * kTile, a.err);
    }
    cp_commit();
  };
#pragma unroll
  for (int p = 0; p < kStages - 1; ++p) issue(p);

  for (int it = 0; it < mine; ++it) {
    cp_wait<kStages - 2>();
    __syncwarp();
    issue(it + kStages - 1);
    const int st = it % kStages;
    const int e0 = k0 + (it * kWarps + warp) * kTile;
    const uint32_t kd = ring + st * stage_bytes<HD>(), vd = kd + stage_bytes<HD>() / 2;
    float sc[MT][2][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[mt][n][e] = 0.f;
    const int lr = (lane & 7) + ((lane >> 4) << 3), lc = (lane >> 3) & 1;
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      uint32_t kf[4];  // b0, b1 of entries 0-7, then of entries 8-15
      ldsm4(kf, kd + tile_off<HD>(lr, 2 * k + lc));
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        mma_f16(sc[mt][0], qf[mt][k], kf[0], kf[1]);
        mma_f16(sc[mt][1], qf[mt][k], kf[2], kf[3]);
      }
    }
    const bool hidden = (bad >> st) & 1;
    uint32_t ph[MT][4], pl[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float mn[2] = {m[mt][0], m[mt][1]};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = e0 + n * 8 + 2 * tq + (e & 1);
          const bool seen = !hidden && j <= lim[mt][e >> 1] && j < len;
          sc[mt][n][e] = seen ? sc[mt][n][e] * a.scale_log2 : -INFINITY;
          mn[e >> 1] = fmaxf(mn[e >> 1], sc[mt][n][e]);
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mn[e] = fmaxf(mn[e], __shfl_xor_sync(0xFFFFFFFFu, mn[e], 1));
        mn[e] = fmaxf(mn[e], __shfl_xor_sync(0xFFFFFFFFu, mn[e], 2));
      }
      const bool grew = mn[0] > m[mt][0] || mn[1] > m[mt][1];
      if (__any_sync(0xFFFFFFFFu, grew)) {
        const float f0 = mn[0] == m[mt][0] ? 1.f : ex2(m[mt][0] - mn[0]);
        const float f1 = mn[1] == m[mt][1] ? 1.f : ex2(m[mt][1] - mn[1]);
        l[mt][0] *= f0;
        l[mt][1] *= f1;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          o[mt][n][0] *= f0;
          o[mt][n][1] *= f0;
          o[mt][n][2] *= f1;
          o[mt][n][3] *= f1;
        }
        m[mt][0] = mn[0];
        m[mt][1] = mn[1];
      }
      const float b0 = mn[0] == -INFINITY ? 0.f : mn[0], b1 = mn[1] == -INFINITY ? 0.f : mn[1];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const float base = e == 0 ? b0 : b1;
          const float x = ex2(sc[mt][n][e] - base), y = ex2(sc[mt][n][e + 1] - base);
          l[mt][e >> 1] += x + y;
          const uint32_t hi = pack_f16(x, y);
          const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&hi));
          ph[mt][2 * n + (e >> 1)] = hi;
          pl[mt][2 * n + (e >> 1)] = pack_f16(x - hf.x, y - hf.y);
        }
    }
    const int vr = (lane & 7) + (((lane >> 3) & 1) << 3), vc = lane >> 4;
#pragma unroll
    for (int n = 0; n < kN; n += 2) {
      uint32_t vf[4];  // b0, b1 of columns 8n.., then of 8n + 8..
      ldsm4t(vf, vd + tile_off<HD>(vr, n + vc));
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        mma_f16(o[mt][n], ph[mt], vf[0], vf[1]);
        mma_f16(o[mt][n + 1], ph[mt], vf[2], vf[3]);
        mma_f16(o[mt][n], pl[mt], vf[0], vf[1]);
        mma_f16(o[mt][n + 1], pl[mt], vf[2], vf[3]);
      }
    }
    __syncwarp();
  }
  cp_wait<0>();
  __syncthreads();  // every warp is done with its ring: it now takes the partial outputs
  float* so = reinterpret_cast<float*>(smem);  // [warp][row][HD]
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float lsum = l[mt][e];
      lsum += __shfl_xor_sync(0xFFFFFFFFu, lsum, 1);
      lsum += __shfl_xor_sync(0xFFFFFFFFu, lsum, 2);
      const int r = mt * 16 + g + 8 * e;
      if (tq == 0) {
        sm_m[warp][r] = m[mt][e];
        sm_l[warp][r] = lsum;
      }
#pragma unroll
      for (int n = 0; n < kN; ++n)
        *reinterpret_cast<float2*>(so + (warp * kRows + r) * HD + n * 8 + 2 * tq) =
            make_float2(o[mt][n][2 * e], o[mt][n][2 * e + 1]);
    }
  __syncthreads();
  // A warp per row: join the warps' parts.
  constexpr int D = HD / 32;
  for (int r = warp; r < nr; r += kWarps) {
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w][r]);
    const float base = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f, acc[D] = {};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2(sm_m[w][r] - base);
      ll += sm_l[w][r] * f;
#pragma unroll
      for (int d = 0; d < D; ++d) acc[d] += so[(w * kRows + r) * HD + lane * D + d] * f;
    }
    const int i = (r0 + r) / a.group, head = h * a.group + (r0 + r) % a.group, t = first + i;
    if (a.n_splits > 1) {
      const long long at = (static_cast<long long>(sp) * a.n_tokens + t) * a.n_q + head;
#pragma unroll
      for (int d = 0; d < D; ++d) a.part_o[at * HD + lane * D + d] = acc[d];
      if (lane == 0) a.part_ml[at] = make_float2(mm, ll);
      continue;
    }
    store_row<HD>(a, s, h, t, head, min(off + i, len - 1), len, acc, mm, ll, lane);
  }
}

// Join the parts of a split cache: a warp per (token, query head).
template <int HD>
__global__ void __launch_bounds__(128) attention_join_kernel(const AttnArgs a) {
  constexpr int D = HD / 32;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long id = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  // (sequence, token within it, head)
  const int head = static_cast<int>(id % a.n_q);
  const int i = static_cast<int>(id / a.n_q % a.max_q);
  const int s = static_cast<int>(id / a.n_q / a.max_q);
  if (s >= a.c.n_seqs) return;
  int first, count;
  seq_rows(a.q_start, s, a.n_tokens, nullptr, &first, &count);
  if (i >= count) return;
  const int t = first + i;
  const int len = seq_len(a.c, s, nullptr);
  const int per = part_len(len, a.n_splits, a.part_unit);
  const int parts = len > 0 ? (len + per - 1) / per : 1;
  const long long step = static_cast<long long>(a.n_tokens) * a.n_q;
  const long long at = static_cast<long long>(t) * a.n_q + head;
  float m = -INFINITY;
  for (int p = lane; p < parts; p += 32) m = fmaxf(m, a.part_ml[p * step + at].x);
#pragma unroll
  for (int k = 16; k > 0; k /= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, k));
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f, acc[D] = {};
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    const float2 ml = a.part_ml[p * step + at];
    const float f = ex2(ml.x - base);
    l += ml.y * f;
    const float* o = a.part_o + (p * step + at) * HD + lane * D;
#pragma unroll
    for (int d = 0; d < D; ++d) acc[d] += o[d] * f;
  }
  store_row<HD>(a, s, head / a.group, t, head, min(len - count + i, len - 1), len, acc, m, l, lane);
}

template <typename F>
cudaError_t launch_pdl(F* k, long long blocks, int threads, int smem, cudaStream_t st,
                       const AttnArgs& a) {
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
  return cudaLaunchKernelEx(&cfg, k, a);
}

template <int HD, int MT>
cudaError_t launch_few(AttnArgs a, cudaStream_t st, int device) {
  static std::atomic<unsigned long long> done{0};
  constexpr int smem = kWarps * kStages * stage_bytes<HD>();
  auto* k = attention_few_kernel<HD, MT>;
  const unsigned long long bit = 1ull << (device & 63);
  if (!(done.load(std::memory_order_relaxed) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_relaxed);
  }
  a.row_tiles = (a.max_q * a.group + 16 * MT - 1) / (16 * MT);
  const long long blocks =
      static_cast<long long>(a.c.n_seqs) * a.row_tiles * a.c.n_kv * a.n_splits;
  return launch_pdl(k, blocks, 32 * kWarps, smem, st, a);
}

}  // namespace

int attention_splits(int n_seqs, int n_kv, int n_tokens, int group, int max_q, long long capacity,
                     int sms) {
  const long long rows = static_cast<long long>(max_q) * group;
  if (attention_is_many(group, max_q))
    return attention_many_splits(attention_many_units(n_seqs, n_tokens, group, max_q), n_kv,
                                 capacity, sms);
  const long long tiles = rows <= 16 ? 1 : (rows + 31) / 32;
  const long long units = tiles * n_kv * n_seqs;
  long long want = (2LL * sms + units - 1) / units;  // two blocks to a multiprocessor
  const long long most = (capacity + 63) / 64;       // 64 entries a part at least
  if (want > most) want = most;
  return want < 1 ? 1 : static_cast<int>(want);
}

size_t attention_part_bytes(int splits, int n_tokens, int n_q, int head_dim) {
  if (splits <= 1) return 0;
  return static_cast<size_t>(splits) * n_tokens * n_q * (static_cast<size_t>(head_dim) * 4 + 8);
}

cudaError_t paged_attention_launch(AttnArgs a, int sms, cudaStream_t st, int device) {
  (void)sms;
  const bool one = a.max_q * a.group <= 16;
  cudaError_t e;
  a.part_unit = attention_is_many(a.group, a.max_q) ? 128 : 64;
  if (attention_is_many(a.group, a.max_q))
    e = attention_many_launch(a, st, device);
  else if (a.c.head_dim == 64)
    e = one ? launch_few<64, 1>(a, st, device) : launch_few<64, 2>(a, st, device);
  else
    e = one ? launch_few<128, 1>(a, st, device) : launch_few<128, 2>(a, st, device);
  if (e != cudaSuccess || a.n_splits == 1) return e;
  const long long rows = static_cast<long long>(a.c.n_seqs) * a.max_q * a.n_q;
  return a.c.head_dim == 64
             ? launch_pdl(attention_join_kernel<64>, (rows + 3) / 4, 128, 0, st, a)
             : launch_pdl(attention_join_kernel<128>, (rows + 3) / 4, 128, 0, st, a);
}

}  // namespace qgemv
