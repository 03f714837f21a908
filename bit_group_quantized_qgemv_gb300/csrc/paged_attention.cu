// paged_attention.cu -- qgemv_paged_attention for few query rows per
// key/value head (decode steps, drafts): split over the cache, mma.sync.
//
// The rows of a (sequence, key/value head) are its new tokens times the query
// heads that share the head, row r = token r / group, head r % group.  A
// thread block takes NT * 8 of them and one part of the cache; its warps take
// tiles of 16 entries in turn, each through a ring of its own (cp.async, no
// block-wide barrier until the end), so the loop is a stream of K and V through
// shared memory.  Per tile, transposed so that the rows are the eight columns
// of m16n8k16 and nothing is padded to 16: S^T = K Q^T, the running maximum and
// sum of the softmax in fp32 registers, and O^T += V^T P^T with P^T made from
// the accumulators by a transpose of 8 x 8 matrices.  (With the rows as the 16 of
// the product, padded, a tile took three times the products; 48 sequences of 900 to
// 20000 entries: 202 against 185 us.)  The warps' (max, sum, O) are joined in
// shared memory, the parts of a split cache through the distributed shared
// memory of a cluster or by a second kernel.
//
// Up to 16 rows P enters as fp16 high and low parts (two products with V): 22 bits of
// a weight down to 2^-9 of the running maximum, below that what lies above 2^-32 of it
// (kLift).  The kernel is bound by HBM there, not by the products.  48 sequences of 900
// to 20000 entries (32/8 heads of 128, 1.23 GB) take 185 us, 6.65 TB/s or 98 % of the
// measured copy bandwidth.  With more rows the products are the bound, and P is rounded
// once to fp16, like every weight of the tcgen05 kernel.  Heads of 128 with more
// rows than 16 take 255 registers and spill 16 bytes (24 rows) and 284 (32).
#include <atomic>

#include "attention_common.cuh"
#include "mma_tile.cuh"
#include "runs.cuh"

namespace qgemv {
namespace {

constexpr int kTile = 16;    // entries per warp and step
constexpr int kStages = 3;   // ring depth of each warp
constexpr int kBlock = 64;      // entries that runs of work are counted in
constexpr int kMinBlocks = 2;   // of a run, at least
constexpr int kRowsMax = 32;    // rows of a unit

template <int HD>
__host__ __device__ constexpr int stage_bytes() {
  return 2 * kTile * HD * 2;
}

constexpr int kMaxCluster = 8;

__device__ __forceinline__ int cluster_rank() {
  int r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// A float of block `rank`'s shared memory, at this block's address of it.
__device__ __forceinline__ float ld_cluster(uint32_t addr, int rank) {
  float v;
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %1, %2;\n ld.shared::cluster.f32 %0, [a];\n}"
      : "=f"(v)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

// Transpose of an 8 x 8 matrix of 16-bit values, two per thread.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Blocks resident on a multiprocessor: two for heads of 128 (by shared memory;
// one of eight warps), for heads of 64 four, by the registers of more rows three or
// two.
__host__ __device__ constexpr int few_resident(int head_dim, int rows, int warps) {
  return warps == 8 ? 1 : head_dim == 128 || rows > 24 ? 2 : rows > 16 ? 3 : 4;
}

template <int HD, int NT, bool LO, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, few_resident(HD, 8 * NT, kWarps))
    attention_few_kernel(const AttnArgs a) {
  constexpr int kM = HD / 16;      // 16-component tiles of the output, k-steps of the scores
  constexpr int kRows = 8 * NT;
  constexpr int kChunks = HD / 8;  // 16-byte chunks per row
  constexpr int kOut = HD + 4;     // floats between output rows in shared memory (banks)
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float sm_m[kWarps][kRows], sm_l[kWarps][kRows];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tq = lane & 3;

  constexpr int D = HD / 32;
  float* so = reinterpret_cast<float*>(smem);  // [warp][row][kOut], once a segment's ring is done

  // Blocks of entries of sequence i's units; its units count as one block each
  // when there is no workspace to join parts of them.
  const bool cut = a.splits != nullptr;
  auto blocks_of = [&](int i) {
    int f, n;
    seq_rows(a.q_start, i, a.n_tokens, a.err, &f, &n);
    if (n > a.max_q) flag_error(a.err);
    const int l = seq_len(a.c, i, a.err);
    return n == 0 ? 0 : cut ? max(1, (l + kBlock - 1) / kBlock) : 1;
  };
  int s, h, j0 = 0;
  long long left = 1, per = 1;
  AttnUnit split{};
  if (a.cluster > 1) {  // a cluster per unit, a part per block of it
    const int unit = blockIdx.x / a.cluster;
    s = unit / a.c.n_kv;
    h = unit % a.c.n_kv;
  } else {
    left = run_start(a.c.n_seqs, a.c.n_kv, cut ? kMinBlocks : 1, lane, blocks_of, &per, &s, &h, &j0);
    if (left <= 0) {
      if (cut && threadIdx.x == 0) a.splits[blockIdx.x] = split;
      return;
    }
  }

  while (true) {
    int first, count;
    int* err = a.cluster > 1 ? a.err : nullptr;  // (the others have looked at every length)
    seq_rows(a.q_start, s, a.n_tokens, err, &first, &count);
    const int len = seq_len(a.c, s, err);
    if (a.cluster > 1) {
      if (count > a.max_q) flag_error(err);
      if (count == 0) return;
    }
    const int nr = min(count, a.max_q) * a.group;
    const int off = len - count;  // token i sees entries up to off + i
    // this segment's entries k0 .. k1, of those that some row sees
    const int see = min(len, off + (nr - 1) / a.group + 1);
    const int n_blocks = max(1, (len + kBlock - 1) / kBlock);
    int k0, k1, slot = -1;
    if (a.cluster > 1) {
      const int part = (n_blocks + a.cluster - 1) / a.cluster * kBlock;
      k0 = cluster_rank() * part;
      k1 = min(see, k0 + part);
    } else if (!cut) {
      k0 = 0;
      k1 = see;
    } else {
      const int j1 = static_cast<int>(min(static_cast<long long>(n_blocks), j0 + left));
      k0 = j0 * kBlock;
      k1 = min(see, j1 * kBlock);
      if (j0 > 0 || j1 < n_blocks) slot = 2 * static_cast<int>(blockIdx.x) + (j0 == 0);
      if (j0 == 0 && j1 < n_blocks)
        split = AttnUnit{1 + static_cast<int>(run_div(n_blocks - j1 + per - 1, per)), s, h, 0, first, nr, off,
                         len};
      // who has the first part of a cut unit; -1: the unit is whole
      if (j0 == 0 && a.first_of != nullptr && threadIdx.x == 0)
        a.first_of[s * a.c.n_kv + h] = j1 < n_blocks ? static_cast<int>(blockIdx.x) : -1;
      left -= j1 - j0;
    }
    if (a.cluster == 1 && !cut) --left;

    const uint32_t ring = smem_u32(smem) + warp * (kStages * stage_bytes<HD>());
    const int tiles = k1 > k0 ? (k1 - k0 + kTile - 1) / kTile : 0;
    const int mine = tiles > warp ? (tiles - warp + kWarps - 1) / kWarps : 0;
    unsigned bad = 0;  // bit st: the tile in stage st lies on a bad page
    int next = mine > 0 ? raw_page(a.c, s, k0 + warp * kTile) : -1;

    // Queries as B fragments: column = row of the block.
    uint32_t qf[NT][kM][2];
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + g;
      const int i = r / a.group, head = h * a.group + r % a.group;
      const __half* q = a.q + static_cast<long long>(first + i) * a.q_stride + head * HD + 2 * tq;
#pragma unroll
      for (int k = 0; k < kM; ++k) {
        qf[nt][k][0] = r < nr ? *reinterpret_cast<const uint32_t*>(q + 16 * k) : 0u;
        qf[nt][k][1] = r < nr ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 8) : 0u;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = nt * 8 + 2 * tq + e;
        lim[nt][e] = c < nr ? off + c / a.group : -1;
      }
    }

    float o[NT][kM][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int d = 0; d < kM; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][d][e] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }

    auto issue = [&](int it) {
      if (it < mine) {
        const int e0 = k0 + (it * kWarps + warp) * kTile;
        const int st = it % kStages;
        const uint32_t kd = ring + st * stage_bytes<HD>(), vd = kd + stage_bytes<HD>() / 2;
        const int page = good_page(a.c, next, a.err);
        const long long base = page >= 0 ? cache_row(a.c, page, h, e0) * HD : 0;
        const int end = page >= 0 ? len : 0;
        bad = page >= 0 ? bad & ~(1u << st) : bad | (1u << st);
#pragma unroll
        for (int c = 0; c < kTile * kChunks / 32; ++c) {
          const int id = c * 32 + lane, r = id / kChunks, ch = id % kChunks;
          // (rows behind the end lie on the page and are not read)
          const bool take = e0 + r < end;
          cp_async16(kd + tile_off<HD>(r, ch), a.c.k + base + id * 8, take);
          cp_async16(vd + tile_off<HD>(r, ch), a.c.v + base + id * 8, take);
        }
        // the next tile's page, a step ahead of its use
        if (it + 1 < mine) next = raw_page(a.c, s, e0 + kWarps * kTile);
      }
      cp_commit();
    };
#pragma unroll
    for (int p = 0; p < kStages - 1; ++p) issue(p);

    const int kr = (lane & 7) + (((lane >> 3) & 1) << 3), kc = lane >> 4;
    const int vr = (lane & 7) + ((lane >> 4) << 3), vc = (lane >> 3) & 1;
    for (int it = 0; it < mine; ++it) {
      cp_wait<kStages - 2>();
      __syncwarp();
      issue(it + kStages - 1);
      const int st = it % kStages;
      const int e0 = k0 + (it * kWarps + warp) * kTile;
      const uint32_t kd = ring + st * stage_bytes<HD>(), vd = kd + stage_bytes<HD>() / 2;
      // S^T: 16 entries x 8 rows per tile of rows, even and odd k-steps apart
      // (two shorter chains of products)
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
      uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x[4];
        bool over = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = e0 + g + 8 * (e >> 1);
          const bool seen = !hidden && j <= lim[nt][e & 1];
          x[e] = seen ? (sc[nt][0][e] + sc[nt][1][e]) * a.scale_log2 : -INFINITY;
          over |= x[e] - m[nt][e & 1] > kTop;  // (from no base at all, -inf, on: infinite)
        }
        // The base is lazy: it moves (and O is rescaled) only where a weight would
        // pass the top, so most tiles cost one vote.
        if (__any_sync(0xFFFFFFFFu, over)) {
          float mn[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mn[e] = fmaxf(x[e], x[e + 2]);
            mn[e] = fmaxf(mn[e], __shfl_xor_sync(0xFFFFFFFFu, mn[e], 4));
            mn[e] = fmaxf(mn[e], __shfl_xor_sync(0xFFFFFFFFu, mn[e], 8));
            mn[e] = fmaxf(mn[e], __shfl_xor_sync(0xFFFFFFFFu, mn[e], 16));
            mn[e] = fmaxf(m[nt][e], base_of(mn[e]));
          }
          const float f0 = mn[0] == m[nt][0] ? 1.f : ex2(m[nt][0] - mn[0]);
          const float f1 = mn[1] == m[nt][1] ? 1.f : ex2(m[nt][1] - mn[1]);
          l[nt][0] *= f0;
          l[nt][1] *= f1;
#pragma unroll
          for (int d = 0; d < kM; ++d) {
            o[nt][d][0] *= f0;
            o[nt][d][1] *= f1;
            o[nt][d][2] *= f0;
            o[nt][d][3] *= f1;
          }
          m[nt][0] = mn[0];
          m[nt][1] = mn[1];
        }
        const float b0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0];
        const float b1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // entry g, then g + 8
          const float u = ex2(x[2 * e] - b0), v = ex2(x[2 * e + 1] - b1);
          l[nt][0] += u;
          l[nt][1] += v;
          const uint32_t hi = pack_f16(u, v);
          ph[nt][e] = transpose8(hi);
          if (LO) {
            const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&hi));
            pl[nt][e] = transpose8(pack_f16(u - hf.x, v - hf.y));
          }
        }
      }
      // O^T += V^T P^T
#pragma unroll
      for (int d = 0; d < kM; ++d) {
        uint32_t vf[4];
        ldsm4t(vf, vd + tile_off<HD>(vr, 2 * d + vc));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(o[nt][d], vf, ph[nt][0], ph[nt][1]);
          if (LO) mma_f16(o[nt][d], vf, pl[nt][0], pl[nt][1]);
        }
      }
      __syncwarp();
    }
    cp_wait<0>();
    __syncthreads();  // every warp is done with its ring: it now takes the partial outputs
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float lsum = l[nt][e];
        lsum += __shfl_xor_sync(0xFFFFFFFFu, lsum, 4);
        lsum += __shfl_xor_sync(0xFFFFFFFFu, lsum, 8);
        lsum += __shfl_xor_sync(0xFFFFFFFFu, lsum, 16);
        if (g == 0) {
          sm_m[warp][nt * 8 + 2 * tq + e] = m[nt][e];
          sm_l[warp][nt * 8 + 2 * tq + e] = lsum;
        }
      }
#pragma unroll
      for (int d = 0; d < kM; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          so[(warp * kRows + nt * 8 + 2 * tq + (e & 1)) * kOut + 16 * d + g + 8 * (e >> 1)] =
              o[nt][d][e];
    }
    __syncthreads();
    // A warp per row: join the warps' parts.
    const auto finish = [&](int r, float mm, float ll, const float* acc) {
      const int i = r / a.group, head = h * a.group + r % a.group, t = first + i;
      if (slot < 0) {
        store_row<HD>(a, s, h, t, head, min(off + i, len - 1), len, acc, mm, ll, lane);
        return;
      }
      const long long at = static_cast<long long>(slot) * kRowsMax + r;
#pragma unroll
      for (int d = 0; d < D; ++d) a.part_o[at * HD + lane * D + d] = acc[d];
      if (lane == 0) a.part_ml[at] = make_float2(mm, ll);
    };
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
        for (int d = 0; d < D; ++d) acc[d] += so[(w * kRows + r) * kOut + lane * D + d] * f;
      }
      if (a.cluster == 1) {
        finish(r, mm, ll, acc);
        continue;
      }
      // (row r is this warp's alone: its sum may take the place of warp 0's part)
      __syncwarp();
#pragma unroll
      for (int d = 0; d < D; ++d) so[r * kOut + lane * D + d] = acc[d];
      if (lane == 0) {
        sm_m[0][r] = mm;
        sm_l[0][r] = ll;
      }
    }
    if (a.cluster > 1) break;
    if (left <= 0) break;
    j0 = 0;
    if (++h == a.c.n_kv) {
      h = 0;
      s = run_next(s, a.c.n_seqs, lane, blocks_of);
      if (s >= a.c.n_seqs) break;
    }
    __syncthreads();  // the next segment's ring takes the place of these outputs
  }
  if (a.cluster == 1) {
    if (cut && threadIdx.x == 0) a.splits[blockIdx.x] = split;
    return;
  }
  // The blocks of a cluster join theirs through distributed shared memory,
  // each for some of the rows.
  int first, count;
  seq_rows(a.q_start, s, a.n_tokens, nullptr, &first, &count);
  const int len = seq_len(a.c, s, nullptr), nr = min(count, a.max_q) * a.group;
  cluster_sync();
  for (int r = cluster_rank() * kWarps + warp; r < nr; r += a.cluster * kWarps) {
    const uint32_t m_at = smem_u32(&sm_m[0][r]), l_at = smem_u32(&sm_l[0][r]);
    const uint32_t o_at = smem_u32(so + r * kOut + lane * D);
    float mm = -INFINITY, pm[kMaxCluster], pl[kMaxCluster], po[kMaxCluster][D];
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {
      pm[c] = -INFINITY;
      pl[c] = 0.f;
      if (c < a.cluster) {
        pm[c] = ld_cluster(m_at, c);
        pl[c] = ld_cluster(l_at, c);
#pragma unroll
        for (int d = 0; d < D; ++d) po[c][d] = ld_cluster(o_at + 4 * d, c);
      } else {
#pragma unroll
        for (int d = 0; d < D; ++d) po[c][d] = 0.f;
      }
      mm = fmaxf(mm, pm[c]);
    }
    const float base = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f, acc[D] = {};
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {
      const float f = ex2(pm[c] - base);
      ll += pl[c] * f;
#pragma unroll
      for (int d = 0; d < D; ++d) acc[d] += po[c][d] * f;
    }
    const int i = r / a.group;
    store_row<HD>(a, s, h, first + i, h * a.group + r % a.group, min(len - count + i, len - 1), len,
                  acc, mm, ll, lane);
  }
  cluster_sync();  // no block ends while another reads its shared memory
}

// Join the parts of cut units: block c of the kernel above has the first part of
// at most one (in its slot 1), the blocks behind it the others (in their slots
// 0).  Four rows a block, the four warps of a row take the parts in turn.  The
// blocks here go over the units where those are fewer (first_of), else over the blocks
// there: mostly empty ones cost 5 us of 26 for four sequences of 21 rows.
constexpr int kJoinWarps = 4, kJoinRows = 4;

template <int HD>
__global__ void __launch_bounds__(32 * kJoinWarps * kJoinRows)
    attention_join_kernel(const AttnArgs a, int row_blocks) {
  constexpr int D = HD / 32;
  __shared__ float s_o[kJoinRows][kJoinWarps][HD], s_m[kJoinRows][kJoinWarps], s_l[kJoinRows][kJoinWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = (threadIdx.x >> 5) % kJoinWarps, row = threadIdx.x / (32 * kJoinWarps);
  const int lane = threadIdx.x & 31;
  int c = blockIdx.x / row_blocks;
  const int r = blockIdx.x % row_blocks * kJoinRows + row;
  if (a.first_of != nullptr) {
    const int s = c / a.c.n_kv;
    int first, count;
    c = a.first_of[c];  // (nobody wrote it for a sequence without tokens)
    seq_rows(a.q_start, s, a.n_tokens, nullptr, &first, &count);
    if (count == 0 || c < 0) return;
  }
  auto& so = s_o[row];
  auto& sm = s_m[row];
  auto& sl = s_l[row];
  const AttnUnit unit = a.splits[c];
  const int parts = unit.parts;
  if (parts == 0 || r >= unit.rows) return;  // all warps of the row
  float m = -INFINITY, l = 0.f, acc[D] = {};
  constexpr int kU = 8;  // parts in flight per warp
  for (int p0 = warp; p0 < parts; p0 += kJoinWarps * kU) {
    float2 ml[kU];
    float o[kU][D];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int p = p0 + u * kJoinWarps;
      ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int d = 0; d < D; ++d) o[u][d] = 0.f;
      if (p < parts) {
        const long long at = static_cast<long long>(p == 0 ? 2 * c + 1 : 2 * (c + p)) * kRowsMax + r;
        ml[u] = a.part_ml[at];
        const float* src = a.part_o + at * HD + lane * D;
        if constexpr (D == 4) {
          const float4 v = *reinterpret_cast<const float4*>(src);
          o[u][0] = v.x, o[u][1] = v.y, o[u][2] = v.z, o[u][3] = v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(src);
          o[u][0] = v.x, o[u][1] = v.y;
        }
      }
    }
    float mn = m;
#pragma unroll
    for (int u = 0; u < kU; ++u) mn = fmaxf(mn, ml[u].x);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float f0 = ex2(m - base);
    l *= f0;
#pragma unroll
    for (int d = 0; d < D; ++d) acc[d] *= f0;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const float f = ex2(ml[u].x - base);
      l += ml[u].y * f;
#pragma unroll
      for (int d = 0; d < D; ++d) acc[d] += o[u][d] * f;
    }
    m = mn;
  }
#pragma unroll
  for (int d = 0; d < D; ++d) so[warp][lane * D + d] = acc[d];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  named_bar_sync(1 + row, 32 * kJoinWarps);  // the warps of this row
  if (warp != 0) return;
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) m = fmaxf(m, sm[w]);
  const float base = m == -INFINITY ? 0.f : m;
  l = 0.f;
#pragma unroll
  for (int d = 0; d < D; ++d) acc[d] = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    const float f = ex2(sm[w] - base);
    l += sl[w] * f;
#pragma unroll
    for (int d = 0; d < D; ++d) acc[d] += so[w][lane * D + d] * f;
  }
  const int i = r / a.group;
  store_row<HD>(a, unit.s, unit.h, unit.first + i, unit.h * a.group + r % a.group,
                min(unit.off + i, unit.len - 1), unit.len, acc, m, l, lane);
}

template <typename F, typename... Args>
cudaError_t launch_pdl(F* k, long long blocks, int threads, int smem, int cluster, cudaStream_t st,
                       Args... args) {
  if (blocks < 1 || blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

// Blocks of a call: as many as are resident at once.
int few_blocks(int head_dim, int rows, int sms) { return sms * few_resident(head_dim, rows, 4); }

template <int HD, int NT, bool LO, int kWarps>
cudaError_t launch_few(const AttnArgs& a, int sms, cudaStream_t st, int device) {
  static std::atomic<unsigned long long> done{0};
  constexpr int smem = kWarps * kStages * stage_bytes<HD>();
  static_assert(kWarps * 8 * NT * (HD + 4) * 4 <= smem, "the warps' outputs take the ring's place");
  auto* k = attention_few_kernel<HD, NT, LO, kWarps>;
  const unsigned long long bit = 1ull << (device & 63);
  if (!(done.load(std::memory_order_relaxed) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_relaxed);
  }
  const long long blocks = a.cluster > 1
                               ? static_cast<long long>(a.c.n_seqs) * a.c.n_kv * a.cluster
                               : few_blocks(HD, a.max_q * a.group, sms);
  return launch_pdl(k, blocks, 32 * kWarps, smem, a.cluster, st, a);
}

// Warps per block: eight where the clusters leave a multiprocessor to each
// block (8 units of 8 blocks; 16 do not fit next to one another: 10.4 us
// against 6.9 for two sequences of 500), four, two blocks to a multiprocessor,
// elsewhere.
int few_warps(int rows, int cluster, int units) {
  return cluster > 1 && units <= 8 && rows <= 16 ? 8 : 4;
}

template <int HD>
cudaError_t launch_few_rows(const AttnArgs& a, int sms, cudaStream_t st, int device) {
  const int rows = a.max_q * a.group;
  const bool wide = few_warps(rows, a.cluster, a.c.n_seqs * a.c.n_kv) == 8;
  if (rows <= 8)
    return wide ? launch_few<HD, 1, true, 8>(a, sms, st, device)
                : launch_few<HD, 1, true, 4>(a, sms, st, device);
  if (rows <= 16)
    return wide ? launch_few<HD, 2, true, 8>(a, sms, st, device)
                : launch_few<HD, 2, true, 4>(a, sms, st, device);
  if (rows <= 24) return launch_few<HD, 3, false, 4>(a, sms, st, device);
  return launch_few<HD, 4, false, 4>(a, sms, st, device);
}

// Whether a cluster of blocks takes each (sequence, head) unit and joins on
// chip, by the number of units and the capacity (the lengths are on the device);
// otherwise the entries are cut into equal runs (runs.cuh), joined by a second
// kernel.  Measured on GB300, four query heads of 128 to a key head, one new token per
// sequence, replayed from a graph, clusters of 8 against runs and their join (us):
//   1 sequence, key heads   1000        4110          8000          12000     entries
//                 8    5.9 and 7.5   8.1 and 10.3  10.0 and 11.1  12.3 and 12.9
//                 4    5.9     6.6   7.9      9.9   9.8     11.1  12.0     11.5
//                 2    5.8     6.2   7.8      9.2   9.6     10.4  11.8     10.5
//                 1    5.6     6.2   7.8      7.2   9.5      8.2  11.8      9.6
//   sequences, key heads    1000        4000
//              2, 4    5.9 and 7.7   7.7 and  9.9
//              4, 2    5.9     7.5   7.8      9.9
//              4, 4    7.2     8.1  10.4     11.2
//              2, 8    7.5      8.7  10.7     12.0
//              4, 8    8.3      8.9  11.9     12.7
// (one sequence of 16000, 8 heads: 15.2 and 14.5; two of 8000: 15.2 and 12.1; clusters
// of 16: 14.7 at one of 4110).  A cluster also saves the workspace and a launch, 4 us of
// a call's time on the host.  So clusters serve one sequence's 8 heads up to parts of 1536
// entries, and more units up to 512 while their blocks fill the machine at most once.
// The rule was cut for 8 key heads; with a single one the runs are ahead on the GPU from
// 4000 entries on, with two and four from 12000.  With longer caches a cluster lasts as long as
// its sequence; a table with room for more than the rule's entries goes to the runs whatever the
// sequence's length.
int few_cluster(int n_seqs, int n_kv, long long capacity, int sms) {
  const long long units = static_cast<long long>(n_kv) * n_seqs;
  const bool fits = capacity > 128 && units <= 2 * sms / kMaxCluster &&
                    capacity <= kMaxCluster * (units <= 8 ? 1536 : 512);
  return fits ? kMaxCluster : 1;
}

}  // namespace

size_t attention_few_bytes(int n_seqs, int n_kv, int rows, int head_dim, long long capacity,
                           int sms) {
  if (few_cluster(n_seqs, n_kv, capacity, sms) > 1 || capacity <= 128) return 0;
  return static_cast<size_t>(few_blocks(head_dim, rows, sms)) *
         (2 * kRowsMax * (static_cast<size_t>(head_dim) * 4 + 8) + sizeof(AttnUnit) + sizeof(int));
}

cudaError_t attention_few_launch(AttnArgs a, int sms, cudaStream_t st, int device, void* workspace,
                                 size_t bytes) {
  const int hd = a.c.head_dim, rows = a.max_q * a.group;
  const long long capacity = static_cast<long long>(a.c.max_pages) << a.c.page_shift;
  const size_t need = attention_few_bytes(a.c.n_seqs, a.c.n_kv, rows, hd, capacity, sms);
  const int blocks = few_blocks(hd, rows, sms);
  a.cluster = few_cluster(a.c.n_seqs, a.c.n_kv, capacity, sms);
  const long long units = static_cast<long long>(a.c.n_seqs) * a.c.n_kv;
  a.splits = nullptr;
  a.first_of = nullptr;
  if (need > 0 && bytes >= need) {  // outputs, {max, sum}, what the join needs
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + 2LL * blocks * kRowsMax * hd);
    a.splits = reinterpret_cast<AttnUnit*>(a.part_ml + 2LL * blocks * kRowsMax);
    if (units <= blocks) a.first_of = reinterpret_cast<int*>(a.splits + blocks);
  }
  auto run = [&] {
    return hd == 64 ? launch_few_rows<64>(a, sms, st, device)
                    : launch_few_rows<128>(a, sms, st, device);
  };
  cudaError_t e = run();
  if (e != cudaSuccess && a.cluster > 1) {  // a device that cannot host the clusters
    cudaGetLastError();
    a.cluster = 1;
    e = run();
  }
  if (e != cudaSuccess || a.splits == nullptr) return e;
  const int row_blocks = (rows + kJoinRows - 1) / kJoinRows, threads = 32 * kJoinWarps * kJoinRows;
  const long long joins = (a.first_of != nullptr ? units : blocks) * row_blocks;
  return hd == 64
             ? launch_pdl(attention_join_kernel<64>, joins, threads, 0, 1, st, a, row_blocks)
             : launch_pdl(attention_join_kernel<128>, joins, threads, 0, 1, st, a, row_blocks);
}

}  // namespace qgemv
