// cache_evict.cu -- qgemv_cache_evict: keep the entries of largest mass of
// each (sequence, key/value head) and close the gaps.
//
// Selection: one block per (sequence, head).  Masses become 32-bit keys whose
// order is the ranking (protected entries highest, NaN lowest), read once and
// kept in shared memory; the keep-th largest key T is found by radix selection
// (2048 bins: with 256 most lanes of a warp met in one, the leading bits of floats
// of like size being the same), and the lowest-index entries equal to T fill up
// what is missing.  Every warp owns a run of consecutive entries, so ranks in
// index order are prefix sums over the warps' counts.  The movers are listed, the
// holes pick theirs from the list, and only then the permuted masses and positions are
// written.  The list lies in shared memory while every block has a
// multiprocessor to itself (one sequence of 4159 entries, 8 heads: 12.4 us a call
// against 14.2), else at the front of pos_out, where it is at most as long as what comes
// there in the end (24 sequences, 192 heads: 90.3 us against 98.7 with the larger
// blocks).  What decides is the capacity, as the host knows no lengths: with
// a table for more than kKeysMax entries the keys are made again at every pass (4159
// entries 14.4 us for 11.4 from a graph, 24 sequences 115 for 103), and a head has one
// block at any length (131072 entries, 8 heads: 155 us).
// Moving: a second kernel copies the rows of k and v whose place changed.
// Sources lie at or beyond the new length and targets below it, so no copy
// reads what another writes.
#include <atomic>

#include "kv_cache.cuh"

namespace qgemv {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;

// Larger key: kept first.  Equal masses (-0 and +0 too) have equal keys.
__device__ __forceinline__ unsigned rank_key(float mass, int pos, int sink, long long recent) {
  if (pos < sink || pos >= recent) return kAll;
  if (mass != mass) return 0u;
  const unsigned b = __float_as_uint(mass == 0.f ? 0.f : mass);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Sums of the warps below this one, and the total over the block.
template <int kWarps>
__device__ __forceinline__ int warps_before(int mine, int* slots, int warp, int lane) {
  __syncthreads();
  if (lane == 0) slots[warp] = mine;
  __syncthreads();
  int below = lane < warp && lane < kWarps ? slots[lane] : 0;
#pragma unroll
  for (int k = 16; k > 0; k /= 2) below += __shfl_xor_sync(kAll, below, k);
  return below;
}

constexpr int kBins = 2048;  // 11 bits a pass: 11, 11, 10

// KEYS: the keys stay in (dynamic) shared memory; else they are made again from
// memory at every pass.  LIST: the movers are listed there too.
constexpr int kThreads = 1024;  // two blocks to a multiprocessor

template <bool KEYS, bool LIST>
__global__ void __launch_bounds__(kThreads, 2) evict_select_kernel(const EvictArgs a) {
  constexpr int kWarps = kThreads / 32;
  constexpr int kOwn = kBins / kThreads;  // bins of a thread in the search, highest first
  extern __shared__ unsigned keys[];
  __shared__ int hist[kBins];
  __shared__ int slots[kWarps];
  __shared__ unsigned s_prefix;
  __shared__ int s_left;
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.x % a.c.n_kv, s = blockIdx.x / a.c.n_kv;
  const int next = a.next_pos[s];
  const int len = seq_len(a.c, s, a.err);
  const int left = min(len, a.keep);
  const long long cap = static_cast<long long>(a.c.max_pages) << a.c.page_shift;
  const long long base = (static_cast<long long>(s) * a.c.n_kv + h) * cap;
  const float* mass = a.mass + base;
  const int* pos = a.entry_pos + base;
  float* mass_out = a.mass_out + base;
  int* pos_out = a.pos_out + base;
  int* kept = a.kept + (static_cast<long long>(s) * a.c.n_kv + h) * a.keep;
  const long long recent = static_cast<long long>(next) - a.n_recent;
  if (h == 0 && threadIdx.x == 0) a.len_out[s] = left;
  for (int i = left + threadIdx.x; i < a.keep; i += kThreads) kept[i] = -1;
  if (len == left) {  // nothing to choose
    for (int i = threadIdx.x; i < left; i += kThreads) {
      kept[i] = i;
      mass_out[i] = mass[i];
      pos_out[i] = pos[i];
    }
    return;
  }

  for (int i = threadIdx.x; i < kBins; i += kThreads) hist[i] = 0;
  // Four consecutive entries per thread and step (16-byte loads where the arrays
  // allow them; the capacity is a multiple of 16).
  const bool wide = ((reinterpret_cast<uintptr_t>(mass) | reinterpret_cast<uintptr_t>(pos)) & 15) == 0;
  auto make4 = [&](int i, unsigned* k) {
    float m[4];
    int p[4];
    if (wide) {
      const float4 m4 = *reinterpret_cast<const float4*>(mass + i);
      const int4 p4 = *reinterpret_cast<const int4*>(pos + i);
      m[0] = m4.x, m[1] = m4.y, m[2] = m4.z, m[3] = m4.w;
      p[0] = p4.x, p[1] = p4.y, p[2] = p4.z, p[3] = p4.w;
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        m[c] = mass[i + c];
        p[c] = pos[i + c];
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) k[c] = rank_key(m[c], p[c], a.n_sink, recent);
  };
  auto load4 = [&](int i, unsigned* k) {
    if constexpr (KEYS) {
      const uint4 v = *reinterpret_cast<const uint4*>(keys + i);
      k[0] = v.x, k[1] = v.y, k[2] = v.z, k[3] = v.w;
    } else {
      make4(i, k);
    }
  };
  if constexpr (KEYS) {
#pragma unroll 4
    for (int i = 4 * threadIdx.x; i < len; i += 4 * kThreads) {
      unsigned k[4];
      make4(i, k);
      *reinterpret_cast<uint4*>(keys + i) = make_uint4(k[0], k[1], k[2], k[3]);
    }
  }
  __syncthreads();

  // T: the left-th largest key; need: how many of the entries equal to it stay
  unsigned prefix = 0, above = 0;
  int need = left;
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const unsigned bins = pass == 2 ? 1023u : 2047u;
    for (int i0 = warp * 128; i0 < len; i0 += 4 * kThreads) {
      const int i = i0 + 4 * lane;
      unsigned k[4] = {0u, 0u, 0u, 0u};
      if (i < len) load4(i, k);
      bool in[4], same = true;
      int bin[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        in[c] = i + c < len && (k[c] & above) == prefix;
        bin[c] = (k[c] >> shift) & bins;
      }
      // entries that all fall into the first one's bin (equal masses) count once
      const int bin0 = __shfl_sync(kAll, bin[0], 0);
#pragma unroll
      for (int c = 0; c < 4; ++c) same &= in[c] && bin[c] == bin0;
      if (__all_sync(kAll, same)) {
        if (lane == 0) atomicAdd(&hist[bin0], 128);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (in[c]) atomicAdd(&hist[bin[c]], 1);
      }
    }
    __syncthreads();
    // the bin in which the need-th largest lies
    int c[kOwn], sum = 0;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      c[k] = hist[kBins - 1 - (threadIdx.x * kOwn + k)];
      sum += c[k];
    }
    int incl = sum;
#pragma unroll
    for (int k = 1; k < 32; k *= 2) {
      const int v = __shfl_up_sync(kAll, incl, k);
      if (lane >= k) incl += v;
    }
    int run = warps_before<kWarps>(__shfl_sync(kAll, incl, 31), slots, warp, lane) + incl - sum;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      const int b = kBins - 1 - (threadIdx.x * kOwn + k);
      if (run < need && run + c[k] >= need) {
        s_prefix = prefix | (static_cast<unsigned>(b) << shift);
        s_left = need - run;
      }
      run += c[k];
      hist[b] = 0;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_left;
    above |= bins << shift;
  }
  const unsigned T = prefix;

  // Runs of whole 128-entry groups per warp, in index order: counts of what
  // stays for certain and of the entries equal to T, below and from `left` on.
  const int per = ((len + 127) / 128 + kWarps - 1) / kWarps * 128;
  const int i_lo = min(len, warp * per), i_hi = min(len, (warp + 1) * per);
  int n_gt_low = 0, n_gt_high = 0, n_eq_low = 0, n_eq_high = 0;  // this lane's
  for (int i = i_lo + 4 * lane; i < i_hi; i += 128) {
    unsigned k[4];
    load4(i, k);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const bool in = i + c < i_hi, low = i + c < left;
      n_gt_low += in && low && k[c] > T;
      n_gt_high += in && !low && k[c] > T;
      n_eq_low += in && low && k[c] == T;
      n_eq_high += in && !low && k[c] == T;
    }
  }
  const int gt_low = __reduce_add_sync(kAll, n_gt_low), gt_high = __reduce_add_sync(kAll, n_gt_high);
  const int eq_low = __reduce_add_sync(kAll, n_eq_low), eq_high = __reduce_add_sync(kAll, n_eq_high);
  // Of the entries equal to T the first `need` in index order stay.
  const int eq0 = warps_before<kWarps>(eq_low + eq_high, slots, warp, lane);
  const int eq_stay = min(max(need - eq0, 0), eq_low + eq_high), eq_stay_low = min(eq_stay, eq_low);
  int nh = warps_before<kWarps>(max(0, min(i_hi, left) - i_lo) - gt_low - eq_stay_low, slots, warp,
                                lane);
  int nm = warps_before<kWarps>(gt_high + eq_stay - eq_stay_low, slots, warp, lane);
  int e = eq0;
  const unsigned below_lane = (1u << lane) - 1u;
  // Where an entry below `left` comes from takes the place of its key (its own
  // thread has read that by then); without keys, kept and the front of pos_out serve.
  int* source = KEYS ? reinterpret_cast<int*>(keys) : kept;
  int* list = LIST ? reinterpret_cast<int*>(keys) + cap : pos_out;
  for (int i0 = i_lo; i0 < i_hi; i0 += 128) {
    const int i = i0 + 4 * lane;
    unsigned k[4] = {0u, 0u, 0u, 0u};
    if (i < i_hi) load4(i, k);
    // ranks in index order: lanes below this one, then this lane's entries in turn
    int e_rank = e, h_rank = nh, m_rank = nm;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const unsigned b = __ballot_sync(kAll, i + c < i_hi && k[c] == T);
      e_rank += __popc(b & below_lane);
      e += __popc(b);
    }
    bool hole[4], mover[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const bool in = i + c < i_hi;
      const bool st = in && (k[c] > T || (k[c] == T && e_rank < need));
      e_rank += in && k[c] == T;
      hole[c] = in && i + c < left && !st;
      mover[c] = i + c >= left && st;
    }
    // (the whole warp lies below `left`, or at and behind it, but for one time)
    if (i0 < left)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const unsigned b = __ballot_sync(kAll, hole[c]);
        h_rank += __popc(b & below_lane);
        nh += __popc(b);
      }
    if (i0 + 128 > left)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const unsigned b = __ballot_sync(kAll, mover[c]);
        m_rank += __popc(b & below_lane);
        nm += __popc(b);
      }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      // a hole notes its rank (negative), a mover enters the list
      if (i + c < i_hi && i + c < left) source[i + c] = hole[c] ? ~h_rank : i + c;
      if (mover[c]) list[m_rank] = i + c;
      h_rank += hole[c];
      m_rank += mover[c];
    }
  }
  __syncthreads();
  if constexpr (!LIST) {  // the list gives way to the positions
#pragma unroll 4
    for (int i = threadIdx.x; i < left; i += kThreads)
      if (source[i] < 0) source[i] = list[~source[i]];
    __syncthreads();
  }
#pragma unroll 4
  for (int i = threadIdx.x; i < left; i += kThreads) {
    int k = source[i];
    if (LIST && k < 0) k = list[~k];
    if (KEYS) kept[i] = k;
    mass_out[i] = mass[k];
    pos_out[i] = pos[k];
  }
}

// A warp per 32 entries of kept: copy the rows that moved, k and v.
template <int HD>
__global__ void __launch_bounds__(128) evict_move_kernel(const EvictArgs a, int chunks) {
  constexpr int kVec = HD / 8;  // 16-byte pieces of a row
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long task = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int ch = static_cast<int>(task % chunks);
  const long long sh = task / chunks;
  const int h = static_cast<int>(sh % a.c.n_kv), s = static_cast<int>(sh / a.c.n_kv);
  if (s >= a.c.n_seqs) return;
  const int i0 = ch * 32, i = i0 + lane;
  const int left = min(seq_len(a.c, s, nullptr), a.keep);
  const int from = i < left ? a.kept[sh * a.keep + i] : i;
  unsigned moved = __ballot_sync(kAll, from != i);
  long long src = -1, dst = -1;
  if (from != i) {
    const int p = page_of(a.c, s, from, a.err), q = page_of(a.c, s, i, a.err);
    if (p >= 0 && q >= 0) {
      src = cache_row(a.c, p, h, from) * HD;
      dst = cache_row(a.c, q, h, i) * HD;
    }
  }
  // An entry is 2 kVec pieces of 16 bytes (its rows of k and v): kPer entries
  // per pass of the warp, kU passes loaded before any is stored.
  constexpr int kPer = 32 / (2 * kVec), kU = 8;
  const int sub = lane / (2 * kVec), rest = lane % (2 * kVec);
  __half* pool = (rest < kVec ? a.c.k : a.c.v) + (rest % kVec) * 8;
  while (moved != 0) {
    uint4 x[kU];
    long long to[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      int mine = -1;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (sub == k && moved != 0) mine = __ffs(moved) - 1;
        moved &= moved - 1;
      }
      const long long sr = __shfl_sync(kAll, src, mine < 0 ? 0 : mine);
      const long long ds = __shfl_sync(kAll, dst, mine < 0 ? 0 : mine);
      to[u] = mine >= 0 && sr >= 0 ? ds : -1;
      if (to[u] >= 0) x[u] = *reinterpret_cast<const uint4*>(pool + sr);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (to[u] >= 0) *reinterpret_cast<uint4*>(pool + to[u]) = x[u];
  }
}

template <typename F, typename... Args>
cudaError_t launch_pdl(F* k, long long blocks, int threads, size_t smem, cudaStream_t st,
                       Args... args) {
  if (blocks < 1 || blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

// Keys of up to this many entries stay in shared memory; with the list of the
// movers, at most half as many, two thirds of it.
constexpr long long kKeysMax = 51200;

template <bool LIST>
cudaError_t launch_select(const EvictArgs& a, long long heads, long long smem, cudaStream_t st,
                          int device) {
  static std::atomic<unsigned long long> done{0};
  auto* k = evict_select_kernel<true, LIST>;
  const unsigned long long bit = 1ull << (device & 63);
  if (!(done.load(std::memory_order_relaxed) & bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeysMax * 4);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_relaxed);
  }
  return launch_pdl(k, heads, kThreads, static_cast<size_t>(smem), st, a);
}

}  // namespace

cudaError_t cache_evict_launch(const EvictArgs& a, int sms, cudaStream_t st, int device) {
  const long long heads = static_cast<long long>(a.c.n_seqs) * a.c.n_kv;
  const long long cap = static_cast<long long>(a.c.max_pages) << a.c.page_shift;
  const long long movers = a.keep < cap / 2 ? a.keep : cap / 2;
  const cudaError_t e =
      cap > kKeysMax
          ? launch_pdl(evict_select_kernel<false, false>, heads, kThreads, 0, st, a)
      : heads <= sms && cap + movers <= kKeysMax
          ? launch_select<true>(a, heads, (cap + movers) * 4, st, device)
          : launch_select<false>(a, heads, cap * 4, st, device);
  if (e != cudaSuccess) return e;
  const int chunks = static_cast<int>((min(static_cast<long long>(a.keep), cap) + 31) / 32);
  const long long blocks = (heads * chunks + 3) / 4;
  return a.c.head_dim == 64 ? launch_pdl(evict_move_kernel<64>, blocks, 128, 0, st, a, chunks)
                            : launch_pdl(evict_move_kernel<128>, blocks, 128, 0, st, a, chunks);
}

}  // namespace qgemv
