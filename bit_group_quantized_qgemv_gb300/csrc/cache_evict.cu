// cache_evict.cu -- qgemv_cache_evict: keep the entries of largest mass of
// each (sequence, key/value head) and close the gaps.
//
// Selection: one block per (sequence, head).  Masses become 32-bit keys whose
// order is the ranking (protected entries highest, NaN lowest); the keep-th
// largest key T is found by radix selection, eight bits at a time, and the
// lowest-index entries equal to T fill up what is missing.  Every warp owns a
// run of consecutive entries, so ranks in index order are prefix sums over
// the warps' counts.  The movers' list is written to the front of pos_out
// first (it is at most as long as what pos_out gets in the end), the holes
// pick their mover from it, and only then the permuted masses and positions
// are written.
// Moving: a second kernel copies the rows of k and v whose place changed.
// Sources lie at or beyond the new length and targets below it, so no copy
// reads what another writes.
#include "kv_cache.cuh"

namespace qgemv {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kAll = 0xFFFFFFFFu;

// Larger key: kept first.  Equal masses (-0 and +0 too) have equal keys.
__device__ __forceinline__ unsigned rank_key(float mass, int pos, int sink, long long recent) {
  if (pos < sink || pos >= recent) return kAll;
  if (mass != mass) return 0u;
  const unsigned b = __float_as_uint(mass == 0.f ? 0.f : mass);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Sums of the warps below this one, and the total over the block.
__device__ __forceinline__ int warps_before(int mine, int* slots, int warp, int lane, int* total) {
  __syncthreads();
  if (lane == 0) slots[warp] = mine;
  __syncthreads();
  int v = slots[lane];
  int below = lane < warp ? v : 0;
#pragma unroll
  for (int k = 16; k > 0; k /= 2) {
    v += __shfl_xor_sync(kAll, v, k);
    below += __shfl_xor_sync(kAll, below, k);
  }
  *total = v;
  return below;
}

__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int slots[kWarps];
  __shared__ unsigned s_prefix;
  __shared__ int s_left;
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.x % a.c.n_kv, s = blockIdx.x / a.c.n_kv;
  const int len = seq_len(a.c, s, a.err);
  const int left = min(len, a.keep);
  const long long cap = static_cast<long long>(a.c.max_pages) << a.c.page_shift;
  const long long base = (static_cast<long long>(s) * a.c.n_kv + h) * cap;
  const float* mass = a.mass + base;
  const int* pos = a.entry_pos + base;
  float* mass_out = a.mass_out + base;
  int* pos_out = a.pos_out + base;
  int* kept = a.kept + (static_cast<long long>(s) * a.c.n_kv + h) * a.keep;
  const long long recent = static_cast<long long>(a.next_pos[s]) - a.n_recent;
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

  // T: the left-th largest key; s_left: how many of the entries equal to it stay
  unsigned prefix = 0;
  int need = left;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += kThreads) hist[i] = 0;
    __syncthreads();
    const unsigned above = shift == 24 ? 0u : kAll << (shift + 8);
    for (int i0 = warp * 32; i0 < len; i0 += kThreads) {
      const int i = i0 + lane;
      unsigned key = 0;
      bool in = i < len;
      if (in) {
        key = rank_key(mass[i], pos[i], a.n_sink, recent);
        in = (key & above) == prefix;
      }
      const unsigned bin = in ? (key >> shift) & 255u : 256u;
      const unsigned same = __match_any_sync(kAll, bin);
      if (in && lane == __ffs(same) - 1) atomicAdd(&hist[bin], __popc(same));
    }
    __syncthreads();
    if (warp == 0) {  // the bin in which the need-th largest lies
      int c[8], sum = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        c[k] = hist[255 - (lane * 8 + k)];
        sum += c[k];
      }
      int incl = sum;
#pragma unroll
      for (int k = 1; k < 32; k *= 2) {
        const int v = __shfl_up_sync(kAll, incl, k);
        if (lane >= k) incl += v;
      }
      int run = incl - sum;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (run < need && run + c[k] >= need) {
          s_prefix = prefix | (static_cast<unsigned>(255 - (lane * 8 + k)) << shift);
          s_left = need - run;
        }
        run += c[k];
      }
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_left;
  }
  const unsigned T = prefix;

  // Runs of whole 32-entry groups per warp, in index order.
  const int groups = (len + 31) / 32, per = (groups + kWarps - 1) / kWarps;
  const int i_lo = warp * per * 32, i_hi = min(len, (warp + 1) * per * 32);
  auto key_at = [&](int i) { return rank_key(mass[i], pos[i], a.n_sink, recent); };
  int eq = 0;
  for (int i0 = i_lo; i0 < i_hi; i0 += 32) {
    const int i = i0 + lane;
    eq += __popc(__ballot_sync(kAll, i < i_hi && key_at(i) == T));
  }
  int total;
  const int eq0 = warps_before(eq, slots, warp, lane, &total);
  const unsigned below_lane = (1u << lane) - 1u;
  int holes = 0, movers = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int e = eq0, nh = holes, nm = movers;  // second pass: ranks of this warp's first
    if (pass == 0) nh = nm = 0;
    for (int i0 = i_lo; i0 < i_hi; i0 += 32) {
      const int i = i0 + lane;
      const unsigned key = i < i_hi ? key_at(i) : 0u;
      const bool is_eq = i < i_hi && key == T;
      const unsigned eqs = __ballot_sync(kAll, is_eq);
      const bool stays = i < i_hi && (key > T || (is_eq && e + __popc(eqs & below_lane) < need));
      e += __popc(eqs);
      const unsigned hb = __ballot_sync(kAll, i < i_hi && i < left && !stays);
      const unsigned mb = __ballot_sync(kAll, i < i_hi && i >= left && stays);
      if (pass == 1) {
        // a hole notes its rank (negative), a mover enters the list
        if (i < i_hi && i < left) kept[i] = stays ? i : ~(nh + __popc(hb & below_lane));
        if ((mb >> lane) & 1u) pos_out[nm + __popc(mb & below_lane)] = i;
      }
      nh += __popc(hb);
      nm += __popc(mb);
    }
    if (pass == 0) {
      holes = warps_before(nh, slots, warp, lane, &total);
      movers = warps_before(nm, slots, warp, lane, &total);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < left; i += kThreads) {
    const int k = kept[i];
    if (k < 0) kept[i] = pos_out[~k];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < left; i += kThreads) {
    const int k = kept[i];
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
  // two rows (k and v of one entry) at a time: half a warp each when HD = 128
  constexpr int kPer = 32 / (2 * kVec);
  while (moved != 0) {
    int at[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      at[k] = moved != 0 ? __ffs(moved) - 1 : -1;
      moved &= moved - 1;
    }
    const int sub = lane / (2 * kVec), rest = lane % (2 * kVec);
    int mine = at[0];
#pragma unroll
    for (int k = 1; k < kPer; ++k) mine = sub == k ? at[k] : mine;
    const long long sr = __shfl_sync(kAll, src, mine < 0 ? 0 : mine);
    const long long ds = __shfl_sync(kAll, dst, mine < 0 ? 0 : mine);
    if (mine >= 0 && sr >= 0) {
      __half* pool = rest < kVec ? a.c.k : a.c.v;
      const int piece = (rest % kVec) * 8;
      *reinterpret_cast<uint4*>(pool + ds + piece) =
          *reinterpret_cast<const uint4*>(pool + sr + piece);
    }
  }
}

template <typename F, typename... Args>
cudaError_t launch_pdl(F* k, long long blocks, int threads, cudaStream_t st, Args... args) {
  if (blocks < 1 || blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

}  // namespace

cudaError_t cache_evict_launch(const EvictArgs& a, int sms, cudaStream_t st) {
  (void)sms;
  const long long heads = static_cast<long long>(a.c.n_seqs) * a.c.n_kv;
  cudaError_t e = launch_pdl(evict_select_kernel, heads, kThreads, st, a);
  if (e != cudaSuccess) return e;
  const int chunks = (a.keep + 31) / 32;
  const long long blocks = (heads * chunks + 3) / 4;
  return a.c.head_dim == 64 ? launch_pdl(evict_move_kernel<64>, blocks, 128, st, a, chunks)
                            : launch_pdl(evict_move_kernel<128>, blocks, 128, st, a, chunks);
}

}  // namespace qgemv
