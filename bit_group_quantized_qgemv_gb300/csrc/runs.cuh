// runs.cuh -- equal shares of ragged work: every (sequence, head) unit has a
// number of blocks of entries that depends on its length, all units are laid end
// to end (by sequence, then by head), and every thread block takes a run of the
// same length.  Found from the lengths on the device, so it does not depend on how
// wide the page table is.
#pragma once

#include <stdint.h>

namespace qgemv {

// What a / b is, in 32 bits where that is enough.
__device__ __forceinline__ long long run_div(long long a, long long b) {
  return (a | b) >> 31 == 0 ? static_cast<long long>(static_cast<unsigned>(a) / static_cast<unsigned>(b))
                            : a / b;
}

__device__ __forceinline__ long long run_scan(long long v, int lane) {
#pragma unroll
  for (int k = 1; k < 32; k *= 2) {
    const long long w = __shfl_up_sync(0xFFFFFFFFu, v, k);
    if (lane >= k) v += w;
  }
  return v;
}

// This thread block's run of the blocks of all units (blocks(s) of each of
// n_kv heads of sequence s): where it starts, its length (0: none) and the length of
// everyone's, least or more.  A whole warp.
template <typename F>
__device__ __forceinline__ long long run_start(int n_seqs, int n_kv, int least, int lane, F blocks,
                                               long long* per, int* s, int* h, int* j) {
  int b = lane < n_seqs ? blocks(lane) : 0;  // sequence `lane` of the 32 at hand
  // Few sequences: the same in 32 bits (the sums stay below 2^30).
  if (n_seqs <= 32 && __all_sync(0xFFFFFFFFu, b <= (1 << 25) / n_kv)) {
    const int mine = b * n_kv, all = __reduce_add_sync(0xFFFFFFFFu, mine);
    const int share = max(least, static_cast<int>((static_cast<unsigned>(all) + gridDim.x - 1) / gridDim.x));
    *per = share;
    const long long at = static_cast<long long>(blockIdx.x) * share;
    if (at >= all) return 0;
    int pos = static_cast<int>(at), each = b;
    *s = 0;
    if (n_seqs > 1) {
      int incl = mine;
#pragma unroll
      for (int k = 1; k < 32; k *= 2) {
        const int w = __shfl_up_sync(0xFFFFFFFFu, incl, k);
        if (lane >= k) incl += w;
      }
      const int l = __ffs(__ballot_sync(0xFFFFFFFFu, pos < incl)) - 1;
      const int left = min(share, all - pos);
      pos -= __shfl_sync(0xFFFFFFFFu, incl - mine, l);
      each = __shfl_sync(0xFFFFFFFFu, b, l);
      *s = l;
      *h = pos / each;
      *j = pos - *h * each;
      return left;
    }
    each = __shfl_sync(0xFFFFFFFFu, b, 0);
    *h = pos / each;
    *j = pos - *h * each;
    return min(share, all - pos);
  }
  long long all = static_cast<long long>(b) * n_kv;
  for (int i = lane + 32; i < n_seqs; i += 32) all += static_cast<long long>(blocks(i)) * n_kv;
#pragma unroll
  for (int k = 16; k > 0; k /= 2) all += __shfl_xor_sync(0xFFFFFFFFu, all, k);
  const long long share = run_div(all + gridDim.x - 1, gridDim.x);
  *per = share > least ? share : least;
  long long pos = blockIdx.x * *per;
  if (pos >= all) return 0;
  const long long mine_of = all - pos < *per ? all - pos : *per;
  for (int s0 = 0; s0 < n_seqs; s0 += 32) {
    if (s0 > 0) b = s0 + lane < n_seqs ? blocks(s0 + lane) : 0;
    const long long mine = static_cast<long long>(b) * n_kv, incl = run_scan(mine, lane);
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, pos < incl);
    if (hit == 0) {
      pos -= __shfl_sync(0xFFFFFFFFu, incl, 31);
      continue;
    }
    const int l = __ffs(hit) - 1;
    const long long rest = pos - __shfl_sync(0xFFFFFFFFu, incl - mine, l);
    const int each = __shfl_sync(0xFFFFFFFFu, b, l);
    *s = s0 + l;
    *h = static_cast<int>(run_div(rest, each));
    *j = static_cast<int>(rest - static_cast<long long>(*h) * each);
    return mine_of;
  }
  return 0;
}

// Blocks of all units, and the unit and block at position pos < that.  A whole
// warp.
template <typename F>
__device__ __forceinline__ long long run_total(int n_seqs, int n_kv, int lane, F blocks) {
  long long t = 0;
  for (int i = lane; i < n_seqs; i += 32) t += blocks(i);
#pragma unroll
  for (int k = 16; k > 0; k /= 2) t += __shfl_xor_sync(0xFFFFFFFFu, t, k);
  return t * n_kv;
}
template <typename F>
__device__ __forceinline__ void run_seek(long long pos, int n_seqs, int n_kv, int lane, F blocks,
                                         int* s, int* h, int* j) {
  *s = *h = *j = 0;
  for (int s0 = 0; s0 < n_seqs; s0 += 32) {
    const int b = s0 + lane < n_seqs ? blocks(s0 + lane) : 0;
    const long long mine = static_cast<long long>(b) * n_kv, incl = run_scan(mine, lane);
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, pos < incl);
    if (hit == 0) {
      pos -= __shfl_sync(0xFFFFFFFFu, incl, 31);
      continue;
    }
    const int l = __ffs(hit) - 1;
    const long long rest = pos - __shfl_sync(0xFFFFFFFFu, incl - mine, l);
    const int each = __shfl_sync(0xFFFFFFFFu, b, l);
    *s = s0 + l;
    *h = static_cast<int>(run_div(rest, each));
    *j = static_cast<int>(rest - static_cast<long long>(*h) * each);
    return;
  }
}

// The next sequence behind s with blocks; n_seqs if there is none.  A whole warp.
template <typename F>
__device__ __forceinline__ int run_next(int s, int n_seqs, int lane, F blocks) {
  for (int s0 = s + 1; s0 < n_seqs; s0 += 32) {
    const unsigned hit =
        __ballot_sync(0xFFFFFFFFu, s0 + lane < n_seqs && blocks(s0 + lane) > 0);
    if (hit != 0) return s0 + __ffs(hit) - 1;
  }
  return n_seqs;
}

}  // namespace qgemv
