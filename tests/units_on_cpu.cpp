// How the many-rows attention kernel shares out its work (attention_units.cuh), run
// on the CPU: a warp is 32 contexts that meet at every warp-wide exchange.
//   stdin:  cases of  blocks n_kv group max_q cut n_seqs, then n_seqs pairs
//           (new tokens, length)
//   stdout: per case the segments "g block s h r0 rows off j0 j1 slot", the cut units
//           "u block parts s h r0", and "end"
#include <ucontext.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <functional>
#include <vector>

#define __device__
#define __host__
#define __forceinline__ inline

namespace {

struct Dim {
  unsigned x;
} gridDim, blockIdx;

constexpr int kLanes = 32;
constexpr size_t kStack = 1 << 17;
ucontext_t home, lanes[kLanes];
std::vector<char> stacks(kLanes* kStack);
int lane_now, met[kLanes];           // what each lane waits in: 0 nothing, -1 it has ended
int phase[kLanes];
long long values[2][kLanes];
std::function<void(int)> work;

void enter() {
  work(lane_now);
  met[lane_now] = -1;
  swapcontext(&lanes[lane_now], &home);
}

void run_warp(std::function<void(int)> f) {
  work = std::move(f);
  for (int l = 0; l < kLanes; ++l) {
    getcontext(&lanes[l]);
    lanes[l].uc_stack.ss_sp = &stacks[l * kStack];
    lanes[l].uc_stack.ss_size = kStack;
    lanes[l].uc_link = &home;
    makecontext(&lanes[l], enter, 0);
    met[l] = phase[l] = 0;
  }
  while (met[0] != -1) {
    for (lane_now = 0; lane_now < kLanes; ++lane_now) swapcontext(&home, &lanes[lane_now]);
    for (int l = 1; l < kLanes; ++l)
      if (met[l] != met[0]) {
        std::printf("lanes apart: %d in %d, 0 in %d\n", l, met[l], met[0]);
        std::exit(1);
      }
  }
}

// Every lane's value, once all have come to the same exchange.
const long long* meet(int kind, long long v) {
  const int l = lane_now;
  long long* all = values[phase[l]++ & 1];
  all[l] = v;
  met[l] = kind;
  swapcontext(&lanes[l], &home);
  return all;
}

using std::max;
using std::min;
template <typename T>
T __shfl_sync(unsigned, T v, int from) {
  return static_cast<T>(meet(1, v)[from & 31]);
}
template <typename T>
T __shfl_up_sync(unsigned, T v, int by) {
  const int l = lane_now;
  return static_cast<T>(meet(2, v)[l >= by ? l - by : l]);
}
template <typename T>
T __shfl_xor_sync(unsigned, T v, int mask) {
  const int l = lane_now;
  return static_cast<T>(meet(3, v)[l ^ mask]);
}
unsigned __ballot_sync(unsigned, bool p) {
  const long long* a = meet(4, p);
  unsigned r = 0;
  for (int i = 0; i < kLanes; ++i) r |= static_cast<unsigned>(a[i] != 0) << i;
  return r;
}
// (sums of 32 bits, as the GPU's)
template <typename T>
T __reduce_add_sync(unsigned, T v) {
  const long long* a = meet(5, v);
  uint32_t r = 0;
  for (int i = 0; i < kLanes; ++i) r += static_cast<uint32_t>(a[i]);
  return static_cast<T>(r);
}
template <typename T>
T __reduce_max_sync(unsigned, T v) {
  const long long* a = meet(6, v);
  return static_cast<T>(*std::max_element(a, a + kLanes));
}
template <typename T>
T __reduce_min_sync(unsigned, T v) {
  const long long* a = meet(7, v);
  return static_cast<T>(*std::min_element(a, a + kLanes));
}
void __syncwarp() { meet(8, 0); }
int __ffs(unsigned v) { return __builtin_ffs(static_cast<int>(v)); }
unsigned long long __umul64hi(unsigned long long a, unsigned long long b) {
  return static_cast<unsigned long long>((static_cast<unsigned __int128>(a) * b) >> 64);
}

}  // namespace

namespace qgemv {

// What the header needs of kv_cache.h and kv_cache.cuh.
struct KvView {
  const int* kv_len;
  int n_kv, n_seqs;
};
struct AttnUnit {
  int parts, s, h, r0, first, rows, off, len;
};
struct AttnArgs {
  KvView c;
  const int* q_start;
  int n_tokens, max_q, group;
  unsigned long long group_inv;
  AttnUnit* splits;
  int* err;
};
inline void flag_error(int*) {}
inline void seq_rows(const int* q_start, int s, int, int*, int* first, int* count) {
  *first = q_start[s];
  *count = q_start[s + 1] - q_start[s];
}
inline int seq_len(const KvView& c, int s, int*) { return c.kv_len[s]; }

}  // namespace qgemv

#include "attention_units.cuh"

int main() {
  using namespace qgemv;
  int blocks, n_kv, group, max_q, cut, n_seqs;
  while (std::scanf("%d %d %d %d %d %d", &blocks, &n_kv, &group, &max_q, &cut, &n_seqs) == 6) {
    std::vector<int> start(n_seqs + 1, 0), len(n_seqs);
    for (int s = 0; s < n_seqs; ++s) {
      if (std::scanf("%d %d", &start[s + 1], &len[s]) != 2) return 1;
      start[s + 1] += start[s];
    }
    gridDim.x = blocks;
    for (blockIdx.x = 0; blockIdx.x < gridDim.x; ++blockIdx.x) {
      AttnUnit dummy, mine[kLanes];
      const AttnArgs a{{len.data(), n_kv, n_seqs}, start.data(), start[n_seqs], max_q, group,
                       ~0ull / static_cast<unsigned>(group) + 1, cut ? &dummy : nullptr, nullptr};
      int span[kMaxBlocks], load[kMaxBlocks];
      uint8_t order[kMaxBlocks];
      run_warp([&](int lane) {
        Scheduler sc(a, lane);
        auto emit = [&](bool, int j0, int j1, int slot) {
          if (lane == 0)
            std::printf("g %u %d %d %d %d %d %d %d %d\n", blockIdx.x, sc.s, sc.h, sc.rt * kUnitRows,
                        sc.rows, sc.len - sc.count, j0, j1, slot);
          __syncwarp();
        };
        mine[lane] = hand_out(a, sc, lane, span, load, order, emit);
      });
      if (mine[0].parts > 0)
        std::printf("u %u %d %d %d %d\n", blockIdx.x, mine[0].parts, mine[0].s, mine[0].h, mine[0].r0);
    }
    std::printf("end\n");
  }
  return 0;
}
