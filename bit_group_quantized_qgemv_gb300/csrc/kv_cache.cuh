// kv_cache.cuh -- device-side helpers shared by the paged-cache kernels.
#pragma once

#include "kv_cache.h"
#include "qgemv_device.cuh"

namespace qgemv {

__device__ __forceinline__ void flag_error(int* err) {
  if (err != nullptr) *err = 1;
}

// Entries of sequence s, clamped to what its page-table row can hold.
__device__ __forceinline__ int seq_len(const KvView& c, int s, int* err) {
  const int n = c.kv_len[s], cap = c.max_pages << c.page_shift;
  if (n < 0 || n > cap) flag_error(err);
  return min(max(n, 0), cap);
}

// First row and number of new tokens of sequence s.
__device__ __forceinline__ void seq_rows(const int* q_start, int s, int n_tokens, int* err,
                                         int* first, int* count) {
  const int a = q_start[s], b = q_start[s + 1];
  if (a < 0 || b < a || b > n_tokens) flag_error(err);
  const int a0 = min(max(a, 0), n_tokens), b0 = min(max(b, a0), n_tokens);
  *first = a0;
  *count = b0 - a0;
}

// Checks of sequence s that a kernel which meets only some sequences makes for all.
__device__ __forceinline__ void check_seq(const KvView& c, const int* q_start, int s, int n_tokens,
                                          int* err) {
  int first, count;
  seq_rows(q_start, s, n_tokens, err, &first, &count);
  seq_len(c, s, err);
}

// Page-table entry for entry i of sequence s, as it stands there.  Loops load it
// a step ahead and look at it (good_page) when they need it: a look right after
// the load would wait for it.
__device__ __forceinline__ int raw_page(const KvView& c, int s, int i) {
  return c.page_table[static_cast<long long>(s) * c.max_pages + (i >> c.page_shift)];
}

// A page number, -1 for a bad one.
__device__ __forceinline__ int good_page(const KvView& c, int p, int* err) {
  if (p >= 0 && p < c.n_pages) return p;
  flag_error(err);
  return -1;
}

__device__ __forceinline__ int page_of(const KvView& c, int s, int i, int* err) {
  return good_page(c, raw_page(c, s, i), err);
}

// Row of entry i on page p for head h, as a row index into k or v.
__device__ __forceinline__ long long cache_row(const KvView& c, int p, int h, int i) {
  return ((static_cast<long long>(p) * c.n_kv + h) << c.page_shift) +
         (i & ((1 << c.page_shift) - 1));
}

// Limit of the waits: what a warp may have to do meanwhile (slow_row) is as long
// as a cache.
constexpr uint64_t kWaitNs = 10000000000ull;

// A bounded wait of a whole warp: every lane gets the same answer, so a wait
// that runs out does not split the warp.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, unsigned* status) {
  return __all_sync(0xFFFFFFFFu, mbar_wait_for(bar, parity, status, kWaitNs));
}

// A bounded wait that answers nothing, for loops whose steps are short: there
// an answer to test at every wait, or to carry along, cost a seventh of the time
// (measured on GB300: 448 against 387 us for 1216 tokens over 30000 entries).  A
// wait of more than kWaitNs sets *failed (in shared memory), after which the
// block's waits last for a thousand tries: its loops go on over whatever they
// find, in bounds and for as many steps as they have, and the results are
// dropped.  CLUSTER: other blocks of the cluster have a part in the phase.
template <bool CLUSTER = false>
__device__ __forceinline__ void step_wait(uint32_t bar, uint32_t parity, volatile int* failed,
                                          unsigned* status) {
  auto look = [&] { return CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
  bool done = look();
  uint64_t t0 = 0;
  for (int i = 1; !done; ++i) {
    done = look();
    if ((i & 1023) == 0) {
      if (*failed != 0) break;
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > kWaitNs) {
        *failed = 1;
        atomicOr(status, kStatusWaitTimeout);
        break;
      }
    }
  }
  if (CLUSTER) mbar_acquire_cluster();
  __syncwarp();
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two floats in a register pair, for instructions that take both: the softmax
// of many rows is bound by the instructions it issues.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// D += A B, 16 x 8 x 16, fp16 operands, fp32 accumulator.
__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace qgemv
