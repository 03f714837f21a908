// attention_mass.cu -- qgemv_attention_mass: the attention weight every
// cached entry receives from the new tokens.
//
//   mass_out[j] = mass[j] + sum_r exp2(scale_log2 q_r . k_j - lse2_r)
// over the rows r = (token, head of the group) that see entry j; lse is known,
// so no softmax statistics are left to carry and every entry is summed on its
// own: a warp keeps 16 entries' keys as A fragments (m16n8k16) and walks the
// rows, eight columns at a time, from shared memory.  The order of the k index
// inside a product is free: thread t of a quad takes the eight components 8t..
// of every 32, one 16-byte load for keys and queries alike.
#include "kv_cache.cuh"

namespace qgemv {
namespace {

constexpr int kWarps = 8;
constexpr int kRowTile = 64;  // query rows staged at a time
constexpr float kLog2e = 1.4426950408889634f;

// Shared-memory stride of a query row, in bytes: 64 more than the row, so
// that the 8 rows x 4 chunks of a load phase fall on different banks.
template <int HD>
__host__ __device__ constexpr int row_stride() {
  return HD * 2 + 64;
}

template <int HD>
__global__ void __launch_bounds__(32 * kWarps) attention_mass_kernel(const MassArgs a,
                                                                     int key_tiles) {
  constexpr int kP = HD / 32;
  __shared__ __align__(16) uint8_t qs[kRowTile * row_stride<HD>()];
  __shared__ float ls[kRowTile];
  __shared__ int lim[kRowTile];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  long long b = blockIdx.x;
  const int kt = static_cast<int>(b % key_tiles);
  b /= key_tiles;
  const int h = static_cast<int>(b % a.c.n_kv);
  const int s = static_cast<int>(b / a.c.n_kv);
  const int len = seq_len(a.c, s, a.err);
  if (kt * 16 * kWarps >= len) return;
  int first, count;
  seq_rows(a.q_start, s, a.n_tokens, a.err, &first, &count);
  if (count > a.max_q) flag_error(a.err);
  const int rows = min(count, a.max_q) * a.group, off = len - count;
  const int e0 = (kt * kWarps + warp) * 16;  // this warp's entries
  const int page = e0 < len ? page_of(a.c, s, e0, a.err) : -1;

  uint4 kf[kP][2];
#pragma unroll
  for (int p = 0; p < kP; ++p)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int j = e0 + g + 8 * e;
      kf[p][e] = page >= 0 && j < len
                     ? *reinterpret_cast<const uint4*>(a.c.k + cache_row(a.c, page, h, j) * HD +
                                                       32 * p + 8 * tq)
                     : make_uint4(0u, 0u, 0u, 0u);
    }
  float sum[2] = {0.f, 0.f};
  // rows whose last entry lies before this block's first see none of it
  const int r_first = max(0, (kt * kWarps * 16 - off) * a.group) / kRowTile * kRowTile;
  for (int rb = r_first; rb < rows; rb += kRowTile) {
    __syncthreads();
    for (int c = threadIdx.x; c < kRowTile * (HD / 8); c += 32 * kWarps) {
      const int r = c / (HD / 8), ch = c % (HD / 8), rr = rb + r;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (rr < rows)
        v = *reinterpret_cast<const uint4*>(a.q + static_cast<long long>(first + rr / a.group) * a.q_stride +
                                            (h * a.group + rr % a.group) * HD + ch * 8);
      *reinterpret_cast<uint4*>(qs + r * row_stride<HD>() + ch * 16) = v;
    }
    for (int r = threadIdx.x; r < kRowTile; r += 32 * kWarps) {
      const int rr = rb + r;
      float v = -INFINITY;
      if (rr < rows)
        v = a.lse[static_cast<long long>(first + rr / a.group) * a.n_q + h * a.group + rr % a.group];
      // a row that saw nothing takes no part
      lim[r] = rr < rows && v != -INFINITY ? off + rr / a.group : -1;
      ls[r] = v * kLog2e;
    }
    __syncthreads();
    if (page < 0) continue;
    for (int n = 0; n < kRowTile && rb + n < rows; n += 8) {
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int p = 0; p < kP; ++p) {
        const uint4 q = *reinterpret_cast<const uint4*>(qs + (n + g) * row_stride<HD>() +
                                                        (4 * p + tq) * 16);
        const uint32_t a0[4] = {kf[p][0].x, kf[p][1].x, kf[p][0].y, kf[p][1].y};
        const uint32_t a1[4] = {kf[p][0].z, kf[p][1].z, kf[p][0].w, kf[p][1].w};
        mma_f16(d, a0, q.x, q.y);
        mma_f16(d, a1, q.z, q.w);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = n + 2 * tq + (e & 1), j = e0 + g + 8 * (e >> 1);
        if (j <= lim[r] && j < len) sum[e >> 1] += ex2(d[e] * a.scale_log2 - ls[r]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], 1);
    sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], 2);
    const int j = e0 + g + 8 * e;
    if (tq == 0 && j < len) {
      const long long at = (static_cast<long long>(s) * a.c.n_kv + h) *
                               (static_cast<long long>(a.c.max_pages) << a.c.page_shift) + j;
      a.mass_out[at] = (a.mass != nullptr ? a.mass[at] : 0.f) + sum[e];
    }
  }
}

template <int HD>
cudaError_t launch_t(const MassArgs& a, cudaStream_t st) {
  const long long cap = static_cast<long long>(a.c.max_pages) << a.c.page_shift;
  const int key_tiles = static_cast<int>((cap + 16 * kWarps - 1) / (16 * kWarps));
  const long long blocks = static_cast<long long>(key_tiles) * a.c.n_kv * a.c.n_seqs;
  if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attention_mass_kernel<HD>, a, key_tiles);
}

}  // namespace

cudaError_t attention_mass_launch(const MassArgs& a, int sms, cudaStream_t st) {
  (void)sms;
  return a.c.head_dim == 64 ? launch_t<64>(a, st) : launch_t<128>(a, st);
}

}  // namespace qgemv
