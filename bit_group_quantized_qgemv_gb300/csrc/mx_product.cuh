// mx_product.cuh -- what the kernels of the MXFP4 products share.
#pragma once

#include <atomic>

#include "kv_cache.cuh"
#include "mma_tile.cuh"
#include "mx.h"
#include "mx_format.cuh"
#include "mx_plan.h"
#include "tcgen05.cuh"
#include "tensor_map.h"

namespace qgemv {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
// A value to another block's shared memory, its bytes counted on a barrier there.
__device__ __forceinline__ void send(uint32_t addr, float v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr),
               "r"(__float_as_uint(v)), "r"(bar)
               : "memory");
}
// (relaxed: the barriers' initialisation has a fence of its own)
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

__device__ __forceinline__ void store_shared(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// silu(z) = z / (1 + e^-z), for z below 0 as z e^z / (1 + e^z): the divisor is between 1 and 2, and
// small results are held for as long as fp32 holds e^z.  By the fast exponential and division:
// 2^-20 of the result off, for z below 0 |z| 2^-22 of it more (there the result is small against z
// and its error, that of a sum of products), and |z| 2^-149 where e^z is subnormal.
// The exact division's branches take a thread's columns one after the other, longer than all
// else of the results: gated 1024 rows of 1024 to 2816 19.1 us for 14.5, 2048 rows of 4096 to 14336
// 169 for 148 in the same tiles (clocks at 1.7 GHz).  Of the latter's 29.4 million MXFP8 codes 37
// differ from those of 64-bit sums and silu; of a plain fp32 form's 28 to 34.
__device__ __forceinline__ float mx_silu(float z) {
  const float e = __expf(-fabsf(z));
  return __fdividef(z < 0.f ? z * e : z, 1.0f + e);
}

// Finished values of weight row n (a lane each) and rows m, m + 1, ... of x, count of them, to
// y and, of the gated product, to the codes and scales.  A whole warp calls this.
template <bool GATED, int C>
__device__ __forceinline__ void write_results(const MxProductArgs& a, int n, int m, int count, const float (&v)[C],
                                              int lane) {
  const bool live = n < a.N;
  const long long at = static_cast<long long>(m) * a.N + n;
  if (a.y != nullptr && live) {
    __half* y = a.y + at;
#pragma unroll
    for (int c = 0; c < C; ++c, y += a.N)
      if (c < count) *y = __float2half_rn(v[c]);
  }
  if constexpr (GATED) {
    if (a.yc == nullptr) return;
    // (N is a multiple of 32: a warp's rows are one block of the output, all there or none)
    int byte[C];
#pragma unroll
    for (int c = 0; c < C; ++c)
      byte[c] = mx_scale_byte<8>(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v[c]) & 0x7FFFFFFFu)));
    if constexpr (C % 4 == 0) {
      // Four columns' codes of four lanes' rows change places: a lane then has four rows of
      // one column, and a warp's store 32 bytes of each of four.
      const int sub = lane & 3;
      uint8_t* to = a.yc + static_cast<long long>(m + sub) * a.N + (n & ~3);
#pragma unroll
      for (int c = 0; c < C; c += 4, to += 4LL * a.N) {
        uint32_t w = mx_codes8(v[c] * mx_inverse(byte[c]), v[c + 1] * mx_inverse(byte[c + 1])) |
                     (mx_codes8(v[c + 2] * mx_inverse(byte[c + 2]), v[c + 3] * mx_inverse(byte[c + 3])) << 16);
        uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, w, 1);
        w = sub & 1 ? __byte_perm(o, w, 0x7351) : __byte_perm(w, o, 0x6240);
        o = __shfl_xor_sync(0xFFFFFFFFu, w, 2);
        w = sub & 2 ? __byte_perm(o, w, 0x7632) : __byte_perm(w, o, 0x5410);
        if (live && c + sub < count) *reinterpret_cast<uint32_t*>(to) = w;
      }
    } else if (live) {
      a.yc[at] = static_cast<uint8_t>(mx_codes8(v[0] * mx_inverse(byte[0]), 0.f));
    }
    if (!live) return;
    // lane c has the scale of row m + c
    int mine = byte[0];
#pragma unroll
    for (int c = 1; c < C; ++c) mine = lane == c ? byte[c] : mine;
    if (lane < C && lane < count)
      a.ys[static_cast<long long>(m + lane) * (a.N / kMxBlock) + n / kMxBlock] = static_cast<uint8_t>(mine);
  }
}

// All shared memory for a kernel, allowed once per device.
template <auto* kKernel>
cudaError_t allow_smem(int device) {
  static std::atomic<unsigned long long> done{0};
  const unsigned long long bit = 1ull << (device & 63);
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMxSmem);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Clusters of 1 << log2 blocks of a kernel that the device runs at a time (0 where it cannot).
template <auto* kKernel>
int clusters_at_a_time(int log2, int threads, int sms, int device) {
  static MxClusterTable table;
  if (log2 == 0) return sms;
  return table.get(log2, device, [&](int* n) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(sms >> log2 << log2));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = kMxSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << log2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (allow_smem<kKernel>(device) == cudaSuccess && cudaOccupancyMaxActiveClusters(n, kKernel, &cfg) == cudaSuccess)
      return true;
    cudaGetLastError();
    return false;
  });
}

// Products by pairs of thread blocks (mx_pair.cu): how many pairs run at a time, whether the
// call's K and addresses allow them, and the launch of a plan on up to `clusters` pairs.
int mx_pair_clusters(bool gated, int sms, int device);
bool mx_pair_takes(const MxProductArgs& a);
cudaError_t mx_pair_launch(const MxProductArgs& a, const MxPairPlan& p, int clusters, int device, cudaStream_t st);
cudaError_t status_mx_pair(unsigned* out);

// Tensor map of rows of codes, boxes of 128 k.
inline bool encode_codes(CUtensorMap* m, const void* p, bool four, long long rows, int k, int box_rows) {
  const EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dim[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows)};
  const cuuint64_t stride[1] = {static_cast<cuuint64_t>(four ? k / 2 : k)};
  const cuuint32_t box[2] = {kMxStep, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estride[2] = {1, 1};
  return fn(m, four ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
            const_cast<void*>(p), dim, stride, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace qgemv
