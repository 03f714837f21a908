// kv_tensor_map.h -- tensor maps of the cache's pools (host only).
#pragma once

#include "kv_cache.h"
#include "tensor_map.h"

namespace qgemv {

// Map of a pool as rows of HD values, boxes of 64 columns and up to 128 rows.
inline bool encode_pool(CUtensorMap* m, const KvView& c, const __half* pool) {
  const EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const int page = 1 << c.page_shift;
  const cuuint64_t dim[2] = {static_cast<cuuint64_t>(c.head_dim),
                             static_cast<cuuint64_t>(c.n_pages) * c.n_kv * page};
  const cuuint64_t stride[1] = {static_cast<cuuint64_t>(c.head_dim) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(page < 128 ? page : 128)};
  const cuuint32_t estride[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<__half*>(pool), dim, stride, box,
            estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace qgemv
