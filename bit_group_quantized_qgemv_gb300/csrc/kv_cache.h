// kv_cache.h -- argument blocks and launch entry points of the paged-cache
// operators (host and device).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace qgemv {

// The cache as the kernels see it (page_size = 1 << page_shift).
struct KvView {
  __half *k, *v;           // [n_pages][n_kv][page_size][head_dim]
  const int* page_table;   // [n_seqs][max_pages]
  const int* kv_len;       // [n_seqs]
  int n_pages, page_shift, n_kv, head_dim, n_seqs, max_pages;
};

struct RopeArgs {
  KvView c;
  const __half* qkv;
  long long qkv_stride;
  int n_tokens, n_q;
  const int* q_start;
  const int* positions;
  const float* inv_freq;
  int rotary_dim, interleaved;
  const __half *q_norm, *k_norm;
  float eps;
  __half* q_out;
  long long q_stride;
  int* entry_pos;
  float* entry_mass;
  int* err;
};

// A unit of query rows whose entries several blocks share: what their join has
// to know.
struct AttnUnit {
  int parts;  // 0: none
  int s, h, r0, first, rows, off, len;
};

struct AttnArgs {
  KvView c;
  const __half* q;
  long long q_stride;
  int n_tokens, n_q, group;  // group: query heads per key/value head
  const int* q_start;
  int max_q;
  float scale_log2;          // scale * log2(e)
  __half* out;
  long long out_stride;
  float* lse;
  // Results of parts of units, two slots per block: part_o [slot][row][head_dim]
  // (not yet divided by the sum), part_ml [slot][row] {max, sum} in log2 units;
  // splits [block], null: units are not cut.
  float* part_o;
  float2* part_ml;
  AttnUnit* splits;
  int* first_of;  // few rows: [unit] the block with its first part, null: not kept
  unsigned long long group_inv;  // floor(2^64 / group) + 1
  int cluster;  // thread blocks that join their parts among themselves (1: none)
  int* err;
};

struct MassArgs {
  KvView c;
  const __half* q;
  long long q_stride;
  int n_tokens, n_q, group;
  const int* q_start;
  int max_q;
  float scale_log2;
  const float *lse, *mass;
  float* mass_out;
  int* err;
};

struct EvictArgs {
  KvView c;
  const float* mass;
  const int *entry_pos, *next_pos;
  int keep, n_sink, n_recent;
  int* kept;
  float* mass_out;
  int* pos_out;
  int* len_out;
  int* err;
};

cudaError_t rope_append_launch(const RopeArgs& a, int sms, cudaStream_t st);
cudaError_t attention_mass_launch(const MassArgs& a, int sms, cudaStream_t st, int device);
cudaError_t cache_evict_launch(const EvictArgs& a, int sms, cudaStream_t st, int device);

// Whether a call has more query rows per key/value head than the mma.sync
// kernel takes in one pass over the cache: those go to the tcgen05 kernel.  At 24 and 32
// rows, 8 key heads, replayed from a graph, the two kernels take (us)
//   heads of 64,  one of 3000  8.6 and 17.7, 10.0 and 17.4;  of 21000  17.5 and 25.1, 19.9 and 24.6;
//                 four of 3000 to 21000  24.6 and 43.4, 28.5 and 42.5
//   heads of 128, one of 3000 13.3 and 20.0, 18.5 and 19.6;  of 21000  23.9 and 29.4, 33.2 and 28.8;
//                 four of 3000 to 21000  44.0 and 53.0, 56.0 and 51.4
inline bool attention_is_many(int group, int max_q) {
  return static_cast<long long>(group) * max_q > 32;
}
size_t attention_many_bytes(int head_dim, int sms);  // workspace it takes
cudaError_t attention_many_launch(const AttnArgs& a, int sms, cudaStream_t st, int device,
                                  void* workspace, size_t bytes);
cudaError_t status_attention(unsigned* out);
cudaError_t status_mass(unsigned* out);
// Workspace of the kernel for few rows (0: it needs none).
size_t attention_few_bytes(int n_seqs, int n_kv, int rows, int head_dim, long long capacity,
                           int sms);
cudaError_t attention_few_launch(AttnArgs a, int sms, cudaStream_t st, int device, void* workspace,
                                 size_t bytes);

}  // namespace qgemv
