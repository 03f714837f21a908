// capi_cache.cu -- the extern "C" boundary of the paged-cache operators
// (declared in include/qgemv.h).  Host code only: checks the arguments and
// enqueues the kernels on the caller's stream.
#include <stdint.h>

#include <cmath>

#include "kv_cache.h"
#include "qgemv.h"

namespace qgemv {
// capi.cu
int report_launch(cudaError_t e);
int device_and_sms(int* dev, int* sms);
}  // namespace qgemv

namespace {

using qgemv::KvView;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_cache(const qgemv_kv_cache* c, KvView* v) {
  if (!c || !c->k || !c->v || !c->page_table || !c->kv_len) return QGEMV_ENULL;
  int shift = 4;
  while (shift < 8 && (1 << shift) != c->page_size) ++shift;
  if ((1 << shift) != c->page_size || (c->head_dim != 64 && c->head_dim != 128) ||
      c->n_pages < 1 || c->n_kv < 1 || c->n_kv > 1024 || c->n_seqs < 1 || c->n_seqs > 65535 ||
      c->max_pages < 1)
    return QGEMV_EINVAL;
  if (static_cast<long long>(c->max_pages) * c->page_size > 1LL << 29 ||
      static_cast<long long>(c->n_pages) * c->n_kv > 0x7FFFFFFFLL / c->page_size)
    return QGEMV_EINVAL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->page_table, 4) ||
      !aligned(c->kv_len, 4))
    return QGEMV_EALIGN;
  v->k = reinterpret_cast<__half*>(c->k);
  v->v = reinterpret_cast<__half*>(c->v);
  v->page_table = c->page_table;
  v->kv_len = c->kv_len;
  v->n_pages = c->n_pages;
  v->page_shift = shift;
  v->n_kv = c->n_kv;
  v->head_dim = c->head_dim;
  v->n_seqs = c->n_seqs;
  v->max_pages = c->max_pages;
  return QGEMV_OK;
}

constexpr float kLog2e = 1.4426950408889634f;

// Query-side shape: n_q a multiple of n_kv, the rows of a sequence countable in
// 30 bits.
int check_queries(const KvView& c, long long q_stride, int n_tokens, int n_q, int max_q,
                  float scale) {
  if (n_tokens < 0 || n_q < 1 || n_q % c.n_kv != 0 || n_q > 65535 || max_q < 1 ||
      max_q > 1 << 24 || !(scale > 0.0f) || !std::isfinite(scale * kLog2e))
    return QGEMV_EINVAL;
  if (q_stride < static_cast<long long>(n_q) * c.head_dim || q_stride % 8 != 0)
    return QGEMV_EINVAL;
  const long long rows = static_cast<long long>(max_q) * (n_q / c.n_kv);
  if (rows > 0x3FFFFFFFLL) return QGEMV_EINVAL;
  return QGEMV_OK;
}

}  // namespace

extern "C" {

int qgemv_qk_norm_rope_append(const qgemv_kv_cache* cache, const uint16_t* qkv,
                              long long qkv_stride, int n_tokens, int n_q, const int32_t* q_start,
                              const int32_t* positions, const float* inv_freq, int rotary_dim,
                              int interleaved, const uint16_t* q_norm, const uint16_t* k_norm,
                              float eps, uint16_t* q_out, long long q_stride, int32_t* entry_pos,
                              float* entry_mass, int* err_flag, void* stream) {
  qgemv::RopeArgs a{};
  if (int rc = check_cache(cache, &a.c)) return rc;
  if (!q_start || (n_tokens != 0 && (!qkv || !positions || !q_out)) || (rotary_dim > 0 && !inv_freq))
    return QGEMV_ENULL;
  if ((q_norm == nullptr) != (k_norm == nullptr)) return QGEMV_ENULL;
  const int hd = a.c.head_dim;
  if (n_tokens < 0 || n_q < 1 || n_q > 65535 || n_q % a.c.n_kv != 0 || rotary_dim < 0 ||
      rotary_dim > hd || rotary_dim % 8 != 0 ||
      qkv_stride < (static_cast<long long>(n_q) + 2 * a.c.n_kv) * hd || qkv_stride % 4 != 0 ||
      q_stride < static_cast<long long>(n_q) * hd || q_stride % 4 != 0 ||
      (q_norm && (!(eps > 0.0f) || !std::isfinite(eps))))
    return QGEMV_EINVAL;
  if (!aligned(qkv, 8) || !aligned(q_out, 8) || !aligned(q_norm, 8) || !aligned(k_norm, 8) ||
      !aligned(q_start, 4) || !aligned(positions, 4) || !aligned(inv_freq, 4) ||
      !aligned(entry_pos, 4) || !aligned(entry_mass, 4) || !aligned(err_flag, 4))
    return QGEMV_EALIGN;
  if (n_tokens == 0) return QGEMV_OK;
  int dev, sms;
  if (int rc = qgemv::device_and_sms(&dev, &sms)) return rc;
  a.qkv = reinterpret_cast<const __half*>(qkv);
  a.qkv_stride = qkv_stride;
  a.n_tokens = n_tokens;
  a.n_q = n_q;
  a.q_start = q_start;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.rotary_dim = rotary_dim;
  a.interleaved = interleaved != 0;
  a.q_norm = reinterpret_cast<const __half*>(q_norm);
  a.k_norm = reinterpret_cast<const __half*>(k_norm);
  a.eps = eps;
  a.q_out = reinterpret_cast<__half*>(q_out);
  a.q_stride = q_stride;
  a.entry_pos = entry_pos;
  a.entry_mass = entry_mass;
  a.err = err_flag;
  return qgemv::report_launch(
      qgemv::rope_append_launch(a, sms, static_cast<cudaStream_t>(stream)));
}

size_t qgemv_paged_attention_workspace_bytes(const qgemv_kv_cache* cache, int n_tokens, int n_q,
                                             int max_q) {
  KvView c{};
  if (check_cache(cache, &c) != QGEMV_OK ||
      check_queries(c, static_cast<long long>(n_q) * c.head_dim, n_tokens, n_q, max_q, 1.0f) !=
          QGEMV_OK ||
      n_tokens == 0)
    return 0;
  int dev, sms;
  if (qgemv::device_and_sms(&dev, &sms) != QGEMV_OK) return 0;
  const int group = n_q / c.n_kv, most = max_q < n_tokens ? max_q : n_tokens;
  if (qgemv::attention_is_many(group, most)) return qgemv::attention_many_bytes(c.head_dim, sms);
  return qgemv::attention_few_bytes(c.n_seqs, c.n_kv, most * group, c.head_dim,
                                    static_cast<long long>(c.max_pages) << c.page_shift, sms);
}

int qgemv_paged_attention(const qgemv_kv_cache* cache, const uint16_t* q, long long q_stride,
                          int n_tokens, int n_q, const int32_t* q_start, int max_q, float scale,
                          uint16_t* out, long long out_stride, float* lse, void* workspace,
                          size_t workspace_bytes, int* err_flag, void* stream) {
  qgemv::AttnArgs a{};
  if (int rc = check_cache(cache, &a.c)) return rc;
  if (!q_start || (n_tokens != 0 && (!q || !out)) || (workspace_bytes > 0 && !workspace))
    return QGEMV_ENULL;
  if (int rc = check_queries(a.c, q_stride, n_tokens, n_q, max_q, scale)) return rc;
  if (out_stride < static_cast<long long>(n_q) * a.c.head_dim || out_stride % 8 != 0)
    return QGEMV_EINVAL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(q_start, 4) || !aligned(lse, 4) ||
      !aligned(workspace, 16) || !aligned(err_flag, 4))
    return QGEMV_EALIGN;
  if (n_tokens == 0) return QGEMV_OK;
  if (out == q) return QGEMV_EINVAL;  // a row may be read again after it has been written
  int dev, sms;
  if (int rc = qgemv::device_and_sms(&dev, &sms)) return rc;
  a.q = reinterpret_cast<const __half*>(q);
  a.q_stride = q_stride;
  a.n_tokens = n_tokens;
  a.n_q = n_q;
  a.group = n_q / a.c.n_kv;
  a.group_inv = ~0ull / static_cast<unsigned>(a.group) + 1;
  a.q_start = q_start;
  a.max_q = max_q < n_tokens ? max_q : n_tokens;
  a.scale_log2 = scale * kLog2e;
  a.out = reinterpret_cast<__half*>(out);
  a.out_stride = out_stride;
  a.lse = lse;
  a.err = err_flag;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (qgemv::attention_is_many(a.group, a.max_q))
    return qgemv::report_launch(
        qgemv::attention_many_launch(a, sms, st, dev, workspace, workspace_bytes));
  return qgemv::report_launch(
      qgemv::attention_few_launch(a, sms, st, dev, workspace, workspace_bytes));
}

int qgemv_attention_mass(const qgemv_kv_cache* cache, const uint16_t* q, long long q_stride,
                         int n_tokens, int n_q, const int32_t* q_start, int max_q, float scale,
                         const float* lse, const float* mass, float* mass_out, int* err_flag,
                         void* stream) {
  qgemv::MassArgs a{};
  if (int rc = check_cache(cache, &a.c)) return rc;
  if (!q_start || !mass_out || (n_tokens != 0 && (!q || !lse))) return QGEMV_ENULL;
  if (int rc = check_queries(a.c, q_stride, n_tokens, n_q, max_q, scale)) return rc;
  if (!aligned(q, 16) || !aligned(q_start, 4) || !aligned(lse, 4) || !aligned(mass, 4) ||
      !aligned(mass_out, 4) || !aligned(err_flag, 4))
    return QGEMV_EALIGN;
  int dev, sms;
  if (int rc = qgemv::device_and_sms(&dev, &sms)) return rc;
  a.q = reinterpret_cast<const __half*>(q);
  a.q_stride = q_stride;
  a.n_tokens = n_tokens;
  a.n_q = n_q;
  a.group = n_q / a.c.n_kv;
  a.q_start = q_start;
  a.max_q = n_tokens > 0 && n_tokens < max_q ? n_tokens : max_q;
  a.scale_log2 = scale * kLog2e;
  a.lse = lse;
  a.mass = mass;
  a.mass_out = mass_out;
  a.err = err_flag;
  return qgemv::report_launch(
      qgemv::attention_mass_launch(a, sms, static_cast<cudaStream_t>(stream), dev));
}

int qgemv_cache_evict(const qgemv_kv_cache* cache, const float* mass, const int32_t* entry_pos,
                      const int32_t* next_pos, int keep, int n_sink, int n_recent, int32_t* kept,
                      float* mass_out, int32_t* pos_out, int32_t* kv_len_out, int* err_flag,
                      void* stream) {
  qgemv::EvictArgs a{};
  if (int rc = check_cache(cache, &a.c)) return rc;
  if (!mass || !entry_pos || !next_pos || !kept || !mass_out || !pos_out || !kv_len_out)
    return QGEMV_ENULL;
  if (keep < 1 || keep > 1 << 30 || n_sink < 0 || n_recent < 0 ||
      static_cast<long long>(n_sink) + n_recent > keep)
    return QGEMV_EINVAL;
  // an output that is an input would be read after it has been written
  if (mass_out == mass || pos_out == entry_pos || kv_len_out == cache->kv_len) return QGEMV_EINVAL;
  if (!aligned(mass, 4) || !aligned(entry_pos, 4) || !aligned(next_pos, 4) || !aligned(kept, 4) ||
      !aligned(mass_out, 4) || !aligned(pos_out, 4) || !aligned(kv_len_out, 4) ||
      !aligned(err_flag, 4))
    return QGEMV_EALIGN;
  int dev, sms;
  if (int rc = qgemv::device_and_sms(&dev, &sms)) return rc;
  a.mass = mass;
  a.entry_pos = entry_pos;
  a.next_pos = next_pos;
  a.keep = keep;
  a.n_sink = n_sink;
  a.n_recent = n_recent;
  a.kept = kept;
  a.mass_out = mass_out;
  a.pos_out = pos_out;
  a.len_out = kv_len_out;
  a.err = err_flag;
  return qgemv::report_launch(
      qgemv::cache_evict_launch(a, sms, static_cast<cudaStream_t>(stream), dev));
}

}  // extern "C"
