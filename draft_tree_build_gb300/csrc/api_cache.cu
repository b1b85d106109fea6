// C ABI of the paged cache: host-side argument checks and launches, in the
// manner of api.cu.
#include <cuda_runtime.h>

#include <initializer_list>

#include "paged.cuh"

namespace bastion {

int launch_paged_append(const Paged &c, const void *k_new, const void *v_new, int n_rows, int64_t st_b,
                        int64_t st_row, int64_t st_head, const int32_t *rows, int m, const int32_t *n_new,
                        const int32_t *seq_len, int32_t *seq_len_out, const int32_t *n_seen,
                        int32_t *n_seen_out, float *acc, int32_t *pos, void *ws, int32_t *status,
                        cudaStream_t stream);
size_t paged_attention_workspace_bytes(int B, int Hq, int Hkv, int D, int64_t cap, int weights);
int launch_paged_attention(const Paged &c, bool half, const void *q, int Hq, int64_t q_st_b, const int32_t *seq_len,
                           float scale, void *out, float *lse, const float *acc, float *acc_out, void *ws,
                           int32_t *status, cudaStream_t stream);
size_t paged_evict_workspace_bytes(int B, int Hkv, int64_t cap);
int launch_paged_evict(const Paged &c, const int32_t *seq_len, const int32_t *n_seen, const float *acc,
                       const int32_t *pos, int budget, int n_sink, int n_recent, int32_t *seq_len_out,
                       float *acc_out, int32_t *pos_out, void *ws, int32_t *status, cudaStream_t stream);

Paged paged_args(const bastion_paged_cache &c) {
  Paged p;
  p.k = static_cast<uint16_t *>(c.k_pool);
  p.v = static_cast<uint16_t *>(c.v_pool);
  p.n_pages = c.n_pages;
  // the stride of a dimension of length 1 is never used: any value is valid
  p.st_page = c.n_pages > 1 ? c.stride_page : c.D;
  p.st_slot = c.stride_slot;
  p.st_head = c.Hkv > 1 ? c.stride_head : c.D;
  p.table = c.page_table;
  p.B = c.B;
  p.Hkv = c.Hkv;
  p.D = c.D;
  p.page = c.page_size;
  p.shift = 0;
  while ((1 << p.shift) < c.page_size) ++p.shift;
  p.max_pages = c.max_pages;
  p.cap = c.max_pages * c.page_size;
  return p;
}

}  // namespace bastion

namespace {

constexpr int64_t kMaxCap = 1LL << 28;
constexpr int kMaxB = bastion::kMaxRequests, kMaxHeads = 65535;  // B * Hkv: a grid's y

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

bool stride_ok(int64_t n, int64_t s, int64_t least) { return n == 1 || (s >= least && s % 8 == 0 && s < (1LL << 38)); }

bool sizes_ok(int B, int Hkv, int64_t cap) {
  return B >= 1 && B <= kMaxB && Hkv >= 1 && (int64_t)B * Hkv <= kMaxHeads && cap >= 1 && cap <= kMaxCap;
}

// Whether an output is its input's array or disjoint from it.
bool apart(const void *a, const void *b, size_t bytes) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x + bytes <= y || y + bytes <= x;
}
bool same_or_apart(const void *a, const void *b, size_t bytes) { return a == b || apart(a, b, bytes); }

// A contiguous array; null where an optional one is left out.
struct Array {
  const void *p;
  size_t bytes;
};
// Whether each of the first is disjoint from each of the second.
bool all_apart(std::initializer_list<Array> a, std::initializer_list<Array> b) {
  for (const Array &x : a)
    for (const Array &y : b) {
      if (!x.p || !y.p) continue;
      const uintptr_t u = (uintptr_t)x.p, v = (uintptr_t)y.p;
      if (u < v + y.bytes && v < u + x.bytes) return false;
    }
  return true;
}

// Whether an array is disjoint from each of n rows, `stride` >= 0 bytes apart.
bool apart_from_rows(Array a, const void *first, int64_t row, int64_t stride, int64_t n) {
  if (!a.p) return true;
  const int64_t lo = (int64_t)((uintptr_t)a.p - (uintptr_t)first), hi = lo + (int64_t)a.bytes;
  if (stride < row) return hi <= 0 || lo >= (n - 1) * stride + row;  // the rows leave no gaps
  const int64_t i = lo < row ? 0 : (lo - row) / stride + 1;  // the first row that ends past the array's begin
  return i >= n || i * stride >= hi;
}

size_t slots_bytes(const bastion_paged_cache *c) {  // of acc and of pos
  return (size_t)c->B * c->Hkv * (size_t)c->max_pages * c->page_size * 4;
}
Array table_of(const bastion_paged_cache *c) { return {c->page_table, (size_t)c->B * c->max_pages * 4}; }

// The batch's 128-key tiles are counted in 31 bits.
bool tiles_ok(const bastion_paged_cache *c) {
  return (int64_t)c->B * c->Hkv * (((int64_t)c->max_pages * c->page_size + 127) / 128) < (1LL << 31);
}

// Checks that every call makes of the cache.
int check_cache(const bastion_paged_cache *c) {
  if (!c || !c->k_pool || !c->v_pool || !c->page_table) return BASTION_ERR_NULL;
  if (c->dtype != BASTION_BF16 && c->dtype != BASTION_F16) return BASTION_ERR_DTYPE;
  if (c->D < 1 || c->page_size < 1 || c->max_pages < 1 || c->n_pages < 1 || c->n_pages >= (1LL << 31) ||
      !sizes_ok(c->B, c->Hkv, (int64_t)c->max_pages * c->page_size))
    return BASTION_ERR_SIZE;
  if ((c->D != 64 && c->D != 128) || c->page_size < 8 || c->page_size > 128 || (c->page_size & (c->page_size - 1)))
    return BASTION_ERR_UNSUPPORTED;
  if (!stride_ok(c->n_pages, c->stride_page, c->D) || !stride_ok(c->page_size, c->stride_slot, c->D) ||
      !stride_ok(c->Hkv, c->stride_head, c->D))
    return BASTION_ERR_SIZE;
  if (!aligned(c->k_pool, 16) || !aligned(c->v_pool, 16) || !aligned(c->page_table, 4)) return BASTION_ERR_ALIGN;
  return BASTION_OK;
}

}  // namespace

extern "C" {

size_t bastion_paged_append_workspace_bytes(int B) {
  if (B < 1 || B > kMaxB) return 0;
  return (size_t)kMaxB * sizeof(uint32_t);  // arrival counters
}

int bastion_paged_append(const bastion_paged_cache *cache, const void *k_new, const void *v_new,
                         int n_rows, int64_t new_stride_b, int64_t new_stride_row,
                         int64_t new_stride_head, const int32_t *rows, int m,
                         const int32_t *n_new, const int32_t *seq_len, int32_t *seq_len_out,
                         const int32_t *n_seen, int32_t *n_seen_out, float *acc, int32_t *pos,
                         void *workspace, size_t workspace_bytes, int32_t *status,
                         bastion_stream_t stream) {
  if (!k_new || !v_new || !seq_len || !seq_len_out || !workspace || !status) return BASTION_ERR_NULL;
  if ((acc == nullptr) != (pos == nullptr) || (n_seen == nullptr) != (n_seen_out == nullptr) || (acc && !n_seen))
    return BASTION_ERR_NULL;
  const int rc = check_cache(cache);
  if (rc != BASTION_OK) return rc;
  if (n_rows < 1 || m < 1 || (rows ? m > 1024 : m > n_rows)) return BASTION_ERR_SIZE;
  if (!stride_ok(cache->B, new_stride_b, 0) || !stride_ok(n_rows, new_stride_row, 0) ||
      !stride_ok(cache->Hkv, new_stride_head, 0))
    return BASTION_ERR_SIZE;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(workspace, 256)) return BASTION_ERR_ALIGN;
  const size_t lens = (size_t)cache->B * 4;
  if (!same_or_apart(seq_len, seq_len_out, lens) || (n_new && !same_or_apart(n_new, seq_len_out, lens)))
    return BASTION_ERR_UNSUPPORTED;
  if (n_seen) {  // where no slot is ever evicted, both counts may be one array
    if (!same_or_apart(n_seen, n_seen_out, lens) || !same_or_apart(n_seen, seq_len_out, lens) ||
        !same_or_apart(seq_len, n_seen_out, lens) || (n_new && !same_or_apart(n_new, n_seen_out, lens)) ||
        !(apart(seq_len_out, n_seen_out, lens) || (seq_len_out == n_seen_out && seq_len == n_seen)))
      return BASTION_ERR_UNSUPPORTED;
  }
  // a request's last CTA writes its lengths while others still read their lists
  const size_t slots = slots_bytes(cache);
  const Array table = table_of(cache), list = {rows, (size_t)cache->B * m * 4}, weights = {acc, slots}, places = {pos, slots},
              flags = {status, lens};
  if (!all_apart({{seq_len_out, lens}, {n_seen_out, lens}}, {list, table, weights, places, flags}) ||
      !all_apart({weights, places, flags}, {{seq_len, lens}, {n_seen, lens}, {n_new, lens}, list, table}) ||
      !all_apart({weights}, {places, flags}) || !all_apart({places}, {flags}))
    return BASTION_ERR_UNSUPPORTED;
  if (workspace_bytes < bastion_paged_append_workspace_bytes(cache->B)) return BASTION_ERR_WORKSPACE;
  return bastion::launch_paged_append(bastion::paged_args(*cache), k_new, v_new, n_rows,
                                      cache->B > 1 ? new_stride_b : 0, n_rows > 1 ? new_stride_row : 0,
                                      cache->Hkv > 1 ? new_stride_head : 0, rows, m, n_new, seq_len, seq_len_out,
                                      n_seen, n_seen_out, acc, pos, workspace, status, (cudaStream_t)stream);
}

size_t bastion_paged_attention_workspace_bytes(int B, int Hq, int Hkv, int D, int64_t cap, int weights) {
  if (!sizes_ok(B, Hkv, cap) || Hq < 1 || Hq % Hkv || Hq / Hkv > 16 || (D != 64 && D != 128)) return 0;
  return bastion::paged_attention_workspace_bytes(B, Hq, Hkv, D, cap, weights);
}

int bastion_paged_attention(const bastion_paged_cache *cache, const void *q, int Hq,
                            int64_t q_stride_b, const int32_t *seq_len, float scale, void *out,
                            float *lse, const float *acc, float *acc_out, void *workspace,
                            size_t workspace_bytes, int32_t *status, bastion_stream_t stream) {
  if (!q || !seq_len || !out || !workspace || !status || (acc == nullptr) != (acc_out == nullptr))
    return BASTION_ERR_NULL;
  const int rc = check_cache(cache);
  if (rc != BASTION_OK) return rc;
  if (Hq < 1 || Hq % cache->Hkv || !(scale > 0.f) || !(scale < 1e30f)) return BASTION_ERR_SIZE;
  if (Hq / cache->Hkv > 16) return BASTION_ERR_UNSUPPORTED;
  if (!tiles_ok(cache)) return BASTION_ERR_SIZE;
  if (!stride_ok(cache->B, q_stride_b, 0)) return BASTION_ERR_SIZE;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 256) || !aligned(acc, 16) || !aligned(acc_out, 16))
    return BASTION_ERR_ALIGN;
  if (acc && !same_or_apart(acc, acc_out, slots_bytes(cache))) return BASTION_ERR_UNSUPPORTED;
  // in place: a head's queries are read by all who need them before its output is written, but not another head's
  const int64_t row = (int64_t)Hq * cache->D, q_st = cache->B > 1 ? q_stride_b : row;
  const uintptr_t q0 = (uintptr_t)q, q1 = q0 + 2 * (uintptr_t)((cache->B - 1) * q_st + row), o0 = (uintptr_t)out;
  if (!(q0 == o0 && q_st == row) && o0 < q1 && q0 < o0 + 2 * (uintptr_t)(cache->B * row)) return BASTION_ERR_UNSUPPORTED;
  const size_t slots = slots_bytes(cache), lens = (size_t)cache->B * 4;
  const Array table = table_of(cache), len = {seq_len, lens}, flags = {status, lens}, result = {out, (size_t)(2 * cache->B * row)},
              logs = {lse, lens * Hq}, weights = {acc, slots}, weights_out = {acc_out, slots};
  if (!all_apart({result, logs, weights_out, flags}, {table, len}) || !all_apart({logs, flags}, {result, weights, weights_out}) ||
      !all_apart({logs}, {flags}) || !all_apart({result}, {weights, weights_out}))
    return BASTION_ERR_UNSUPPORTED;
  for (const Array &x : {logs, weights_out, flags})
    if (!apart_from_rows(x, q, 2 * row, 2 * q_st, cache->B)) return BASTION_ERR_UNSUPPORTED;
  if (workspace_bytes < bastion_paged_attention_workspace_bytes(cache->B, Hq, cache->Hkv, cache->D,
                                                                (int64_t)cache->max_pages * cache->page_size,
                                                                acc != nullptr))
    return BASTION_ERR_WORKSPACE;
  return bastion::launch_paged_attention(bastion::paged_args(*cache), cache->dtype == BASTION_F16, q, Hq,
                                         cache->B > 1 ? q_stride_b : 0, seq_len, scale, out, lse, acc, acc_out,
                                         workspace, status, (cudaStream_t)stream);
}

size_t bastion_paged_evict_workspace_bytes(int B, int Hkv, int64_t cap) {
  if (!sizes_ok(B, Hkv, cap)) return 0;
  return bastion::paged_evict_workspace_bytes(B, Hkv, cap);
}

int bastion_paged_evict(const bastion_paged_cache *cache, const int32_t *seq_len,
                        const int32_t *n_seen, const float *acc, const int32_t *pos, int budget,
                        int n_sink, int n_recent, int32_t *seq_len_out, float *acc_out,
                        int32_t *pos_out, void *workspace, size_t workspace_bytes,
                        int32_t *status, bastion_stream_t stream) {
  if (!seq_len || !n_seen || !acc || !pos || !seq_len_out || !acc_out || !pos_out || !workspace || !status)
    return BASTION_ERR_NULL;
  const int rc = check_cache(cache);
  if (rc != BASTION_OK) return rc;
  if (budget < 1 || n_sink < 0 || n_recent < 0 || (int64_t)n_sink + n_recent > budget) return BASTION_ERR_SIZE;
  if (!aligned(workspace, 256) || !aligned(acc, 16) || !aligned(pos, 16) || !aligned(acc_out, 16) ||
      !aligned(pos_out, 16))
    return BASTION_ERR_ALIGN;
  const size_t lens = (size_t)cache->B * 4;
  if (!same_or_apart(seq_len, seq_len_out, lens) || !apart(n_seen, seq_len_out, lens) ||
      !same_or_apart(acc, acc_out, slots_bytes(cache)) || !same_or_apart(pos, pos_out, slots_bytes(cache)))
    return BASTION_ERR_UNSUPPORTED;
  const size_t slots = slots_bytes(cache);
  const Array table = table_of(cache), len = {seq_len, lens}, len_out = {seq_len_out, lens}, seen = {n_seen, lens},
              weights = {acc, slots}, weights_out = {acc_out, slots}, places = {pos, slots}, places_out = {pos_out, slots},
              flags = {status, lens};
  if (!all_apart({len_out, flags}, {table, weights, weights_out, places, places_out}) ||
      !all_apart({flags}, {len, len_out, seen}) || !all_apart({weights_out, places_out}, {table, len, seen}) ||
      !all_apart({weights_out}, {places, places_out}) || !all_apart({places_out}, {weights}))
    return BASTION_ERR_UNSUPPORTED;
  if (workspace_bytes < bastion_paged_evict_workspace_bytes(cache->B, cache->Hkv,
                                                            (int64_t)cache->max_pages * cache->page_size))
    return BASTION_ERR_WORKSPACE;
  return bastion::launch_paged_evict(bastion::paged_args(*cache), seq_len, n_seen, acc, pos, budget, n_sink, n_recent,
                                     seq_len_out, acc_out, pos_out, workspace, status, (cudaStream_t)stream);
}

}  // extern "C"
