// C ABI of the paged cache: host-side argument checks and launches, in the
// manner of api.cu.
#include <cuda_runtime.h>

#include <initializer_list>

#include "paged.cuh"

namespace bastion {

int launch_paged_append(const Paged &c, const int32_t *held, const void *k_new, const void *v_new, int n_rows, int64_t st_b,
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
int launch_paged_plan(int32_t *table, int B, int max_pages, int page, int64_t n_pages, const int32_t *seq_len,
                      const int32_t *n_new, int m, int32_t *seq_len_out, const int32_t *held, int32_t *held_out,
                      int32_t *free_pages, const int32_t *n_free, int32_t *n_free_out, int trim, int64_t *slots,
                      int32_t *pos, int64_t n_rows, int32_t *row_start, const int32_t *pos_offset, void *ws,
                      int32_t *status, cudaStream_t stream);
int launch_qk_norm_rope(bool half, int T, int Hq, int Hkv, int D, const void *q, int64_t q_st_t, int64_t q_st_h,
                        const void *k, int64_t k_st_t, int64_t k_st_h, const void *v, int64_t v_st_t, int64_t v_st_h,
                        const void *q_weight, const void *k_weight, float eps, const int32_t *pos,
                        const double *inv_freq, int rot, bool pairs, float factor, void *q_out, int64_t q_out_st_t,
                        int64_t q_out_st_h, void *k_out, int64_t k_out_st_t, int64_t k_out_st_h, const Paged &c,
                        const int64_t *slots, int32_t *status, cudaStream_t stream);
size_t paged_prefix_workspace_bytes(int B, int Hq, int Hkv, int D, int n_groups);
int launch_paged_prefix(const Paged &c, bool half, const int32_t *prefix_table, int max_prefix_pages,
                        const int32_t *prefix_len, const int32_t *group_start, int n_groups, const void *q, int Hq,
                        int64_t q_st_b, const int32_t *seq_len, float scale, void *out, float *lse, void *ws,
                        int32_t *status, cudaStream_t stream);

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

// Rows of T tokens and H heads of D elements, at st_t and st_h elements.
struct Rows {
  const void *p;
  int64_t T, st_t, H, st_h, D;
  int64_t token() const { return (H - 1) * st_h + D; }  // from a token's first element to past its last
  Array span() const { return {p, (size_t)(2 * ((T - 1) * st_t + token()))}; }
};
// Whether two such arrays are disjoint: apart as a whole, or slices of the same tokens' rows.
bool rows_apart(const Rows &a, const Rows &b) {
  if (!a.p || !b.p || all_apart({a.span()}, {b.span()})) return true;
  if (a.T == 1 || b.T == 1 || a.st_t != b.st_t || a.token() > a.st_t || b.token() > b.st_t) return false;
  const int64_t diff = (int64_t)((uintptr_t)b.p - (uintptr_t)a.p);
  if (diff % 2) return false;
  const int64_t off = ((diff / 2) % a.st_t + a.st_t) % a.st_t;  // where b's tokens begin within a's
  return off >= a.token() && off + b.token() <= a.st_t;
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

// held: null, or the pages that each request holds.
int append(const bastion_paged_cache *cache, const int32_t *held, const void *k_new, const void *v_new, int n_rows,
           int64_t new_stride_b, int64_t new_stride_row, int64_t new_stride_head, const int32_t *rows, int m,
           const int32_t *n_new, const int32_t *seq_len, int32_t *seq_len_out, const int32_t *n_seen, int32_t *n_seen_out,
           float *acc, int32_t *pos, void *workspace, size_t workspace_bytes, int32_t *status, bastion_stream_t stream) {
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
              flags = {status, lens}, have = {held, lens};
  if (!all_apart({{seq_len_out, lens}, {n_seen_out, lens}}, {list, table, weights, places, flags, have}) ||
      !all_apart({weights, places, flags}, {{seq_len, lens}, {n_seen, lens}, {n_new, lens}, list, table, have}) ||
      !all_apart({weights}, {places, flags}) || !all_apart({places}, {flags}))
    return BASTION_ERR_UNSUPPORTED;
  if (workspace_bytes < bastion_paged_append_workspace_bytes(cache->B)) return BASTION_ERR_WORKSPACE;
  return bastion::launch_paged_append(bastion::paged_args(*cache), held, k_new, v_new, n_rows,
                                      cache->B > 1 ? new_stride_b : 0, n_rows > 1 ? new_stride_row : 0,
                                      cache->Hkv > 1 ? new_stride_head : 0, rows, m, n_new, seq_len, seq_len_out,
                                      n_seen, n_seen_out, acc, pos, workspace, status, (cudaStream_t)stream);
}

// pos_offset: null, or what is added to each request's positions.
int plan(int32_t *page_table, int B, int max_pages, int page_size, int64_t n_pages, const int32_t *seq_len,
         const int32_t *n_new, int m, int32_t *seq_len_out, const int32_t *held, int32_t *held_out, int32_t *free_pages,
         const int32_t *n_free, int32_t *n_free_out, int trim, int64_t *slots, int32_t *pos, int64_t n_rows,
         int32_t *row_start, const int32_t *pos_offset, void *workspace, size_t workspace_bytes, int32_t *status,
         bastion_stream_t stream) {
  if (!page_table || !seq_len || !held || !held_out || !free_pages || !n_free || !n_free_out || !slots || !pos ||
      !workspace || !status)
    return BASTION_ERR_NULL;
  const int64_t cap = (int64_t)max_pages * page_size;
  if (B < 1 || B > kMaxB || max_pages < 1 || page_size < 1 || cap > kMaxCap || n_pages < 1 || n_pages >= (1LL << 31) ||
      m < 1 || m > cap || n_rows < 1 || n_rows >= (1LL << 31) || (!row_start && n_rows != (int64_t)B * m))
    return BASTION_ERR_SIZE;
  if (page_size < 8 || page_size > 128 || (page_size & (page_size - 1))) return BASTION_ERR_UNSUPPORTED;
  if (!aligned(workspace, 256) || !aligned(slots, 8) || !aligned(pos, 4) || !aligned(page_table, 4)) return BASTION_ERR_ALIGN;
  const size_t lens = (size_t)B * 4;
  if ((seq_len_out && !same_or_apart(seq_len, seq_len_out, lens)) || !same_or_apart(held, held_out, lens) ||
      !same_or_apart(n_free, n_free_out, 4))
    return BASTION_ERR_UNSUPPORTED;
  const Array table = {page_table, (size_t)B * max_pages * 4}, stack = {free_pages, (size_t)n_pages * 4},
              len = {seq_len, lens}, len_out = {seq_len_out, lens}, add = {n_new, lens}, have = {held, lens},
              have_out = {held_out, lens}, left = {n_free, 4}, left_out = {n_free_out, 4},
              at = {slots, (size_t)n_rows * 8}, place = {pos, (size_t)n_rows * 4}, begin = {row_start, lens + 4},
              flags = {status, lens}, shift = {pos_offset, lens};
  // every output against every other array but its own pair's
  if (!all_apart({table}, {shift, stack, len, len_out, add, have, have_out, left, left_out, at, place, begin, flags}) ||
      !all_apart({stack}, {shift, len, len_out, add, have, have_out, left, left_out, at, place, begin, flags}) ||
      !all_apart({at}, {shift, len, len_out, add, have, have_out, left, left_out, place, begin, flags}) ||
      !all_apart({place}, {shift, len, len_out, add, have, have_out, left, left_out, begin, flags}) ||
      !all_apart({begin}, {shift, len, len_out, add, have, have_out, left, left_out, flags}) ||
      !all_apart({flags}, {shift, len, len_out, add, have, have_out, left, left_out}) ||
      !all_apart({len_out}, {shift, add, have, have_out, left, left_out}) ||
      !all_apart({have_out}, {shift, len, add, left, left_out}) || !all_apart({left_out}, {shift, len, add, have}))
    return BASTION_ERR_UNSUPPORTED;
  if (workspace_bytes < bastion_paged_plan_workspace_bytes(B)) return BASTION_ERR_WORKSPACE;
  return bastion::launch_paged_plan(page_table, B, max_pages, page_size, n_pages, seq_len, n_new, m, seq_len_out, held,
                                    held_out, free_pages, n_free, n_free_out, trim, slots, pos, n_rows, row_start,
                                    pos_offset, workspace, status, (cudaStream_t)stream);
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
  return append(cache, nullptr, k_new, v_new, n_rows, new_stride_b, new_stride_row, new_stride_head, rows, m, n_new, seq_len,
                seq_len_out, n_seen, n_seen_out, acc, pos, workspace, workspace_bytes, status, stream);
}

int bastion_paged_append_held(const bastion_paged_cache *cache, const int32_t *held, const void *k_new,
                              const void *v_new, int n_rows, int64_t new_stride_b, int64_t new_stride_row,
                              int64_t new_stride_head, const int32_t *rows, int m, const int32_t *n_new,
                              const int32_t *seq_len, int32_t *seq_len_out, const int32_t *n_seen,
                              int32_t *n_seen_out, float *acc, int32_t *pos, void *workspace,
                              size_t workspace_bytes, int32_t *status, bastion_stream_t stream) {
  if (!held) return BASTION_ERR_NULL;
  return append(cache, held, k_new, v_new, n_rows, new_stride_b, new_stride_row, new_stride_head, rows, m, n_new, seq_len,
                seq_len_out, n_seen, n_seen_out, acc, pos, workspace, workspace_bytes, status, stream);
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

size_t bastion_paged_plan_workspace_bytes(int B) {
  if (B < 1 || B > kMaxB) return 0;
  return (size_t)kMaxB * sizeof(uint32_t);  // an arrival counter
}

int bastion_paged_plan(int32_t *page_table, int B, int max_pages, int page_size, int64_t n_pages,
                       const int32_t *seq_len, const int32_t *n_new, int m, int32_t *seq_len_out,
                       const int32_t *held, int32_t *held_out, int32_t *free_pages,
                       const int32_t *n_free, int32_t *n_free_out, int trim, int64_t *slots,
                       int32_t *pos, int64_t n_rows, int32_t *row_start, void *workspace,
                       size_t workspace_bytes, int32_t *status, bastion_stream_t stream) {
  return plan(page_table, B, max_pages, page_size, n_pages, seq_len, n_new, m, seq_len_out, held, held_out, free_pages, n_free,
              n_free_out, trim, slots, pos, n_rows, row_start, nullptr, workspace, workspace_bytes, status, stream);
}

int bastion_paged_plan_offset(int32_t *page_table, int B, int max_pages, int page_size, int64_t n_pages,
                              const int32_t *seq_len, const int32_t *n_new, int m, int32_t *seq_len_out,
                              const int32_t *held, int32_t *held_out, int32_t *free_pages,
                              const int32_t *n_free, int32_t *n_free_out, int trim, int64_t *slots,
                              int32_t *pos, int64_t n_rows, int32_t *row_start, const int32_t *pos_offset,
                              void *workspace, size_t workspace_bytes, int32_t *status,
                              bastion_stream_t stream) {
  if (!pos_offset) return BASTION_ERR_NULL;
  return plan(page_table, B, max_pages, page_size, n_pages, seq_len, n_new, m, seq_len_out, held, held_out, free_pages, n_free,
              n_free_out, trim, slots, pos, n_rows, row_start, pos_offset, workspace, workspace_bytes, status, stream);
}

int bastion_qk_norm_rope(int dtype, int T, int Hq, int Hkv, int D, const void *q, int64_t q_st_t,
                         int64_t q_st_h, const void *k, int64_t k_st_t, int64_t k_st_h,
                         const void *v, int64_t v_st_t, int64_t v_st_h, const void *q_weight,
                         const void *k_weight, float eps, const int32_t *pos,
                         const double *inv_freq, int rot_dim, int interleaved, float factor,
                         void *q_out, int64_t q_out_st_t, int64_t q_out_st_h, void *k_out,
                         int64_t k_out_st_t, int64_t k_out_st_h, const bastion_paged_cache *cache,
                         const int64_t *slots, int32_t *status, bastion_stream_t stream) {
  if (!q || !k || !pos || !status || (rot_dim > 0 && !inv_freq) || (q_weight == nullptr) != (k_weight == nullptr) ||
      (cache == nullptr) != (slots == nullptr) || (cache == nullptr) != (v == nullptr) || (!q_out && !k_out && !cache))
    return BASTION_ERR_NULL;
  if (dtype != BASTION_BF16 && dtype != BASTION_F16) return BASTION_ERR_DTYPE;
  if (T < 1 || Hq < 1 || Hkv < 1 || D < 1 || (int64_t)Hq + 2 * (int64_t)Hkv > 65535 ||
      (int64_t)T * ((int64_t)Hq + 2 * (int64_t)Hkv) >= (1LL << 31))
    return BASTION_ERR_SIZE;
  if (D != 64 && D != 128) return BASTION_ERR_UNSUPPORTED;
  if (rot_dim < 0 || rot_dim > D || rot_dim % 16 || !(eps >= 0.f) || !(eps < 1e30f) || !(factor > -1e30f) ||
      !(factor < 1e30f))
    return BASTION_ERR_SIZE;
  if (cache) {
    const int rc = check_cache(cache);
    if (rc != BASTION_OK) return rc;
    if (cache->dtype != dtype) return BASTION_ERR_DTYPE;
    if (cache->D != D || cache->Hkv != Hkv) return BASTION_ERR_SIZE;
  }
  // the stride of a dimension of length 1 is never used
  auto rows = [&](const void *p, int64_t st_t, int64_t H, int64_t st_h) {
    return Rows{p, T, T > 1 ? st_t : 0, H, H > 1 ? st_h : D, D};
  };
  const Rows rq = rows(q, q_st_t, Hq, q_st_h), rk = rows(k, k_st_t, Hkv, k_st_h), rv = rows(v, v_st_t, Hkv, v_st_h),
             oq = rows(q_out, q_out_st_t, Hq, q_out_st_h), ok = rows(k_out, k_out_st_t, Hkv, k_out_st_h);
  for (const Rows *x : {&rq, &rk, &rv})
    if (x->p && (!stride_ok(T, x->st_t, 0) || !stride_ok(x->H, x->st_h, D))) return BASTION_ERR_SIZE;
  for (const Rows *x : {&oq, &ok})
    if (x->p && (!stride_ok(x->H, x->st_h, D) || !stride_ok(T, x->st_t, x->token()))) return BASTION_ERR_SIZE;
  for (const void *p : {q, k, v, (const void *)q_out, (const void *)k_out, q_weight, k_weight})
    if (!aligned(p, 16)) return BASTION_ERR_ALIGN;
  if (!aligned(inv_freq, 8) || !aligned(slots, 8)) return BASTION_ERR_ALIGN;
  auto in_place = [](const Rows &x, const Rows &y) { return x.p == y.p && x.st_t == y.st_t && x.st_h == y.st_h; };
  if (!(in_place(oq, rq) || rows_apart(oq, rq)) || !(in_place(ok, rk) || rows_apart(ok, rk)) || !rows_apart(oq, rk) ||
      !rows_apart(oq, rv) || !rows_apart(ok, rq) || !rows_apart(ok, rv) || !rows_apart(oq, ok))
    return BASTION_ERR_UNSUPPORTED;
  const size_t tokens = (size_t)T;
  auto span = [](const Rows &x) { return x.p ? x.span() : Array{nullptr, 0}; };
  const Array qw = {q_weight, (size_t)D * 2}, kw = {k_weight, (size_t)D * 2}, places = {pos, tokens * 4},
              freq = {rot_dim ? inv_freq : nullptr, (size_t)rot_dim * 4}, at = {slots, tokens * 8}, flags = {status, 4};
  if (!all_apart({span(oq), span(ok)}, {qw, kw, places, freq, at, flags}) ||
      !all_apart({flags}, {span(rq), span(rk), span(rv), qw, kw, places, freq, at}))
    return BASTION_ERR_UNSUPPORTED;
  return bastion::launch_qk_norm_rope(dtype == BASTION_F16, T, Hq, Hkv, D, q, rq.st_t, rq.st_h, k, rk.st_t, rk.st_h, v,
                                      rv.st_t, rv.st_h, q_weight, k_weight, eps, pos, inv_freq, rot_dim,
                                      interleaved != 0, factor, q_out, oq.st_t, oq.st_h, k_out, ok.st_t, ok.st_h,
                                      cache ? bastion::paged_args(*cache) : bastion::Paged{}, slots, status,
                                      (cudaStream_t)stream);
}

size_t bastion_paged_prefix_attention_workspace_bytes(int B, int Hq, int Hkv, int D, int n_groups) {
  if (!sizes_ok(B, Hkv, 1) || Hq < 1 || Hq % Hkv || Hq / Hkv > 16 || (D != 64 && D != 128) || n_groups < 1 ||
      n_groups > kMaxB)
    return 0;
  return bastion::paged_prefix_workspace_bytes(B, Hq, Hkv, D, n_groups);
}

int bastion_paged_prefix_attention(const bastion_paged_cache *cache, const int32_t *prefix_table,
                                   int max_prefix_pages, const int32_t *prefix_len,
                                   const int32_t *group_start, int n_groups, const void *q, int Hq,
                                   int64_t q_stride_b, const int32_t *seq_len, float scale,
                                   void *out, float *lse, void *workspace, size_t workspace_bytes,
                                   int32_t *status, bastion_stream_t stream) {
  if (!q || !seq_len || !out || !workspace || !status || !prefix_table || !prefix_len || !group_start)
    return BASTION_ERR_NULL;
  const int rc = check_cache(cache);
  if (rc != BASTION_OK) return rc;
  if (Hq < 1 || Hq % cache->Hkv || !(scale > 0.f) || !(scale < 1e30f)) return BASTION_ERR_SIZE;
  const int G = Hq / cache->Hkv;
  if (G > 16) return BASTION_ERR_UNSUPPORTED;
  const int64_t cap = (int64_t)max_prefix_pages * cache->page_size;
  if (n_groups < 1 || n_groups > kMaxB || max_prefix_pages < 1 || cap > kMaxCap || !tiles_ok(cache) ||
      cache->Hkv * ((cap + 127) / 128) * (n_groups + (int64_t)cache->B * G / 112) >= (1LL << 31))
    return BASTION_ERR_SIZE;
  if (!stride_ok(cache->B, q_stride_b, (int64_t)Hq * cache->D)) return BASTION_ERR_SIZE;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 256) || !aligned(prefix_table, 4))
    return BASTION_ERR_ALIGN;
  const int64_t row = (int64_t)Hq * cache->D, q_st = cache->B > 1 ? q_stride_b : row;
  const size_t lens = (size_t)cache->B * 4;
  const Array table = table_of(cache), len = {seq_len, lens}, flags = {status, lens},
              result = {out, (size_t)(2 * cache->B * row)}, logs = {lse, lens * Hq},
              pre = {prefix_table, (size_t)n_groups * max_prefix_pages * 4}, pre_len = {prefix_len, (size_t)n_groups * 4},
              start = {group_start, (size_t)(n_groups + 1) * 4};
  if (!(out == q && q_st == row) && !apart_from_rows(result, q, 2 * row, 2 * q_st, cache->B)) return BASTION_ERR_UNSUPPORTED;
  if (!all_apart({result, logs, flags}, {table, len, pre, pre_len, start}) || !all_apart({logs, flags}, {result}) ||
      !all_apart({logs}, {flags}))
    return BASTION_ERR_UNSUPPORTED;
  for (const Array &x : {logs, flags})
    if (!apart_from_rows(x, q, 2 * row, 2 * q_st, cache->B)) return BASTION_ERR_UNSUPPORTED;
  if (workspace_bytes < bastion_paged_prefix_attention_workspace_bytes(cache->B, Hq, cache->Hkv, cache->D, n_groups))
    return BASTION_ERR_WORKSPACE;
  return bastion::launch_paged_prefix(bastion::paged_args(*cache), cache->dtype == BASTION_F16, prefix_table,
                                      max_prefix_pages, prefix_len, group_start, n_groups, q, Hq,
                                      cache->B > 1 ? q_stride_b : 0, seq_len, scale, out, lse, workspace, status,
                                      (cudaStream_t)stream);
}

}  // extern "C"
