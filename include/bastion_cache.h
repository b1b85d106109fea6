/*
 * bastion_cache.h -- the paged key-value cache of the target model: append,
 * one-token attention, eviction by accumulated attention weight, and what a step
 * of a layer needs around them: pages and slots for new tokens, norm and rotation
 * of queries and keys on their way into the cache, attention over shared prefixes.
 *
 * What bastion_tree_attention does for a drafted tree, these calls do for the
 * steps around it: the accepted path of a verified tree enters the cache
 * (bastion_paged_append takes bastion_verify_greedy's accept_nodes as its row
 * list), a request is decoded without a tree where speculation does not pay
 * (the step whose latency is L_AR), and the cache is kept within a budget.
 * Conventions (device pointers, return codes, status bits, workspaces,
 * streams) are bastion.h's; status is [B] int32, OR-ed.
 *
 * The cache.  Keys and values live in two pools of n_pages pages of page_size
 * slots: element (page, slot, head, d) is at
 *   page * stride_page + slot * stride_slot + head * stride_head + d
 * elements, the same strides for both pools, so that both slot-major
 * [page][slot][head][D] and head-major [page][head][slot][D] pools, and keys
 * and values that share an allocation, are read in place.  Slot j of request r
 * is slot j % page_size of page page_table[r][j / page_size].  Requests may
 * share pages that are only read; a page that append or evict writes belongs
 * to one request, and appears in its table once.  A contiguous cache
 * [B, L_cap, Hkv, D] whose L_cap is a multiple of page_size is such a pool
 * with page_table[r][i] = r * L_cap / page_size + i: the same memory serves
 * bastion_tree_attention.
 * One workspace that is large enough for each may serve all calls, at all
 * sizes, one after the other.  A workspace that a call with
 * BASTION_STATUS_TIMEOUT has used is cleared before its next use.
 * Page table entries past a request's last used page are not read.  Slots at
 * or past seq_len[r] never affect a result (they may hold NaN) and are left as
 * they are by every call except for the slots that append fills.
 *
 * Limits of every call: dtype BASTION_BF16 or BASTION_F16, D = 64 or 128,
 * page_size a power of two in [8, 128] (BASTION_ERR_UNSUPPORTED otherwise);
 * 1 <= B <= 1024, 1 <= Hkv, B * Hkv <= 65535, n_pages < 2^31,
 * max_pages * page_size <= 2^28; strides of dimensions longer than 1 are
 * multiples of 8 elements and at least D (BASTION_ERR_SIZE otherwise); pools
 * 16-byte aligned.
 * An output array that may be its input's own must be that array exactly or
 * lie apart from it (BASTION_ERR_UNSUPPORTED when they overlap otherwise).
 * A seq_len outside [0, max_pages * page_size] sets BASTION_STATUS_KV_OVERFLOW
 * and a used page table entry outside [0, n_pages) BASTION_STATUS_BAD_PAGE;
 * nothing outside the pools is read or written then.
 */
#ifndef BASTION_CACHE_H_
#define BASTION_CACHE_H_

#include "bastion.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Host struct, read before the call returns. */
typedef struct {
  void *k_pool, *v_pool;
  int64_t n_pages, stride_page, stride_slot, stride_head;
  const int32_t *page_table; /* [B, max_pages] */
  int32_t dtype, B, Hkv, D, page_size, max_pages;
} bastion_paged_cache;

/* ---------------------------------------------------------------------------
 * Append: row i of request r's list goes to slot seq_len[r] + i.
 *
 * k_new, v_new  rows [B, n_rows, Hkv, D] at strides new_stride_b,
 *               new_stride_row, new_stride_head elements (multiples of 8;
 *               0 is allowed), 16-byte aligned; must not overlap the pools.
 * rows          [B, m] int32 or NULL: the rows to append in order; the first
 *               negative entry ends a request's list (accept_nodes [B, b+1]
 *               fits as it is, with n_rows = n_max).  m <= 1024 with a list.
 *               NULL: rows 0 .. m-1 (m <= n_rows).  An entry >= n_rows sets
 *               BASTION_STATUS_BAD_ROW.
 * n_new         [B] int32 or NULL: at most that many rows of request r
 *               (negative counts as 0).
 * seq_len, seq_len_out  [B] int32: used slots before and after; the same array
 *               or disjoint ones.
 * n_seen, n_seen_out    [B] int32: tokens ever appended, before and after (the
 *               position of the next token); the same or disjoint.  Needed
 *               with acc and pos, else both may be NULL.  Where nothing is ever
 *               evicted they may be seq_len and seq_len_out.
 *               No output (the lengths, acc, pos, status) overlaps part of
 *               another input or output (BASTION_ERR_UNSUPPORTED; the pools and
 *               the new rows are the caller's to keep apart).
 * acc, pos      [B, Hkv, max_pages * page_size], both or neither NULL: the new
 *               slots get weight 0 and their token's position.
 * A request whose rows do not fit (seq_len + rows > max_pages * page_size)
 * sets BASTION_STATUS_KV_OVERFLOW, gets nothing and keeps its lengths.
 * Workspace: bastion_paged_append_workspace_bytes(B) bytes.  One launch.
 */
size_t bastion_paged_append_workspace_bytes(int B);
int bastion_paged_append(const bastion_paged_cache *cache, const void *k_new, const void *v_new,
                         int n_rows, int64_t new_stride_b, int64_t new_stride_row,
                         int64_t new_stride_head, const int32_t *rows, int m,
                         const int32_t *n_new, const int32_t *seq_len, int32_t *seq_len_out,
                         const int32_t *n_seen, int32_t *n_seen_out, float *acc, int32_t *pos,
                         void *workspace, size_t workspace_bytes, int32_t *status,
                         bastion_stream_t stream);
/* The same into a table that bastion_paged_plan keeps: request r holds the pages of
 * its first held[r] entries, and later entries may name pages that it gave back and
 * that are others' now.  A request whose rows would reach past them sets
 * BASTION_STATUS_NO_PAGE, one whose held[r] is outside [0, max_pages]
 * BASTION_STATUS_BAD_PAGE: it gets nothing and keeps its lengths.  held [B] int32
 * (BASTION_ERR_NULL without it), apart from the outputs. */
int bastion_paged_append_held(const bastion_paged_cache *cache, const int32_t *held,
                              const void *k_new, const void *v_new, int n_rows, int64_t new_stride_b,
                              int64_t new_stride_row, int64_t new_stride_head, const int32_t *rows,
                              int m, const int32_t *n_new, const int32_t *seq_len,
                              int32_t *seq_len_out, const int32_t *n_seen, int32_t *n_seen_out,
                              float *acc, int32_t *pos, void *workspace, size_t workspace_bytes,
                              int32_t *status, bastion_stream_t stream);

/* ---------------------------------------------------------------------------
 * Attention of one new token per request over its used slots.
 *
 *   s_j = scale * q[r,h] . k_j,  lse[r,h] = log sum_{j < seq_len[r]} exp(s_j),
 *   out[r,h] = sum_j exp(s_j - lse) v_j,         k_j, v_j of head h / (Hq/Hkv),
 *   acc_out[r,g,j] = acc[r,g,j] + sum_{h of group g} exp(s_j - lse[r,h]).
 *
 * q        [B, Hq, D] at q_stride_b elements per request (a multiple of 8),
 *          the cache's dtype, 16-byte aligned.
 * seq_len  [B] int32.  A request without slots, or a head whose scores are all
 *          -inf, gives out = 0 and lse = -inf.
 * out      [B, Hq, D] contiguous, the cache's dtype (rounded once to nearest
 *          even), 16-byte aligned; q itself where q is contiguous, or apart from
 *          it (BASTION_ERR_UNSUPPORTED otherwise).
 * lse      [B, Hq] float or NULL.
 * acc, acc_out  [B, Hkv, max_pages * page_size] float, 16-byte aligned, both or
 *          neither NULL; the same array or disjoint ones.  Slots at or past seq_len[r] of
 *          acc_out are left as they are.
 * out, lse, acc_out and status lie apart from one another and, but for the two
 * places in place above, from every input (BASTION_ERR_UNSUPPORTED; the pools
 * are the caller's to keep apart).
 * scale    > 0 and < 1e30, else BASTION_ERR_SIZE.
 * NaN in a used key or query gives NaN in the heads that see it.
 * A request that BASTION_STATUS_TIMEOUT flags may lack the outputs of some or
 * all of its heads; acc_out is acc where a group's were not finished.
 * Scores, sums and outputs are accumulated in 32 bits, the outputs' sums by
 * instructions that cut where others round: an output lacks about 1e-5 of itself at
 * 16,384 slots in one CTA's share (64 requests of them), 1e-4 at 131,072.  A weight exp(s_j - lse)
 * enters the product with v_j as two 16-bit terms: off by 2^-17 of itself with
 * bf16, by 2^-22 of itself or 2^-31 of the row's largest weight with half
 * precision.  Results do not depend on the order in which the parts of a split
 * row finish.
 * Limits: Hq a multiple of Hkv (BASTION_ERR_SIZE), Hq / Hkv <= 16
 * (BASTION_ERR_UNSUPPORTED), B * Hkv * ceil(max_pages * page_size / 128) < 2^31
 * (BASTION_ERR_SIZE).
 * Workspace: bastion_paged_attention_workspace_bytes(B, Hq, Hkv, D,
 * max_pages * page_size, acc != NULL) bytes; with acc 4 bytes a query head and
 * slot of capacity among them.  One launch, two with acc.  Attention's time goes
 * by the used slots; the second launch passes over the whole capacity (32
 * requests of 2,065 tokens, 32/8 heads: 54 us with max_pages * page_size =
 * 2,080, 81 us with 32,768, 159 us with 131,072), so that tables no wider than
 * needed are faster.
 */
size_t bastion_paged_attention_workspace_bytes(int B, int Hq, int Hkv, int D, int64_t cap,
                                               int weights);
int bastion_paged_attention(const bastion_paged_cache *cache, const void *q, int Hq,
                            int64_t q_stride_b, const int32_t *seq_len, float scale, void *out,
                            float *lse, const float *acc, float *acc_out, void *workspace,
                            size_t workspace_bytes, int32_t *status, bastion_stream_t stream);

/* ---------------------------------------------------------------------------
 * Eviction: every request and KV head keeps the `budget` slots with the
 * largest accumulated weights.
 *
 * For request r with n = seq_len[r] > budget, each head keeps the slots whose
 * position is below n_sink or at least n_seen[r] - n_recent (in slot order,
 * should there be more than budget of them), then those with the largest acc
 * (ties: the lower slot), budget slots in all.  The slots below budget that
 * are not kept are refilled, in ascending order, by the kept slots at or past
 * budget, in ascending order; no other slot changes, so that a step that
 * evicts few tokens moves few.  Slot order is therefore not token order: pos
 * names each slot's token.  Attention does not depend on the order.
 *
 * acc, pos      [B, Hkv, max_pages * page_size]: weights and positions, 16-byte
 *               aligned (as acc_out and pos_out).  A NaN weight sets
 *               BASTION_STATUS_NONFINITE and counts as +inf.
 * seq_len_out   [B]: min(seq_len, budget).
 * acc_out, pos_out: slots below min(seq_len, budget) are written, the others
 *               left as they are.
 * Each output is its input's array or disjoint from every input, and from the
 * other outputs and status (BASTION_ERR_UNSUPPORTED otherwise; the pools are the
 * caller's to keep apart).
 * Limits: 1 <= budget, n_sink, n_recent >= 0, n_sink + n_recent <= budget
 * (BASTION_ERR_SIZE).
 * Workspace: bastion_paged_evict_workspace_bytes(B, Hkv,
 * max_pages * page_size) bytes.  One launch, whose shape goes by the capacity (32
 * requests of 2,065 tokens and 8 heads cut to 2,048: 11 us with max_pages *
 * page_size = 2,080, 22 us with 32,768, 79 us with 131,072).
 */
size_t bastion_paged_evict_workspace_bytes(int B, int Hkv, int64_t cap);
int bastion_paged_evict(const bastion_paged_cache *cache, const int32_t *seq_len,
                        const int32_t *n_seen, const float *acc, const int32_t *pos, int budget,
                        int n_sink, int n_recent, int32_t *seq_len_out, float *acc_out,
                        int32_t *pos_out, void *workspace, size_t workspace_bytes,
                        int32_t *status, bastion_stream_t stream);

/* ---------------------------------------------------------------------------
 * Page plan: the pages and slots of each request's next tokens, found on the
 * GPU from the requests' lengths.
 *
 * Request r, with n = seq_len[r] used slots and held[r] pages, gets
 * c = min(m, max(n_new[r], 0)) new slots (m where n_new is NULL), and pages for
 * them where ceil((n + c) / page_size) exceeds held[r]; with trim != 0 it gives
 * back the pages that it holds beyond that many (a request that has ended:
 * seq_len = n_new = 0).  The free pages are a stack, free_pages[0 .. n_free[0]):
 * first the pages given back are pushed, requests in order and each one's in the
 * order of its table, then new pages are popped, requests in order.
 *
 * page_table    [B, max_pages] int32: entries [held[r], ceil((n + c) /
 *               page_size)) are written, the others left as they are (those of
 *               pages given back among them, which are no longer the request's).
 * seq_len, n_new, seq_len_out  [B] int32; n_new may be NULL (m for each) and
 *               seq_len_out NULL or seq_len: n + c.  NULL where the pages are for
 *               rows that bastion_paged_append_held brings, which counts them.
 * held, held_out  [B] int32: pages held before and after; may be one array.
 * free_pages    [n_pages] int32, n_free, n_free_out [1] int32 (may be one).
 *               Entries at or past n_free are written where more pages come
 *               back than go, the others left as they are.
 * slots, pos    [n_rows] int64 and int32: slot (page * page_size + slot in the
 *               page) and position n + i of every new token, -1 in rows that have
 *               none.  row_start NULL: request r's are rows r * m + i, and
 *               n_rows = B * m (BASTION_ERR_SIZE otherwise).  row_start [B+1]
 *               int32: they are packed, request r's are rows row_start[r] + i.
 *               Positions count the request's own slots: behind a shared prefix
 *               of P tokens a model's is P + n + i, which
 *               bastion_paged_plan_offset gives.
 * A request that cannot be served gets no rows and no pages, gives none back and
 * keeps its length: seq_len outside [0, max_pages * page_size] or n + c beyond
 * it, or packed rows that would end past n_rows (BASTION_STATUS_KV_OVERFLOW);
 * held outside [0, max_pages], or held pages too few for n slots
 * (BASTION_STATUS_BAD_PAGE); too few free pages (BASTION_STATUS_NO_PAGE: first
 * come, first served; after the first such request none that needs a page gets
 * one).  Packed rows are first come, first served too.
 * A page number outside [0, n_pages) sets BASTION_STATUS_BAD_PAGE, for the request
 * whose rows it would hold, whose slots are -1 there, and for one that gives it back
 * (it goes on the list as it is).  n_free is taken as lying in [0, n_pages]; where it does not
 * status[0] gets BASTION_STATUS_BAD_PAGE.
 * Limits: as the cache's; 1 <= m <= max_pages * page_size, 1 <= n_rows < 2^31.
 * Apart from the pairs above no output overlaps another array
 * (BASTION_ERR_UNSUPPORTED).
 * Workspace: bastion_paged_plan_workspace_bytes(B) bytes.  One launch.
 */
size_t bastion_paged_plan_workspace_bytes(int B);
int bastion_paged_plan(int32_t *page_table, int B, int max_pages, int page_size, int64_t n_pages,
                       const int32_t *seq_len, const int32_t *n_new, int m, int32_t *seq_len_out,
                       const int32_t *held, int32_t *held_out, int32_t *free_pages,
                       const int32_t *n_free, int32_t *n_free_out, int trim, int64_t *slots,
                       int32_t *pos, int64_t n_rows, int32_t *row_start, void *workspace,
                       size_t workspace_bytes, int32_t *status, bastion_stream_t stream);
/* The same with positions pos_offset[r] + n + i, -1 in rows without a token as
 * before: own slots behind a shared prefix of pos_offset[r] tokens.  pos_offset [B]
 * int32 (BASTION_ERR_NULL without it), apart from the outputs; a request whose
 * offset is outside [0, 2^31 - 1 - max_pages * page_size] cannot be served and sets
 * BASTION_STATUS_KV_OVERFLOW. */
int bastion_paged_plan_offset(int32_t *page_table, int B, int max_pages, int page_size, int64_t n_pages,
                              const int32_t *seq_len, const int32_t *n_new, int m, int32_t *seq_len_out,
                              const int32_t *held, int32_t *held_out, int32_t *free_pages,
                              const int32_t *n_free, int32_t *n_free_out, int trim, int64_t *slots,
                              int32_t *pos, int64_t n_rows, int32_t *row_start,
                              const int32_t *pos_offset, void *workspace, size_t workspace_bytes,
                              int32_t *status, bastion_stream_t stream);

/* ---------------------------------------------------------------------------
 * Norm and rotation of T tokens' queries and keys, in one pass that may also
 * store keys and values into the cache.
 *
 * Each head x of q and k is normed, where weights are given,
 *   y = x / sqrt(mean(x^2) + eps) * weight,
 * and its first rot_dim elements turned by the token's position: the pair
 * (a, b), number i, becomes factor * (a cos t - b sin t, b cos t + a sin t)
 * with t = pos * inv_freq[i].  Pair i is elements (i, i + rot_dim / 2), or
 * (2 i, 2 i + 1) with interleaved != 0.  Sums and products are formed in 32 bits
 * and rounded once; t is reduced to a fraction of a turn in 64-bit fixed point,
 * exactly, so that far positions are as good as near ones.
 *
 * q, k, v       [T, Hq, D], [T, Hkv, D], [T, Hkv, D] at *_st_t elements a token
 *               and *_st_h a head (multiples of 8, st_h >= D), 16-byte aligned:
 *               slices of one projection's output fit.  v with a cache only.
 * q_weight, k_weight  [D], of the same dtype, 16-byte aligned; both or neither
 *               NULL (no norm).  eps >= 0, finite.
 * pos           [T] int32.  A token whose position is negative is left out: none
 *               of its outputs is written.
 * inv_freq      [rot_dim / 2] double (8-byte aligned), finite; scaled for a long
 *               context by the caller.  rot_dim a multiple of 16 in [0, D]; 0:
 *               nothing is turned, inv_freq may be NULL.
 * q_out, k_out  as q and k (tokens' rows not overlapping), or NULL: not written.
 *               q_out may be q, k_out k, with the same strides; otherwise they lie
 *               apart from one another and from every input, as whole arrays or as
 *               slices of tokens' rows of one stride (BASTION_ERR_UNSUPPORTED
 *               otherwise).
 * cache, slots  NULL, or the cache and [T] int64: the token's key and value go to
 *               slot slots[t] (as bastion_paged_plan gives it); a negative slot
 *               stores nothing, one past the pools sets BASTION_STATUS_BAD_PAGE.
 *               A slot listed twice holds one of the two rows' values in each of
 *               its 16-byte pieces.  The cache's B, page_table and max_pages are
 *               checked and not used; its pools lie apart from the other arrays.
 * status        [1] int32.
 * Limits: D = 64 or 128 (BASTION_ERR_UNSUPPORTED); T, Hq, Hkv >= 1, Hq + 2 Hkv
 * <= 65535, T * (Hq + 2 Hkv) < 2^31; factor finite.  One launch.  Serving only:
 * the library trains nothing, and has no backward passes.
 */
int bastion_qk_norm_rope(int dtype, int T, int Hq, int Hkv, int D, const void *q, int64_t q_st_t,
                         int64_t q_st_h, const void *k, int64_t k_st_t, int64_t k_st_h,
                         const void *v, int64_t v_st_t, int64_t v_st_h, const void *q_weight,
                         const void *k_weight, float eps, const int32_t *pos,
                         const double *inv_freq, int rot_dim, int interleaved, float factor,
                         void *q_out, int64_t q_out_st_t, int64_t q_out_st_h, void *k_out,
                         int64_t k_out_st_t, int64_t k_out_st_h, const bastion_paged_cache *cache,
                         const int64_t *slots, int32_t *status, bastion_stream_t stream);

/* ---------------------------------------------------------------------------
 * Attention of one new token per request, over a prefix that its group of
 * requests shares and then its own used slots: bastion_paged_attention over
 * both, with the prefix's keys and values read once for the whole group.
 *
 * prefix_table  [n_groups, max_prefix_pages] int32: the pages of each group's
 *               prefix, in the cache's pools.
 * prefix_len    [n_groups] int32: the prefix's slots.
 * group_start   [n_groups+1] int32, ascending: group g is the requests
 *               group_start[g] .. group_start[g+1] - 1.  A request of no group
 *               attends to its own slots alone.  A group outside [0, B], or that
 *               ends before it begins, is left out and sets
 *               BASTION_STATUS_BAD_GROUP (in the status of its first request, taken
 *               to the nearest of the batch); what a group shares with the groups
 *               before it, up to the largest end among them, is not its own.
 * cache, q, seq_len, scale, out, lse, status: as bastion_paged_attention; the
 *               cache's page_table and seq_len are of the request's own slots, and
 *               q_stride_b is at least Hq * D.
 *               A group's prefix_len outside [0, max_prefix_pages * page_size] or
 *               page outside the pool sets its first request's status bit.
 * Limits: as bastion_paged_attention; 1 <= n_groups <= 1024, max_prefix_pages *
 * page_size <= 2^28, Hkv * ceil(max_prefix_pages * page_size / 128) * (n_groups +
 * B * Hq / Hkv / 112) < 2^31 (BASTION_ERR_SIZE).
 * Weights enter the products as there: as two 16-bit terms.  The prefix's sums
 * are formed in 32 bits by instructions that cut where others round, in chains of
 * at most 8,192 keys a row (16,384 in two interleaved halves): an output lacks 2^-15
 * of itself at most on average, whatever the prefix's length.  Results do not
 * depend on the order in which the parts of a split prefix finish.
 * Workspace: bastion_paged_prefix_attention_workspace_bytes(B, Hq, Hkv, D,
 * n_groups) bytes, about 12 bytes an element of q and 55 MB.  Three launches: own
 * slots, prefixes, join, 10 us at the least.  bastion_paged_attention with the
 * prefix's pages in every request's table, one launch that reads them once a
 * request, is faster where requests are few or the prefix is short: with 8 KV
 * heads of 128, 4 queries each and 32 own slots up to a prefix of 16,384 slots for 2
 * requests, 4,096 for 4, 1,024 for 8, 512 for 16 and 320 for 64 (512 own slots:
 * 16,384, 8,192, 4,096, 2,048 and 512); with 2 KV heads of 64, 7 queries each, past
 * 16,384 for up to 8 requests, to 2,048 for 16 and 320 for 64.
 */
size_t bastion_paged_prefix_attention_workspace_bytes(int B, int Hq, int Hkv, int D, int n_groups);
int bastion_paged_prefix_attention(const bastion_paged_cache *cache, const int32_t *prefix_table,
                                   int max_prefix_pages, const int32_t *prefix_len,
                                   const int32_t *group_start, int n_groups, const void *q, int Hq,
                                   int64_t q_stride_b, const int32_t *seq_len, float scale,
                                   void *out, float *lse, void *workspace, size_t workspace_bytes,
                                   int32_t *status, bastion_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BASTION_CACHE_H_ */
