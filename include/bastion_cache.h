/*
 * bastion_cache.h -- the paged key-value cache of the target model: append,
 * one-token attention and eviction by accumulated attention weight.
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
 * One workspace that is large enough for each may serve all three calls, at
 * all sizes, one after the other.  A workspace that a call with
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
 * Scores, sums and outputs are accumulated in 32 bits.  A weight exp(s_j - lse)
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

#ifdef __cplusplus
}
#endif

#endif /* BASTION_CACHE_H_ */
