// What the kernels of the paged cache share: its geometry on the device.
#pragma once

#include <atomic>

#include "bastion_cache.h"
#include "common.cuh"

namespace bastion {

// Every call's arrival counters lie in the first bytes of its workspace and
// nothing else does, so that calls of all sizes, and of all three kinds, can
// share one: 2 * kMaxParts counters of groups, then one per (request, KV head).
constexpr int kMaxParts = 192;      // CTAs of an attention launch, at most
constexpr int kMaxUnits = 65536;    // B * Hkv
constexpr int kMaxRequests = 1024;  // B
constexpr size_t kCounterBytes = (2 * kMaxParts + kMaxUnits) * sizeof(uint32_t);
static_assert(kCounterBytes % 256 == 0 && kCounterBytes >= kMaxRequests * sizeof(uint32_t), "counters");

struct Paged {
  uint16_t *k, *v;
  int64_t n_pages, st_page, st_slot, st_head;
  const int32_t *table;
  int B, Hkv, D, page, shift, max_pages;  // page = 1 << shift
  int cap;                                // max_pages * page
};

// The used slots of a request, in [0, cap]; a length outside it sets the status bit.
__device__ __forceinline__ int paged_len(const Paged &c, const int32_t *seq_len, int r, int32_t *status) {
  const int n = seq_len[r];
  if (n >= 0 && n <= c.cap) return n;
  atomicOr(&status[r], BASTION_STATUS_KV_OVERFLOW);
  return n < 0 ? 0 : c.cap;
}

// The page that holds slot j < cap of request r, or -1 (and the status bit)
// when the table's entry is not a page of the pool.
__device__ __forceinline__ int paged_page(const Paged &c, int r, int j, int32_t *status) {
  const int p = c.table[(size_t)r * c.max_pages + (j >> c.shift)];
  if (p >= 0 && p < c.n_pages) return p;
  atomicOr(&status[r], BASTION_STATUS_BAD_PAGE);
  return -1;
}

// Element offset of slot j's row of head h, given its page.
__device__ __forceinline__ int64_t paged_row(const Paged &c, int page, int j, int h) {
  return page * c.st_page + (int64_t)(j & (c.page - 1)) * c.st_slot + h * c.st_head;
}

Paged paged_args(const bastion_paged_cache &c);

// Lets a kernel have that much dynamic shared memory on device dev, once per
// device: asking again costs 0.4 us a call.  done: the kernel's own, a bit a device.
template <typename K>
inline cudaError_t allow_smem(K *kernel, int bytes, int dev, std::atomic<uint64_t> &done) {
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace bastion
