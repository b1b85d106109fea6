// Page plan: which pages and slots the requests' next tokens get, from their
// lengths alone.
//
//   need = ceil((n + c) / page), back = max(0, held - need), more = max(0, need - held)
//
// The free pages are a stack.  With R pages given back in all, the x-th page
// taken is the stack's entry n_free + R - 1 - x, where entries from n_free on
// are the pages given back, in request order: prefix sums of back and more over
// the requests say which page goes where, and no request waits for another.
//
// Bound by latency: 12 bytes a row are nothing (2.9 MB in the largest case),
// what counts is the launch and the dependent reads of lengths, free list and
// table.  So there is one launch: every CTA forms the sums of all requests (at
// most 4 a thread) and then writes its share of the rows, four a thread, and of
// the table.  Nothing that a CTA writes is read by another: table entries from
// held on, and free entries from n_free on, are only written.  The lengths, which
// may be updated in place, are written by the last CTA to have read them.
#include "paged.cuh"

namespace bastion {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = kMaxRequests / kThreads;  // requests of a thread, at most

struct PlanArgs {
  int32_t *table;
  int B, max_pages, page, shift, cap, m, trim;
  int64_t n_pages, n_rows;
  const int32_t *seq_len, *n_new, *held, *n_free;
  const int32_t *offset;  // null, or what is added to each request's positions
  int32_t *seq_len_out, *held_out, *n_free_out, *free_pages;
  int64_t *slots;
  int32_t *pos, *row_start;
  int vec;  // slots and pos are 16-byte aligned
  uint32_t *arrived;
  int32_t *status;
};

// Exclusive prefix sums over the threads, in order, of N values at once; the totals in all.
template <int N>
__device__ __forceinline__ void scan(int64_t (&x)[N], int64_t (*warp_sum)[kThreads / 32], int64_t (&all)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t y[N];
#pragma unroll
  for (int k = 0; k < N; ++k) y[k] = x[k];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int64_t z = __shfl_up_sync(kFull, y[k], o);
      if (lane >= o) y[k] += z;
    }
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (lane == 31) warp_sum[k][warp] = y[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    int64_t before = 0;
    all[k] = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const int64_t z = warp_sum[k][w];
      before += w < warp ? z : 0;
      all[k] += z;
    }
    x[k] = before + y[k] - x[k];
  }
}

// The last of n ascending entries that is at most x.
template <typename T>
__device__ __forceinline__ int last_at_most(const T *a, int n, T x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) paged_plan_kernel(PlanArgs a) {
  // per request: used slots, pages held, pages needed, new rows, and what comes before it of
  // pages given back, pages taken and packed rows (one more entry: the totals)
  __shared__ int s_n[kMaxRequests], s_held[kMaxRequests], s_need[kMaxRequests], s_count[kMaxRequests], s_offset[kMaxRequests];
  __shared__ int64_t s_back[kMaxRequests + 1], s_more[kMaxRequests + 1];
  __shared__ int s_row[kMaxRequests + 1];
  __shared__ int64_t sums[4][kThreads / 32];
  __shared__ bool s_last;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, chunk = (a.B + kThreads - 1) / kThreads, r0 = tid * chunk;
  const bool tell = blockIdx.x == 0;
  int n[kPer], held[kPer], need[kPer], count[kPer], offset[kPer], bad[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = r0 + i;
    bad[i] = 0;
    n[i] = held[i] = need[i] = count[i] = offset[i] = 0;
    if (i >= chunk || r >= a.B) continue;
    n[i] = a.seq_len[r];
    held[i] = a.held[r];
    count[i] = a.n_new ? min(a.m, max(a.n_new[r], 0)) : a.m;
    if (a.offset) offset[i] = a.offset[r];
  }
  const int free_in = *a.n_free;
  const int64_t n_free = min((int64_t)max(free_in, 0), a.n_pages);
  // everything that may be updated in place has been read
  __syncthreads();
  if (tid == 0) {
    s_last = true;
    if (gridDim.x > 1) {
      __threadfence();
      s_last = atomicAdd(a.arrived, 1u) == gridDim.x - 1;
      if (s_last) *a.arrived = 0;
    }
    if (tell && n_free != free_in) atomicOr(&a.status[0], BASTION_STATUS_BAD_PAGE);
  }
  int64_t rows[1] = {0}, all[1];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (n[i] < 0 || (int64_t)n[i] + count[i] > a.cap || offset[i] < 0 || offset[i] > INT32_MAX - a.cap)
      bad[i] = BASTION_STATUS_KV_OVERFLOW;
    else if (held[i] < 0 || held[i] > a.max_pages || ((int64_t)held[i] << a.shift) < n[i]) bad[i] = BASTION_STATUS_BAD_PAGE;
    need[i] = bad[i] ? held[i] : (n[i] + count[i] + a.page - 1) >> a.shift;
    rows[0] += bad[i] ? 0 : count[i];
  }
  if (a.row_start) {  // packed rows: first come, first served
    scan(rows, &sums[0], all);
    int64_t at = rows[0];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (bad[i]) continue;
      at += count[i];
      if (count[i] > 0 && at > a.n_rows) {
        bad[i] = BASTION_STATUS_KV_OVERFLOW;
        need[i] = held[i];
      }
    }
  }
  int64_t both[2] = {0, 0}, totals[2];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (need[i] < held[i]) {
      if (a.trim) both[0] += held[i] - need[i];
      else need[i] = held[i];
    }
    both[1] += max(0, need[i] - held[i]);
  }
  scan(both, &sums[1], totals);
  int64_t back = both[0], more = both[1];
  const int64_t all_back = totals[0], all_more = totals[1], there = n_free + all_back;
  rows[0] = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = r0 + i;
    const bool here = i < chunk && r < a.B;
    if (here) {
      s_back[r] = back;
      s_more[r] = more;
    }
    back += max(0, held[i] - need[i]);
    const int k = max(0, need[i] - held[i]);
    more += k;
    if (k > 0 && more > there) {
      bad[i] = BASTION_STATUS_NO_PAGE;
      need[i] = held[i];
    }
    if (bad[i]) count[i] = 0;
    rows[0] += count[i];
    if (!here) continue;
    s_n[r] = n[i];
    s_held[r] = held[i];
    s_need[r] = need[i];
    s_count[r] = count[i];
    s_offset[r] = offset[i];
    if (bad[i] && tell) atomicOr(&a.status[r], bad[i]);
  }
  int total_rows = 0;  // at most n_rows
  if (a.row_start) {
    scan(rows, &sums[3], all);
    total_rows = (int)all[0];
    int row = (int)rows[0];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = r0 + i;
      if (i < chunk && r < a.B) {
        s_row[r] = row;
        if (tell) a.row_start[r] = row;
      }
      row += count[i];
    }
  }
  if (tid == 0) {
    s_back[a.B] = all_back;
    s_more[a.B] = all_more;
    s_row[a.B] = total_rows;
    if (a.row_start && tell) a.row_start[a.B] = total_rows;
  }
  __syncthreads();

  // the y-th page given back, and the request that gives it; the page of entry idx >= held of request r
  auto given_by = [&](int64_t y, int &r) {
    r = last_at_most(s_back, a.B, y);
    return a.table[(int64_t)r * a.max_pages + s_need[r] + (y - s_back[r])];
  };
  auto given = [&](int64_t y) {
    int r;
    return given_by(y, r);
  };
  auto taken = [&](int r, int idx) {
    const int64_t x = s_more[r] + (idx - s_held[r]);
    return x < all_back ? given(all_back - 1 - x) : a.free_pages[there - 1 - x];
  };

  // ------------------------------------------------------------ rows
  const int64_t stride = (int64_t)gridDim.x * kThreads, first = (int64_t)blockIdx.x * kThreads + tid;
  for (int64_t e = 4 * first; e < a.n_rows; e += 4 * stride) {
    int64_t slot[4];
    int pos[4];
    int r, i;
    if (a.row_start) {
      r = e < total_rows ? last_at_most(s_row, a.B, (int)e) : a.B;
      i = r < a.B ? (int)e - s_row[r] : 0;
    } else {
      r = (int)(e / a.m);
      i = (int)(e - (int64_t)r * a.m);
    }
    int last_idx = -1, page = -1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      slot[u] = -1;
      pos[u] = -1;
      if (r < a.B) {
        if (i < s_count[r]) {
          const int j = s_n[r] + i, idx = j >> a.shift;
          if (idx != last_idx) {
            page = idx < s_held[r] ? a.table[(int64_t)r * a.max_pages + idx] : taken(r, idx);
            last_idx = idx;
            if (page < 0 || page >= a.n_pages) {
              atomicOr(&a.status[r], BASTION_STATUS_BAD_PAGE);
              page = -1;
            }
          }
          pos[u] = s_offset[r] + j;
          if (page >= 0) slot[u] = ((int64_t)page << a.shift) + (j & (a.page - 1));
        }
        ++i;
        // on to the next request that has rows
        while (r < a.B && i >= (a.row_start ? s_count[r] : a.m)) {
          ++r;
          i = 0;
          last_idx = -1;
        }
      }
    }
    if (a.vec && e + 4 <= a.n_rows) {
      reinterpret_cast<longlong2 *>(a.slots + e)[0] = make_longlong2(slot[0], slot[1]);
      reinterpret_cast<longlong2 *>(a.slots + e)[1] = make_longlong2(slot[2], slot[3]);
      *reinterpret_cast<int4 *>(a.pos + e) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (e + u < a.n_rows) {
          a.slots[e + u] = slot[u];
          a.pos[e + u] = pos[u];
        }
    }
  }

  // ------------------------------------------------------------ table and free list
  const int64_t most = min(all_more, there);
  for (int64_t x = first; x < most; x += stride) {
    const int r = last_at_most(s_more, a.B, x), idx = s_held[r] + (int)(x - s_more[r]);
    if (idx >= s_need[r]) continue;  // refused
    const int p = taken(r, idx);
    a.table[(int64_t)r * a.max_pages + idx] = p;
    if (p < 0 || p >= a.n_pages) atomicOr(&a.status[r], BASTION_STATUS_BAD_PAGE);
  }
  // the first request that was refused, if any, is where the sum of pages passes what there is
  int64_t used = all_more;
  if (all_more > there) used = s_more[last_at_most(s_more, a.B + 1, there)];
  const int64_t left = there - used;
  for (int64_t y = first; y < all_back; y += stride) {  // those that other requests take at once are looked at, too
    int r;
    const int p = given_by(y, r);
    if (p < 0 || p >= a.n_pages) atomicOr(&a.status[r], BASTION_STATUS_BAD_PAGE);
    if (n_free + y < left && n_free + y < a.n_pages) a.free_pages[n_free + y] = p;
  }
  if (s_last) {
    for (int r = tid; r < a.B; r += kThreads) {
      a.held_out[r] = s_need[r];
      if (a.seq_len_out) a.seq_len_out[r] = s_n[r] + s_count[r];
    }
    if (tid == 0) {
      *a.n_free_out = (int)min(left, a.n_pages);
      if (left > a.n_pages) atomicOr(&a.status[0], BASTION_STATUS_BAD_PAGE);
    }
  }
}

}  // namespace

int launch_paged_plan(int32_t *table, int B, int max_pages, int page, int64_t n_pages, const int32_t *seq_len,
                      const int32_t *n_new, int m, int32_t *seq_len_out, const int32_t *held, int32_t *held_out,
                      int32_t *free_pages, const int32_t *n_free, int32_t *n_free_out, int trim, int64_t *slots,
                      int32_t *pos, int64_t n_rows, int32_t *row_start, const int32_t *pos_offset, void *ws,
                      int32_t *status, cudaStream_t stream) {
  PlanArgs a;
  a.offset = pos_offset;
  a.table = table;
  a.B = B;
  a.max_pages = max_pages;
  a.page = page;
  a.shift = 0;
  while ((1 << a.shift) < page) ++a.shift;
  a.cap = max_pages * page;
  a.m = m;
  a.trim = trim;
  a.n_pages = n_pages;
  a.n_rows = n_rows;
  a.seq_len = seq_len;
  a.n_new = n_new;
  a.held = held;
  a.n_free = n_free;
  a.seq_len_out = seq_len_out;
  a.held_out = held_out;
  a.n_free_out = n_free_out;
  a.free_pages = free_pages;
  a.slots = slots;
  a.pos = pos;
  a.row_start = row_start;
  a.vec = ((uintptr_t)slots % 16 == 0) && ((uintptr_t)pos % 16 == 0);
  a.arrived = static_cast<uint32_t *>(ws);
  a.status = status;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return BASTION_ERR_LAUNCH;
  const int64_t want = (n_rows + 4 * kThreads - 1) / (4 * kThreads), most = 2 * (int64_t)sms;
  const dim3 grid((unsigned)(want < most ? want : most));
  const cudaError_t e = launch_pdl(paged_plan_kernel, grid, dim3(kThreads), 0, stream, a);
  return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? BASTION_OK : BASTION_ERR_LAUNCH;
}

}  // namespace bastion
