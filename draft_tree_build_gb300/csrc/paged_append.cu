// Append to the paged cache: the rows of new tokens (a prompt, a token, or the
// accepted root path of a verified tree) are copied into the request's next
// slots.  A copy, bound by HBM: each row is read once and written once, 16
// bytes a thread with eight loads in flight, consecutive threads on consecutive
// bytes of a row (rows of 2 * D bytes, or Hkv of them in a slot-major pool).
// Prompts (8 requests of up to 8,192 tokens, 292 MB both ways): 50.0 us, 86% of
// the copy bandwidth (four loads in flight: 3% slower).  The accepted paths of 32
// requests (17 rows): 4.0 us, a launch and three dependent reads (as a captured graph
// replays them; a call from Python takes the host 8.4).
#include "paged.cuh"

namespace bastion {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 16;  // rows of one CTA
constexpr int kVecs = 4;      // 16-byte vectors of K, and of V, that a thread has in flight

struct AppendArgs {
  const uint16_t *k_new, *v_new;
  int64_t st_b, st_row, st_head;
  const int32_t *rows, *n_new, *seq_len, *n_seen;
  int32_t *seq_len_out, *n_seen_out;
  float *acc;
  int32_t *pos;
  int n_rows, m, T;  // T rows per CTA
  uint32_t *arrived;
  int32_t *status;
};

__global__ void __launch_bounds__(kThreads) paged_append_kernel(Paged c, AppendArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int r = blockIdx.y, tid = threadIdx.x;
  __shared__ int s_count;
  __shared__ int64_t s_src[kMaxRows], s_dst[kMaxRows];  // element offsets; dst < 0: skipped
  const int start = a.seq_len[r], seen = a.n_seen ? a.n_seen[r] : 0;
  const int limit = a.n_new ? min(a.m, max(a.n_new[r], 0)) : a.m;
  int count = limit;
  if (a.rows) {  // the first negative entry ends the list
    if (tid == 0) s_count = limit;
    __syncthreads();
    for (int i = tid; i < limit; i += kThreads)
      if (a.rows[(size_t)r * a.m + i] < 0) {
        atomicMin(&s_count, i);
        break;
      }
    __syncthreads();
    count = s_count;
  }
  if (start < 0 || (int64_t)start + count > c.cap) {
    if (tid == 0 && blockIdx.x == 0) atomicOr(&a.status[r], BASTION_STATUS_KV_OVERFLOW);
    count = 0;
  }
  const int i0 = blockIdx.x * a.T, n = min(a.T, count - i0);
  if (tid < n) {
    const int i = i0 + tid, slot = start + i;
    const int row = a.rows ? a.rows[(size_t)r * a.m + i] : i;
    int64_t dst = -1;
    if (row >= a.n_rows) {
      atomicOr(&a.status[r], BASTION_STATUS_BAD_ROW);
    } else {
      const int p = paged_page(c, r, slot, a.status);
      if (p >= 0) dst = paged_row(c, p, slot, 0);
    }
    s_src[tid] = r * a.st_b + (int64_t)row * a.st_row;
    s_dst[tid] = dst;
  }
  __syncthreads();
  if (n > 0) {
    // vector v of the CTA's rows: 16 bytes of row v / (Hkv * D / 8), K and V alike
    const int dv = c.D >> 3, per_row = c.Hkv * dv, dsh = c.D == 128 ? 4 : 3;
    const int total = n * per_row;
    for (int v0 = tid; v0 < total; v0 += kVecs * kThreads) {
      uint4 kk[kVecs], vv[kVecs];
      int64_t dst[kVecs];
#pragma unroll
      for (int u = 0; u < kVecs; ++u) {
        const int v = v0 + u * kThreads;
        dst[u] = -1;
        if (v < total) {
          const int i = v / per_row, w = v - i * per_row, h = w >> dsh, d = (w & (dv - 1)) * 8;
          if (s_dst[i] >= 0) {
            dst[u] = s_dst[i] + h * c.st_head + d;
            const int64_t src = s_src[i] + h * a.st_head + d;
            kk[u] = ld_stream_v4(a.k_new + src);
            vv[u] = ld_stream_v4(a.v_new + src);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kVecs; ++u)
        if (dst[u] >= 0) {
          *reinterpret_cast<uint4 *>(c.k + dst[u]) = kk[u];
          *reinterpret_cast<uint4 *>(c.v + dst[u]) = vv[u];
        }
    }
    if (a.acc) {
      for (int v = tid; v < n * c.Hkv; v += kThreads) {
        const int h = v / n, i = v - h * n;
        const size_t at = ((size_t)r * c.Hkv + h) * c.cap + start + i0 + i;
        a.acc[at] = 0.f;
        a.pos[at] = seen + i0 + i;
      }
    }
  }
  // the lengths may be updated in place: the request's last CTA writes them,
  // after every CTA of the request has read them
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    if (atomicAdd(&a.arrived[r], 1u) == gridDim.x - 1) {
      a.arrived[r] = 0;
      a.seq_len_out[r] = start + count;
      if (a.n_seen) a.n_seen_out[r] = seen + count;
    }
  }
}

}  // namespace

int launch_paged_append(const Paged &c, const void *k_new, const void *v_new, int n_rows, int64_t st_b,
                        int64_t st_row, int64_t st_head, const int32_t *rows, int m, const int32_t *n_new,
                        const int32_t *seq_len, int32_t *seq_len_out, const int32_t *n_seen,
                        int32_t *n_seen_out, float *acc, int32_t *pos, void *ws, int32_t *status,
                        cudaStream_t stream) {
  AppendArgs a;
  a.k_new = static_cast<const uint16_t *>(k_new);
  a.v_new = static_cast<const uint16_t *>(v_new);
  a.st_b = st_b;
  a.st_row = st_row;
  a.st_head = st_head;
  a.rows = rows;
  a.n_new = n_new;
  a.seq_len = seq_len;
  a.n_seen = n_seen;
  a.seq_len_out = seq_len_out;
  a.n_seen_out = n_seen_out;
  a.acc = acc;
  a.pos = pos;
  a.n_rows = n_rows;
  a.m = m;
  a.arrived = static_cast<uint32_t *>(ws);
  a.status = status;
  // fewer rows a CTA while the device has SMs to spare (17 rows of 32 requests: 5.7 us with 16, 4.5 with 8, 4.2 with 4, 2
  // and the 1 that this takes; prompts of 8 x 8,192 rows: 51 us with 16, as this takes, 56 with 8, 69 with 4)
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return BASTION_ERR_LAUNCH;
  a.T = kMaxRows;
  while (a.T > 1 && (int64_t)c.B * ((m + a.T - 1) / a.T) < 2 * sms) a.T /= 2;
  const dim3 grid((unsigned)((m + a.T - 1) / a.T), (unsigned)c.B);
  const cudaError_t e = launch_pdl(paged_append_kernel, grid, dim3(kThreads), 0, stream, c, a);
  return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? BASTION_OK : BASTION_ERR_LAUNCH;
}

}  // namespace bastion
