// Attention of one new token per request over its group's shared prefix and its
// own slots.  A warp a query head: lane = D / 32 elements of the head, one key
// after the other with a running maximum and sum.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged.cuh"

namespace bastion {

namespace {

constexpr int kThreads = 256;

struct PrefixArgs {
  const int32_t *table, *len, *start;  // the groups' prefixes
  int n_groups, max_pages, cap;
  const uint16_t *q;
  int64_t q_st_b;
  int Hq, G;
  const int32_t *seq_len;
  float scale;
  uint16_t *out;
  float *lse;
  int32_t *status;
};

template <bool kHalf>
__device__ __forceinline__ float to32(uint16_t x) {
  return kHalf ? __half2float(__ushort_as_half(x)) : __bfloat162float(__ushort_as_bfloat16(x));
}
template <bool kHalf>
__device__ __forceinline__ uint16_t to16(float x) {
  return kHalf ? __half_as_ushort(__float2half_rn(x)) : __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

__device__ __forceinline__ bool group_ok(const PrefixArgs &a, int B, int g) {
  const int x = a.start[g], y = a.start[g + 1];
  return x >= 0 && x <= y && y <= B;
}

template <bool kHalf, int D>
__global__ void __launch_bounds__(kThreads) paged_prefix_simple(Paged c, PrefixArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, row = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (blockIdx.x == 0)
    for (int g = threadIdx.x; g < a.n_groups; g += kThreads) {
      const int first = min(max(a.start[g], 0), c.B - 1);
      if (!group_ok(a, c.B, g)) atomicOr(&a.status[first], BASTION_STATUS_BAD_GROUP);
      else if (a.start[g] < a.start[g + 1] && (a.len[g] < 0 || a.len[g] > a.cap)) atomicOr(&a.status[first], BASTION_STATUS_KV_OVERFLOW);
    }
  if (row >= c.B * a.Hq) return;
  const int r = row / a.Hq, h = row % a.Hq, head = h / a.G;
  int g = -1;
  for (int g0 = 0; g0 < a.n_groups && g < 0; g0 += 32) {
    const int x = g0 + lane;
    const bool on = x < a.n_groups && group_ok(a, c.B, x) && a.start[x] <= r && r < a.start[x + 1];
    const unsigned m = __ballot_sync(kFull, on);
    if (m) g = g0 + __ffs(m) - 1;
  }
  constexpr int E = D / 32;
  float q[E], o[E] = {}, top = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) q[e] = to32<kHalf>(a.q[r * a.q_st_b + (int64_t)h * D + lane + 32 * e]);
  auto over = [&](const int32_t *table, int n, int told) {
    int page = 0;
    for (int j = 0; j < n; ++j) {
      if ((j & (c.page - 1)) == 0) {
        page = table[j >> c.shift];
        if (page < 0 || page >= c.n_pages) {
          if (lane == 0) atomicOr(&a.status[told], BASTION_STATUS_BAD_PAGE);
          page = 0;
        }
      }
      const int64_t at = paged_row(c, page, j, head) + lane;
      float s = 0.f;
      for (int e = 0; e < E; ++e) s += q[e] * to32<kHalf>(c.k[at + 32 * e]);
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(kFull, s, x);
      s *= a.scale;
      const float m = fmaxf(top, s);
      if (m == -INFINITY && s == s) continue;
      const float f = expf(top - m), p = expf(s - m);
      l = l * f + p;
      for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * to32<kHalf>(c.v[at + 32 * e]);
      top = m;
    }
  };
  if (g >= 0) over(a.table + (int64_t)g * a.max_pages, min(max(a.len[g], 0), a.cap), a.start[g]);
  over(c.table + (int64_t)r * c.max_pages, paged_len(c, a.seq_len, r, a.status), r);
  for (int e = 0; e < E; ++e) a.out[(int64_t)row * D + lane + 32 * e] = to16<kHalf>(l == 0.f ? 0.f : o[e] / l);
  if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : top + logf(l);
}

}  // namespace

size_t paged_prefix_workspace_bytes(int B, int Hq, int Hkv, int D, int n_groups) { return kCounterBytes; }

int launch_paged_prefix(const Paged &c, bool half, const int32_t *prefix_table, int max_prefix_pages,
                        const int32_t *prefix_len, const int32_t *group_start, int n_groups, const void *q, int Hq,
                        int64_t q_st_b, const int32_t *seq_len, float scale, void *out, float *lse, void *ws,
                        int32_t *status, cudaStream_t stream) {
  PrefixArgs a;
  a.table = prefix_table;
  a.len = prefix_len;
  a.start = group_start;
  a.n_groups = n_groups;
  a.max_pages = max_prefix_pages;
  a.cap = max_prefix_pages * c.page;
  a.q = static_cast<const uint16_t *>(q);
  a.q_st_b = q_st_b;
  a.Hq = Hq;
  a.G = Hq / c.Hkv;
  a.seq_len = seq_len;
  a.scale = scale;
  a.out = static_cast<uint16_t *>(out);
  a.lse = lse;
  a.status = status;
  const dim3 grid((unsigned)((c.B * Hq + 7) / 8));
  const cudaError_t e =
      half ? (c.D == 128 ? launch_pdl(paged_prefix_simple<true, 128>, grid, dim3(kThreads), 0, stream, c, a)
                         : launch_pdl(paged_prefix_simple<true, 64>, grid, dim3(kThreads), 0, stream, c, a))
           : (c.D == 128 ? launch_pdl(paged_prefix_simple<false, 128>, grid, dim3(kThreads), 0, stream, c, a)
                         : launch_pdl(paged_prefix_simple<false, 64>, grid, dim3(kThreads), 0, stream, c, a));
  return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? BASTION_OK : BASTION_ERR_LAUNCH;
}

}  // namespace bastion
