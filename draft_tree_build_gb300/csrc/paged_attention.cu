// Attention of one new token per request over the paged cache.
//
//   s_j = scale q.k_j, out = sum_j exp(s_j - lse) v_j, lse = log sum_j exp(s_j)
//
// One CTA per (request, query head): each warp takes every fourth key with a
// running maximum m, sum l and output o (o and l are rescaled by 2^(m - m')
// when the maximum moves), a lane holding D / 32 of the elements; the warps'
// parts are joined at the end.  With weights, the scores are kept and a second
// kernel adds sum_h exp(s - lse_h) to each slot's accumulated weight.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged.cuh"

namespace bastion {

namespace {

constexpr int kTileKeys = 128;
constexpr int kMaxUnits = 65536;       // B * Hkv
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct AttendArgs {
  const uint16_t *q;
  int64_t q_st_b;
  int Hq, G;
  const int32_t *seq_len;
  float scale_log2;
  uint16_t *out;
  float *lse;
  const float *acc;
  float *acc_out;
  float *lse2;    // [B, Hq] base-2 log of the sum, of the scores in base 2
  float *scores;  // [B, Hkv, tiles, G, 128], in base 2
  int tiles_cap;
  int32_t *status;
};

template <bool kHalf>
__device__ __forceinline__ float from16(uint16_t x) {
  return kHalf ? __half2float(__ushort_as_half(x)) : __uint_as_float((uint32_t)x << 16);
}
template <bool kHalf>
__device__ __forceinline__ uint16_t to16(float x) {
  return kHalf ? __half_as_ushort(__float2half_rn(x)) : __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

template <bool kHalf>
__global__ void __launch_bounds__(128) paged_attention_kernel(Paged c, AttendArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int r = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq, g = h / a.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = paged_len(c, a.seq_len, r, a.status);
  const int e = c.D >> 5;  // elements per lane: d = lane + 32 i
  float q[4], o[4] = {};
  for (int i = 0; i < e; ++i) q[i] = from16<kHalf>(a.q[r * a.q_st_b + h * c.D + lane + 32 * i]) * a.scale_log2;
  float m = -INFINITY, l = 0.f;
  for (int j = warp; j < n; j += 4) {
    const int p = paged_page(c, r, j, a.status);
    if (p < 0) continue;
    const int64_t row = paged_row(c, p, j, g);
    float s = 0.f;
    for (int i = 0; i < e; ++i) s += q[i] * from16<kHalf>(c.k[row + lane + 32 * i]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(kFull, s, x);
    if (a.scores && lane == 0)
      a.scores[((((size_t)r * c.Hkv + g) * a.tiles_cap + j / kTileKeys) * a.G + h % a.G) * kTileKeys + j % kTileKeys] = s;
    const float mn = fmaxf(m, s);
    const float f = m == -INFINITY ? 0.f : exp2f(m - mn), w = s == -INFINITY ? 0.f : exp2f(s - mn);
    l = l * f + w;
    for (int i = 0; i < e; ++i) o[i] = o[i] * f + w * from16<kHalf>(c.v[row + lane + 32 * i]);
    m = mn;
  }
  __shared__ float s_m[4], s_l[4], s_o[4][128];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  for (int i = 0; i < e; ++i) s_o[warp][lane + 32 * i] = o[i];
  __syncthreads();
  const float M = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  float L = 0.f, O = 0.f;
  const int d = threadIdx.x;
  for (int w = 0; w < 4; ++w) {
    const float f = s_m[w] == -INFINITY ? 0.f : exp2f(s_m[w] - M);
    L += s_l[w] * f;
    if (d < c.D) O += s_o[w][d] * f;
  }
  const float lse2 = L == 0.f ? -INFINITY : M + log2f(L);
  if (d < c.D) a.out[((size_t)r * a.Hq + h) * c.D + d] = to16<kHalf>(L == 0.f ? 0.f : O / L);
  if (d == 0) {
    if (a.lse) a.lse[(size_t)r * a.Hq + h] = lse2 * kLn2;
    if (a.acc) a.lse2[(size_t)r * a.Hq + h] = lse2;
  }
}

// acc_out = acc + sum over the group's heads of exp2(s - lse2), in head order.
__global__ void __launch_bounds__(256) paged_weights_kernel(Paged c, AttendArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int unit = blockIdx.y, r = unit / c.Hkv, g = unit % c.Hkv;
  const int j = blockIdx.x * 256 + threadIdx.x;
  int n = a.seq_len[r];
  n = min(max(n, 0), c.cap);
  if (j >= n) return;
  const float *s = a.scores + ((size_t)unit * a.tiles_cap + j / kTileKeys) * a.G * kTileKeys + j % kTileKeys;
  const float *lse2 = a.lse2 + (size_t)r * a.Hq + g * a.G;
  float w = 0.f;
  for (int h = 0; h < a.G; ++h) {
    const float x = lse2[h];
    if (x != -INFINITY) w += exp2f(s[h * kTileKeys] - x);
  }
  const size_t at = (size_t)unit * c.cap + j;
  a.acc_out[at] = a.acc[at] + w;
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

size_t paged_attention_workspace_bytes(int B, int Hq, int Hkv, int D, int64_t cap, int weights) {
  (void)D;
  size_t n = 256;
  if (weights) {
    n += up256((size_t)B * Hq * sizeof(float));
    n += (size_t)B * Hq * ((cap + kTileKeys - 1) / kTileKeys) * kTileKeys * sizeof(float);
  }
  return n;
}

int launch_paged_attention(const Paged &c, bool half, const void *q, int Hq, int64_t q_st_b, const int32_t *seq_len,
                           float scale, void *out, float *lse, const float *acc, float *acc_out, void *ws,
                           int32_t *status, cudaStream_t stream) {
  AttendArgs a;
  a.q = static_cast<const uint16_t *>(q);
  a.q_st_b = q_st_b;
  a.Hq = Hq;
  a.G = Hq / c.Hkv;
  a.seq_len = seq_len;
  a.scale_log2 = scale * kLog2e;
  a.out = static_cast<uint16_t *>(out);
  a.lse = lse;
  a.acc = acc;
  a.acc_out = acc_out;
  a.tiles_cap = (c.cap + kTileKeys - 1) / kTileKeys;
  a.lse2 = reinterpret_cast<float *>(static_cast<char *>(ws) + 256);
  a.scores = acc ? reinterpret_cast<float *>(static_cast<char *>(ws) + 256 + up256((size_t)c.B * Hq * 4)) : nullptr;
  a.status = status;
  cudaError_t e = launch_pdl(half ? paged_attention_kernel<true> : paged_attention_kernel<false>,
                             dim3((unsigned)(c.B * Hq)), dim3(128), 0, stream, c, a);
  if (e == cudaSuccess && acc)
    e = launch_pdl(paged_weights_kernel, dim3((unsigned)((c.cap + 255) / 256), (unsigned)(c.B * c.Hkv)), dim3(256), 0,
                   stream, c, a);
  return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? BASTION_OK : BASTION_ERR_LAUNCH;
}

}  // namespace bastion
