// The join of shared-prefix attention: a row's parts scaled by the largest of their
// references and added, in the order of their keys, over the sum.  Bound by L2, where
// the parts lie: 512 bytes a part and row of 128 elements (20 parts a row where 64
// requests share one prefix, 21 MB).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged_prefix.cuh"

namespace bastion {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr float kLn2 = 0.6931471805599453f;

template <bool kHalf>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  if (kHalf) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 2^(part's reference - base), and 0 for a part that has seen nothing, whose rows do not count.
__device__ __forceinline__ float factor(float2 ml, float base) {
  if (ml.x == -INFINITY && ml.y == ml.y) return 0.f;
  return exp2f(ml.x == -INFINITY ? 0.f : ml.x - base);
}

// A row's parts: its own slots', then those of its prefix.  A thread takes kWide
// elements of a row, of every kSplit-th part, two parts in flight; the lanes of a
// warp are consecutive rows of a KV head, which lie side by side in the parts.  The
// CTAs are made for one wave (64 requests: 512 of them; 1,024 of half the width
// took 12 us for 7).
constexpr int kWide = 16, kFly = 2;
template <bool kHalf, int D, int kSplit>
__global__ void __launch_bounds__(kThreads, 3) paged_prefix_join(Paged c, PrefixArgs a) {
  __shared__ float s_ref[kWarps][32], s_sum[kWarps][32], s_o[kWarps][kWide][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part0 = warp % kSplit;
  const int i = blockIdx.x * 32 + lane, head = blockIdx.y, d0 = kWide * (blockIdx.z * (kWarps / kSplit) + warp / kSplit);
  const bool on = i < c.B * a.G;
  const int b = on ? i / a.G : 0, h = on ? i - b * a.G : 0;
  const size_t row = (size_t)b * a.Hq + head * a.G + h;
  griddep_wait();
  griddep_launch_dependents();
  const PartsRec x = a.rec[b * c.Hkv + head];
  const float *part = x.whole ? a.rows : a.parts;
  const float2 *part_ml = x.whole ? a.rows_ml : a.parts_ml;
  const int in_tile = x.first + h;
  float o[kWide] = {}, ref = -INFINITY, l = 0.f;
  if (on) {
    for (int p0 = part0; p0 <= x.parts; p0 += kFly * kSplit) {  // part 0 is the own slots', part p of the prefix p + 1
      float4 v[kFly][kWide / 4];
      float2 ml[kFly];
      float to = ref;
#pragma unroll
      for (int u = 0; u < kFly; ++u) {
        const int p = p0 + u * kSplit;
        ml[u] = make_float2(-INFINITY, 0.f);
        if (p > x.parts) continue;
        const float4 *src;
        int step = 1;
        if (p == 0) {
          ml[u] = make_float2(a.own_lse[row], 1.f);
          src = reinterpret_cast<const float4 *>(a.own + row * D + d0);
        } else {
          const int cta = (p - 1) >> x.two, plane = (p - 1) & x.two;
          const size_t place = (cta == 0 ? x.place0 : x.place1 + (cta - 1) * 512) + plane * x.step;
          ml[u] = __ldcg(part_ml + place + in_tile);
          src = reinterpret_cast<const float4 *>(part + place * D) + (d0 / 4) * x.rows + in_tile;
          step = x.rows;
        }
#pragma unroll
        for (int y = 0; y < kWide / 4; ++y) v[u][y] = __ldcg(src + y * step);
      }
#pragma unroll
      for (int u = 0; u < kFly; ++u) to = fmaxf(to, ml[u].x);
      const float base = to == -INFINITY ? 0.f : to, f0 = ref == -INFINITY ? 1.f : exp2f(ref - base);
      ref = to;
      l *= f0;
#pragma unroll
      for (int y = 0; y < kWide; ++y) o[y] *= f0;
#pragma unroll
      for (int u = 0; u < kFly; ++u) {
        const float f = factor(ml[u], base);
        if (f != 0.f) {
          l += f * ml[u].y;
#pragma unroll
          for (int y = 0; y < kWide / 4; ++y) {
            o[4 * y] += f * v[u][y].x;
            o[4 * y + 1] += f * v[u][y].y;
            o[4 * y + 2] += f * v[u][y].z;
            o[4 * y + 3] += f * v[u][y].w;
          }
        }
      }
    }
  }
  {
    s_ref[warp][lane] = ref;
    s_sum[warp][lane] = l;
#pragma unroll
    for (int y = 0; y < kWide; ++y) s_o[warp][y][lane] = o[y];
    __syncthreads();
    // the elements of a chunk are dealt to its warps
    constexpr int kMine = kWide / kSplit;
    const int w0 = warp - part0;
#pragma unroll
    for (int w = 0; w < kSplit; ++w) ref = fmaxf(ref, s_ref[w0 + w][lane]);
    const float base = ref == -INFINITY ? 0.f : ref;
    float r[kMine] = {};
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kSplit; ++w) {
      const float f = factor(make_float2(s_ref[w0 + w][lane], s_sum[w0 + w][lane]), base);
      if (f != 0.f) {
        l += f * s_sum[w0 + w][lane];
#pragma unroll
        for (int y = 0; y < kMine; ++y) r[y] += f * s_o[w0 + w][part0 * kMine + y][lane];
      }
    }
    if (!on) return;
    uint32_t z[kMine / 2];
#pragma unroll
    for (int y = 0; y < kMine; y += 2) z[y / 2] = l == 0.f ? 0u : pack<kHalf>(__fdividef(r[y], l), __fdividef(r[y + 1], l));
    uint16_t *dst = a.out + row * D + d0 + part0 * kMine;
    if (kMine == 2) *reinterpret_cast<uint32_t *>(dst) = z[0];
#pragma unroll
    for (int y = 0; y + 3 < kMine / 2; y += 4) *reinterpret_cast<uint4 *>(dst + 2 * y) = make_uint4(z[y], z[y + 1], z[y + 2], z[y + 3]);
  }
  if (a.lse && d0 == 0 && part0 == 0) a.lse[row] = l == 0.f ? -INFINITY : (ref + log2f(l)) * kLn2;
}

template <bool kHalf, int D>
cudaError_t launch(int sms, const Paged &c, const PrefixArgs &a, cudaStream_t stream) {
  // Eight warps to a row's parts where rows are few and their parts, then, many; else two.  Whole calls over 16,384 shared
  // tokens, 32/8 heads of 128, eight and two: 1,024 rows 31 and 40 us, 2,048 39.8 and 41.8, 2,560 48.7 and 49.5, 4,096 60.8 and
  // 59.4, 8,192 103 and 99.  (64-element heads over 2,048 tokens: 17.6 and 21.0 at 2,560 rows, 21.3 and 21.4 at 4,096.)
  const unsigned x = (unsigned)((c.B * a.G + 31) / 32), y = (unsigned)c.Hkv;
  return c.B * a.Hq <= 16 * sms ? launch_pdl(paged_prefix_join<kHalf, D, 8>, dim3(x, y, D / kWide), dim3(kThreads), 0, stream, c, a)
                                : launch_pdl(paged_prefix_join<kHalf, D, 2>, dim3(x, y, D / (4 * kWide)), dim3(kThreads), 0, stream, c, a);
}

}  // namespace

cudaError_t launch_prefix_join(bool half, int sms, const Paged &c, const PrefixArgs &a, cudaStream_t stream) {
  if (half) return c.D == 128 ? launch<true, 128>(sms, c, a, stream) : launch<true, 64>(sms, c, a, stream);
  return c.D == 128 ? launch<false, 128>(sms, c, a, stream) : launch<false, 64>(sms, c, a, stream);
}

}  // namespace bastion
