// Attention over short own slots, for the join of shared-prefix attention: outputs in
// 32 bits and the logarithms of their sums in base 2, as the one-token kernel of
// paged_attention.cu leaves them.
//
// Behind a long prefix the own slots are few, and what the one-token kernel does for
// long rows (persistent CTAs, rings of 128-key tiles, parts) costs it 2 us a request
// and KV head.  Here a warp, or a CTA of four or eight, takes a request and KV head (a unit), and
// enough of them are on an SM to hide one another's latency.  A tile of the tensor cores' asynchronous
// instructions (128 rows or keys) would be nearly empty, and its chain of copy, product,
// softmax, product is latency that a few keys cannot hide: a warp takes 16 keys at a time
// from global memory straight into the fragments of synchronous products, m16n8k16,
// whose 16 rows are the G query heads:
//  * S = Q K^T: a dot product does not mind the order of its elements, so that thread t
//    of a key's four takes 16-byte pieces t, t + 4, ... of the key, and of Q likewise;
//  * O += P V: S comes out as P goes in.  A thread takes 16-byte pieces of four value
//    rows, of whose elements it pairs two keys' each; the output's columns are in the
//    pieces' order.
// P is a high and a low 16-bit term, as in the other attention kernels.
#include "paged_prefix.cuh"
#include "paged_tc.cuh"

namespace bastion {

namespace {

constexpr int warps_of(int share) { return share > 4 ? share : 4; }  // of a CTA
constexpr int kTurn = 16;  // keys of a warp's turn

// D (16 x 8, 32 bits) += A (16 x 16) B (16 x 8), 16-bit A and B.
template <bool kHalf>
__device__ __forceinline__ void product(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kHalf)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool kHalf, int D, int kShare, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, (D == 64 ? 16 : 8) / kWarps) paged_prefix_own(Paged c, PrefixArgs a) {
  constexpr float kBias = kHalf ? 6.0f : 0.0f;  // weights are scaled by 2^kBias: a low term ends at 2^-24
  constexpr int kQk = D / 32, kPv = D / 64;     // 16-byte pieces of a key, of a value row, that a thread has
  __shared__ int s_pages[kWarps / kShare][own_slots(D) / 8];
  __shared__ float2 s_ml[kShare == 1 ? 1 : kWarps][16];
  __shared__ __align__(16) float s_o[kShare == 1 ? 1 : kWarps][16][D];
  griddep_wait();  // first: the prefix launch, which follows, counts on it
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int warp = (threadIdx.x >> 5) % kShare, tid = threadIdx.x % (32 * kShare);  // of the unit's
  const int place = threadIdx.x / (32 * kShare), unit = blockIdx.x * (kWarps / kShare) + place;
  if (unit >= c.B * c.Hkv) return;  // with kShare == 1 only, where warps do not wait for one another
  const int b = unit / c.Hkv, head = unit - b * c.Hkv;
  int *s_page = s_pages[place];
  const int n_raw = a.seq_len[b], n = min(max(n_raw, 0), c.cap);
  if (tid == 0 && head == 0 && n != n_raw) atomicOr(&a.status[b], BASTION_STATUS_KV_OVERFLOW);
  // rows g and g + 8 of Q; k step 2 i + e: words 2 e and 2 e + 1 of piece i
  uint4 q[2][kQk];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int i = 0; i < kQk; ++i) {
      q[r][i] = make_uint4(0, 0, 0, 0);
      if (g + 8 * r < a.G)
        q[r][i] = *reinterpret_cast<const uint4 *>(a.q + b * a.q_st_b + ((int64_t)head * a.G + g + 8 * r) * D + i * 32 + t * 8);
    }
  for (int i = tid; (i << c.shift) < n; i += 32 * kShare) {
    int p = c.table[(size_t)b * c.max_pages + i];
    if (p < 0 || p >= c.n_pages) {  // no page of the pool: page 0 stands in
      atomicOr(&a.status[b], BASTION_STATUS_BAD_PAGE);
      p = 0;
    }
    s_page[i] = p;
  }
  float o[kPv * 8][4] = {};  // [piece][element]: rows g (0, 1) and g + 8 (2, 3), columns 2 t and 2 t + 1
  float ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  if (kShare == 1) __syncwarp(); else __syncthreads();
#pragma unroll 1
  for (int j0 = warp * kTurn; j0 < n; j0 += kShare * kTurn) {
    uint4 kk[2][kQk], vv[4][kPv];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int j = j0 + 8 * x + g;
      const uint16_t *src = c.k + paged_row(c, s_page[min(j, n - 1) >> c.shift], j, head) + t * 8;
#pragma unroll
      for (int i = 0; i < kQk; ++i) {
        kk[x][i] = make_uint4(0, 0, 0, 0);
        if (j < n) kk[x][i] = ld_stream_v4(src + i * 32);
      }
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int j = j0 + 2 * t + (x & 1) + 8 * (x >> 1);
      const uint16_t *src = c.v + paged_row(c, s_page[min(j, n - 1) >> c.shift], j, head) + g * 8;
#pragma unroll
      for (int i = 0; i < kPv; ++i) {
        vv[x][i] = make_uint4(0, 0, 0, 0);  // past the end: weight 0 of value 0, whatever the slot holds
        if (j < n) vv[x][i] = ld_stream_v4(src + i * 64);
      }
    }
    float s[2][4] = {};  // keys 8 x + 2 t and + 1 of rows g (0, 1) and g + 8 (2, 3)
#pragma unroll
    for (int i = 0; i < kQk; ++i) {
      const uint32_t lo[4] = {q[0][i].x, q[1][i].x, q[0][i].y, q[1][i].y}, hi[4] = {q[0][i].z, q[1][i].z, q[0][i].w, q[1][i].w};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        product<kHalf>(s[x], lo, kk[x][i].x, kk[x][i].y);
        product<kHalf>(s[x], hi, kk[x][i].z, kk[x][i].w);
      }
    }
    uint32_t p_hi[4], p_lo[4];  // as A: rows g, g + 8 of keys 2 t, 2 t + 1; then of 2 t + 8, 2 t + 9
    float alpha[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float y[4];
      float top = -INFINITY;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int j = j0 + 8 * (x >> 1) + 2 * t + (x & 1);
        y[x] = j < n ? s[x >> 1][2 * r + (x & 1)] * a.scale_log2 : -INFINITY;
        top = fmaxf(top, y[x]);
      }
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
      const float to = fmaxf(ref[r], top - kBias), base = to == -INFINITY ? 0.f : to;
      alpha[r] = to == ref[r] ? 1.f : exp2f(ref[r] - to);
      ref[r] = to;
      l[r] *= alpha[r];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        y[x] = exp2f(y[x] - base);
        l[r] += y[x];
      }
      split2<kHalf>(y[0], y[1], p_hi[r], p_lo[r]);
      split2<kHalf>(y[2], y[3], p_hi[2 + r], p_lo[2 + r]);
    }
    if (__any_sync(kFull, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
      for (int x = 0; x < kPv * 8; ++x) {
        o[x][0] *= alpha[0];
        o[x][1] *= alpha[0];
        o[x][2] *= alpha[1];
        o[x][3] *= alpha[1];
      }
    }
#pragma unroll
    for (int i = 0; i < kPv; ++i) {
      const uint32_t w[4][4] = {{vv[0][i].x, vv[0][i].y, vv[0][i].z, vv[0][i].w}, {vv[1][i].x, vv[1][i].y, vv[1][i].z, vv[1][i].w},
                                {vv[2][i].x, vv[2][i].y, vv[2][i].z, vv[2][i].w}, {vv[3][i].x, vv[3][i].y, vv[3][i].z, vv[3][i].w}};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t sel = e & 1 ? 0x7632 : 0x5410;
        const uint32_t b0 = __byte_perm(w[0][e / 2], w[1][e / 2], sel), b1 = __byte_perm(w[2][e / 2], w[3][e / 2], sel);
        product<kHalf>(o[i * 8 + e], p_hi, b0, b1);
        product<kHalf>(o[i * 8 + e], p_lo, b0, b1);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(kFull, l[r], 1);
    l[r] += __shfl_xor_sync(kFull, l[r], 2);
    if (kShare == 1) {  // the row is whole
      if (g + 8 * r < a.G) {
        const size_t row = (size_t)b * a.Hq + (size_t)head * a.G + g + 8 * r;
        const float inv = l[r] == 0.f ? 0.f : __fdividef(1.f, l[r]);  // no key with a score above -inf: 0
#pragma unroll
        for (int i = 0; i < kPv; ++i)
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
              const int k = 2 * r + y;
              float4 x = make_float4(o[i * 8 + e][k], o[i * 8 + e + 1][k], o[i * 8 + e + 2][k], o[i * 8 + e + 3][k]);
              x = l[r] == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
              *reinterpret_cast<float4 *>(a.own + row * D + i * 64 + (2 * t + y) * 8 + e) = x;
            }
        if (t == 0) a.own_lse[row] = l[r] == 0.f ? -INFINITY : ref[r] + log2f(l[r]);
      }
      continue;
    }
    if (t == 0) s_ml[warp][g + 8 * r] = make_float2(ref[r], l[r]);
    // column 2 t + y of piece i, element e: element i * 64 + (2 t + y) * 8 + e of the head
    if (g + 8 * r < a.G) {
#pragma unroll
      for (int i = 0; i < kPv; ++i)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            const int k = 2 * r + y;
            *reinterpret_cast<float4 *>(&s_o[warp][g + 8 * r][i * 64 + (2 * t + y) * 8 + e]) =
                make_float4(o[i * 8 + e][k], o[i * 8 + e + 1][k], o[i * 8 + e + 2][k], o[i * 8 + e + 3][k]);
          }
    }
  }
  if (kShare == 1) return;
  __syncthreads();
  for (int i = tid; i < a.G * (D / 4); i += 32 * kShare) {
    const int h = i / (D / 4), quad = i - h * (D / 4);
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kShare; ++w) top = fmaxf(top, s_ml[w][h].x);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kShare; ++w) {
      const float2 ml = s_ml[w][h];
      // a warp without a finite score: nothing, or NaN
      const float f = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : exp2f(ml.x - top);
      const float4 x = *reinterpret_cast<const float4 *>(&s_o[w][h][quad * 4]);
      sum += f * ml.y;
      acc = make_float4(acc.x + f * x.x, acc.y + f * x.y, acc.z + f * x.z, acc.w + f * x.w);
    }
    const float inv = sum == 0.f ? 0.f : __fdividef(1.f, sum);  // no key with a score above -inf: 0
    const size_t row = (size_t)b * a.Hq + (size_t)head * a.G + h;
    *reinterpret_cast<float4 *>(a.own + row * D + quad * 4) =
        sum == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (quad == 0) a.own_lse[row] = sum == 0.f ? -INFINITY : top + log2f(sum);
  }
}

template <bool kHalf, int D, int kShare>
cudaError_t launch_share(const Paged &c, const PrefixArgs &a, cudaStream_t stream) {
  constexpr int kWarps = warps_of(kShare), kUnits = kWarps / kShare;
  return launch_pdl(paged_prefix_own<kHalf, D, kShare, kWarps>, dim3((unsigned)((c.B * c.Hkv + kUnits - 1) / kUnits)),
                    dim3(32 * kWarps), 0, stream, c, a);
}

// Warps of a unit: one where keys are few (16 slots, 150 requests of 32/8 heads of 64: 22.9 us for 27.0 with four) or
// units many (256 slots, 256 requests: 49.8 for 54.6); eight where the units are one wave (512 slots, 8 requests: 20.5 for
// 23.6); else four (256 slots, 64 requests: 25.3 for 35.7 with one, 33.6 with eight).
template <bool kHalf>
cudaError_t launch(int sms, const Paged &c, const PrefixArgs &a, cudaStream_t stream) {
  static_assert(own_slots(128) <= 64, "D = 128: one warp");
  if (c.D == 128) return launch_share<kHalf, 128, 1>(c, a, stream);
  const int units = c.B * c.Hkv;
  if (c.cap <= 64 || units >= 12 * sms) return launch_share<kHalf, 64, 1>(c, a, stream);
  return units <= 2 * sms ? launch_share<kHalf, 64, 8>(c, a, stream) : launch_share<kHalf, 64, 4>(c, a, stream);
}

}  // namespace

cudaError_t launch_prefix_own(bool half, int sms, const Paged &c, const PrefixArgs &a, cudaStream_t stream) {
  return half ? launch<true>(sms, c, a, stream) : launch<false>(sms, c, a, stream);
}

}  // namespace bastion
