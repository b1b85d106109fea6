// Norm and rotation of queries and keys, and their way into the cache.
//
//   y = x / sqrt(mean(x^2) + eps) * w;  (a, b) -> factor (a cos t - b sin t, b cos t + a sin t),  t = pos f_i
//
// Bound by HBM: every element is read once and written once (a token of 32/8
// heads of 128: 24.6 KB both ways).  A warp takes a token, or a range of its
// heads where there are few tokens; 8 or 16 lanes hold a head, 16 bytes each, so
// that a head's sum of squares is 3 or 4 shuffles and its partner elements are in
// the lane itself (pairs 2i, 2i + 1) or one shuffle away (i, i + rot / 2).  Norm
// weights, cosines and sines fold into two factors an element, formed once per
// token and kind,
//   out_e = r (x_e A_e + x_partner B_e),  r = 1 / sqrt(mean + eps),
// so that a head costs 2 products and a sum an element.
//
// The angle is reduced exactly: f_i / 2 pi is held as a 64-bit fraction of a
// turn, and pos times it wraps modulo one turn by itself.  Its error is pos *
// 2^-53 f_i turns from f_i's own rounding, where a product in 32 bits would be off
// by pos * 2^-24 (6% of a radian at a million tokens).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged.cuh"

namespace bastion {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;  // 16-byte vectors that a lane has in flight

struct Strided {
  uint16_t *p;
  int64_t st_t, st_h;
};

struct RopeArgs {
  Strided q, k, v, q_out, k_out;
  const uint16_t *q_weight, *k_weight;
  float eps, factor;
  const int32_t *pos;
  const double *inv_freq;
  const int64_t *slots;
  int T, Hq, Hkv, rot;
  int chunks, per;  // a token's iterations are dealt to `chunks` warps, `per` each
  int32_t *status;
};

template <bool kHalf>
__device__ __forceinline__ float2 unpack(uint32_t w) {
  if (kHalf) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
  return make_float2(bf16lo(w), bf16hi(w));
}
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

template <bool kHalf, int D, bool kPairs>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(Paged c, RopeArgs a) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;  // lanes of a head, heads of a warp
  __shared__ uint64_t turn[D / 2];                     // of pair i per position, in 2^-64 turns
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  const int sub = lane % kLanes, head0 = lane / kLanes, half = a.rot / 2;
  for (int i = tid; i < half; i += kThreads) {
    const double x = a.inv_freq[i] * 0.15915494309189533577, f = x - floor(x);  // turns
    turn[i] = (uint64_t)__double2ull_rn(f * 18446744073709551616.0);
  }
  __syncthreads();
  const bool norm = a.q_weight != nullptr, turned = sub * 8 < a.rot;
  // the lane that holds the partners of this one's elements
  const int other = kPairs || !turned ? lane : sub * 8 < half ? lane + half / 8 : lane - half / 8;
  const int iq = (a.Hq + kHeads - 1) / kHeads, ik = (a.Hkv + kHeads - 1) / kHeads, iv = c.k ? ik : 0;
  const int items = a.T * a.chunks, warps = gridDim.x * (kThreads / 32);
  for (int item = blockIdx.x * (kThreads / 32) + (tid >> 5); item < items; item += warps) {
    const int t = item / a.chunks, from = (item - t * a.chunks) * a.per, to = min(from + a.per, iq + ik + iv);
    const int pos = a.pos ? a.pos[t] : 0;
    if (pos < 0) continue;
    int64_t slot = -1;  // element offset of the token's row in the pools
    if (c.k && to > iq) {
      slot = a.slots[t];
      if (slot >= 0) {
        const int64_t page = slot >> c.shift;
        if (page < c.n_pages) {
          slot = page * c.st_page + (slot & (c.page - 1)) * c.st_slot;
        } else {
          if (lane == 0) atomicOr(a.status, BASTION_STATUS_BAD_PAGE);
          slot = -1;
        }
      }
    }
    float cs[8], sn[8];  // factor * cos, and the sine with its sign
#pragma unroll
    for (int e = 0; e < 8; e += kPairs ? 2 : 1) {
      float cv = 1.f, sv = 0.f;
      if (turned) {
        const int x = sub * 8 + e, i = kPairs ? x >> 1 : x < half ? x : x - half;
        // the signed fraction of a turn, in half turns
        const float y = (float)(int32_t)((turn[i] * (uint64_t)(uint32_t)pos) >> 32) * 0x1p-31f;
        sincospif(y, &sv, &cv);
        cv *= a.factor;
        sv *= a.factor;
      }
      cs[e] = cv;
      if (kPairs) {
        cs[e + 1] = cv;
        sn[e] = -sv;
        sn[e + 1] = sv;
      } else {
        sn[e] = sub * 8 + e < half ? -sv : sv;
      }
    }
    auto kind = [&](const Strided &in, const Strided &out, const uint16_t *weight, int heads, int i0, int i1,
                    uint16_t *pool) {
      float A[8], B[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        A[e] = cs[e];
        B[e] = sn[e];
      }
      if (norm) {
        const uint4 w = *reinterpret_cast<const uint4 *>(weight + sub * 8);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float2 f = unpack<kHalf>(ww[e / 2]);
          const uint32_t pw = kPairs ? __byte_perm(ww[e / 2], 0, 0x1032) : __shfl_sync(kFull, ww[e / 2], other);
          const float2 g = unpack<kHalf>(pw);
          A[e] *= f.x;
          A[e + 1] *= f.y;
          B[e] *= g.x;
          B[e + 1] *= g.y;
        }
      }
      const uint16_t *src = in.p + t * in.st_t + sub * 8;
      for (int i = i0; i < i1; i += kRows) {
        uint4 x[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          const int h = (i + u) * kHeads + head0;
          x[u] = make_uint4(0, 0, 0, 0);
          if (i + u < i1 && h < heads) x[u] = *reinterpret_cast<const uint4 *>(src + h * in.st_h);
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          const int h = (i + u) * kHeads + head0;
          const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
          float y[8], r = 1.f;
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float2 f = unpack<kHalf>(w[e / 2]);
            y[e] = f.x;
            y[e + 1] = f.y;
          }
          if (norm) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s += y[e] * y[e];
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
            r = rsqrtf(s * (1.f / D) + a.eps);
          }
          uint32_t z[4];
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const uint32_t got = kPairs ? __byte_perm(w[e / 2], 0, 0x1032) : __shfl_sync(kFull, w[e / 2], other);
            float2 p = unpack<kHalf>(got);
            if (!turned) p = make_float2(0.f, 0.f);  // an infinity that is not turned stays one
            z[e / 2] = pack<kHalf>((y[e] * A[e] + p.x * B[e]) * r, (y[e + 1] * A[e + 1] + p.y * B[e + 1]) * r);
          }
          if (i + u < i1 && h < heads) {
            const uint4 zz = make_uint4(z[0], z[1], z[2], z[3]);
            if (out.p) *reinterpret_cast<uint4 *>(out.p + t * out.st_t + h * out.st_h + sub * 8) = zz;
            if (pool && slot >= 0) *reinterpret_cast<uint4 *>(pool + slot + h * c.st_head + sub * 8) = zz;
          }
        }
      }
    };
    if (from < iq && a.q_out.p) kind(a.q, a.q_out, a.q_weight, a.Hq, from, min(to, iq), nullptr);
    if (to > iq && from < iq + ik && (a.k_out.p || slot >= 0))
      kind(a.k, a.k_out, a.k_weight, a.Hkv, max(from - iq, 0), min(to - iq, ik), c.k);
    if (slot >= 0 && to > iq + ik) {
      const uint16_t *src = a.v.p + t * a.v.st_t + sub * 8;
      const int i1 = to - iq - ik;
      for (int i = max(from - iq - ik, 0); i < i1; i += kRows) {
        uint4 x[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          const int h = (i + u) * kHeads + head0;
          if (i + u < i1 && h < a.Hkv) x[u] = ld_stream_v4(src + h * a.v.st_h);
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          const int h = (i + u) * kHeads + head0;
          if (i + u < i1 && h < a.Hkv) *reinterpret_cast<uint4 *>(c.v + slot + h * c.st_head + sub * 8) = x[u];
        }
      }
    }
  }
}

template <bool kHalf, int D>
cudaError_t launch(bool pairs, dim3 grid, const Paged &c, const RopeArgs &a, cudaStream_t stream) {
  return pairs ? launch_pdl(qk_norm_rope_kernel<kHalf, D, true>, grid, dim3(kThreads), 0, stream, c, a)
               : launch_pdl(qk_norm_rope_kernel<kHalf, D, false>, grid, dim3(kThreads), 0, stream, c, a);
}

}  // namespace

int launch_qk_norm_rope(bool half, int T, int Hq, int Hkv, int D, const void *q, int64_t q_st_t, int64_t q_st_h,
                        const void *k, int64_t k_st_t, int64_t k_st_h, const void *v, int64_t v_st_t, int64_t v_st_h,
                        const void *q_weight, const void *k_weight, float eps, const int32_t *pos,
                        const double *inv_freq, int rot, bool pairs, float factor, void *q_out, int64_t q_out_st_t,
                        int64_t q_out_st_h, void *k_out, int64_t k_out_st_t, int64_t k_out_st_h, const Paged &c,
                        const int64_t *slots, int32_t *status, cudaStream_t stream) {
  auto arr = [](const void *p, int64_t st_t, int64_t st_h) {
    return Strided{const_cast<uint16_t *>(static_cast<const uint16_t *>(p)), st_t, st_h};
  };
  RopeArgs a;
  a.q = arr(q, q_st_t, q_st_h);
  a.k = arr(k, k_st_t, k_st_h);
  a.v = arr(v, v_st_t, v_st_h);
  a.q_out = arr(q_out, q_out_st_t, q_out_st_h);
  a.k_out = arr(k_out, k_out_st_t, k_out_st_h);
  a.q_weight = static_cast<const uint16_t *>(q_weight);
  a.k_weight = static_cast<const uint16_t *>(k_weight);
  a.eps = eps;
  a.factor = factor;
  a.pos = pos;
  a.inv_freq = inv_freq;
  a.slots = slots;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.rot = rot;
  a.status = status;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return BASTION_ERR_LAUNCH;
  const int per_warp = 256 / D, iq = (Hq + per_warp - 1) / per_warp, ik = (Hkv + per_warp - 1) / per_warp;
  const int iters = iq + ik + (c.k ? ik : 0);
  a.per = iters;
  while (a.per > 1 && (int64_t)T * ((iters + a.per - 1) / a.per) < 16 * sms) a.per = (a.per + 1) / 2;
  a.chunks = (iters + a.per - 1) / a.per;
  const int64_t want = ((int64_t)T * a.chunks + 7) / 8, most = 8 * (int64_t)sms;
  const dim3 grid((unsigned)(want < most ? want : most));
  const cudaError_t e = half ? (D == 128 ? launch<true, 128>(pairs, grid, c, a, stream) : launch<true, 64>(pairs, grid, c, a, stream))
                             : (D == 128 ? launch<false, 128>(pairs, grid, c, a, stream) : launch<false, 64>(pairs, grid, c, a, stream));
  return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? BASTION_OK : BASTION_ERR_LAUNCH;
}

}  // namespace bastion
