// Norm and rotation of queries and keys, and their way into the cache.
//
//   y = x / sqrt(mean(x^2) + eps) * w;  (a, b) -> factor (a cos t - b sin t, b cos t + a sin t),  t = pos f_i
//
// Bound by HBM: every element is read once and written once (a token of 32/8
// heads of 128: 24.6 KB both ways), if the arithmetic is kept short.  A token's
// heads are a list of 16-byte vectors a lane, queries, keys, values, four of them in
// flight.  Neighbouring warps take neighbouring tokens, one each, as long as there
// are as many as warps (shares far apart: 5% slower), and equal shares of what is
// left, which cut tokens (whole ones: 10% slower with 4,096).  8 or 16 lanes hold a
// head, so that a head's sum of squares is 3 or 4 shuffles and its partner elements
// are in the lane itself (pairs 2i, 2i + 1) or one shuffle away (i, i + rot / 2).
// The lanes form a token's cosines and sines, a pair or two each, and pass them on through shared memory; norm weights,
// cosines and sines fold into two factors an element,
//   out_e = r (x_e A_e + x_partner B_e),  r = 1 / sqrt(mean + eps),
// so that a head costs 2 products and a sum an element, two elements an
// instruction.
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
constexpr int kRows = 4;    // 16-byte vectors that a lane has in flight
constexpr int kBlocks = 3;  // CTAs an SM

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

// Read once; rows may be written in place, so that this is no read-only load.
__device__ __forceinline__ uint4 ld_once(const uint16_t *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Two floats in one register pair.
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpair2(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
template <bool kHalf>
__device__ __forceinline__ uint64_t unpack2(uint32_t w) {
  const float2 f = unpack<kHalf>(w);
  return pair2(f.x, f.y);
}

template <bool kHalf, int D, bool kPairs>
__global__ void __launch_bounds__(kThreads, kBlocks) qk_norm_rope_kernel(Paged c, RopeArgs a) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;  // lanes of a head, heads of a warp
  __shared__ uint64_t turn[D / 2];                     // of pair i per position, in 2^-64 turns
  __shared__ __align__(16) float s_cos[kThreads / 32][D / 2], s_sin[kThreads / 32][D / 2];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sub = lane % kLanes, head0 = lane / kLanes, half = a.rot / 2;
  for (int i = tid; i < half; i += kThreads) {
    const double x = a.inv_freq[i] * 0.15915494309189533577, f = x - floor(x);  // turns
    turn[i] = (uint64_t)__double2ull_rn(f * 18446744073709551616.0);
  }
  __syncthreads();
  const bool norm = a.q_weight != nullptr, turned = sub * 8 < a.rot;
  // the lane that holds the partners of this one's elements
  const int other = kPairs || !turned ? lane : sub * 8 < half ? lane + half / 8 : lane - half / 8;
  const uint32_t keep = turned ? 0xffffffffu : 0u;  // an infinity that is not turned stays one
  const int iq = (a.Hq + kHeads - 1) / kHeads, ik = (a.Hkv + kHeads - 1) / kHeads, iv = c.k ? ik : 0;
  const int per_token = iq + ik + iv, warps = gridDim.x * (kThreads / 32), me = blockIdx.x * (kThreads / 32) + warp;
  const int even = a.T / warps * warps;
  const int64_t rest = (int64_t)(a.T - even) * per_token, end = rest * (me + 1) / warps;
  int64_t at = rest * me / warps;
  for (int step = me;; step += warps) {
    int t = step, from = 0, to = per_token;
    if (step >= even) {
      if (at >= end) break;
      t = even + (int)(at / per_token);
      from = (int)(at % per_token);
      to = (int)min((int64_t)per_token, from + (end - at));
      at += to - from;
    }
    const int pos = a.pos[t];
    int64_t slot = -1;  // element offset of the token's row in the pools
    if (c.k && to > iq) slot = a.slots[t];
    if (pos < 0) continue;
    if (slot >= 0) {
      const int64_t page = slot >> c.shift;
      if (page < c.n_pages) {
        slot = page * c.st_page + (slot & (c.page - 1)) * c.st_slot;
      } else {
        if (lane == 0) atomicOr(a.status, BASTION_STATUS_BAD_PAGE);
        slot = -1;
      }
    }
    if (from < iq + ik) {
      __syncwarp();  // the warp's last token has been read
#pragma unroll
      for (int k = 0; k < D / 64; ++k) {
        const int i = lane + 32 * k;
        if (i < half) {
          // the signed fraction of a turn, in half turns
          const float y = (float)(int32_t)((turn[i] * (uint64_t)(uint32_t)pos) >> 32) * 0x1p-31f;
          float sv, cv;
          sincospif(y, &sv, &cv);
          s_cos[warp][i] = cv * a.factor;
          s_sin[warp][i] = sv * a.factor;
        }
      }
      __syncwarp();
    }
    // vectors [i0, i1) of the token's queries or keys
    auto kind = [&](const Strided &in, const Strided &out, const uint16_t *weight, int heads, int i0, int i1,
                    uint16_t *pool) {
      uint64_t A[4], B[4];
      if (turned) {
        const int i = kPairs ? sub * 4 : sub * 8 < half ? sub * 8 : sub * 8 - half;
        const float sign = sub * 8 < half ? -1.f : 1.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (kPairs) {
            const float cv = s_cos[warp][i + e], sv = s_sin[warp][i + e];
            A[e] = pair2(cv, cv);
            B[e] = pair2(-sv, sv);
          } else {
            const float2 cv = *reinterpret_cast<const float2 *>(&s_cos[warp][i + 2 * e]);
            const float2 sv = *reinterpret_cast<const float2 *>(&s_sin[warp][i + 2 * e]);
            A[e] = pair2(cv.x, cv.y);
            B[e] = pair2(sign * sv.x, sign * sv.y);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          A[e] = pair2(1.f, 1.f);
          B[e] = 0;
        }
      }
      if (norm) {
        const uint4 w = *reinterpret_cast<const uint4 *>(weight + sub * 8);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          A[e] = mul2(A[e], unpack2<kHalf>(ww[e]));
          B[e] = mul2(B[e], unpack2<kHalf>(kPairs ? __byte_perm(ww[e], 0, 0x1032) : __shfl_sync(kFull, ww[e], other)));
        }
      }
      const int lim = min(i1, (heads - head0 + kHeads - 1) / kHeads);  // this lane's heads
      const int64_t in_st = kHeads * in.st_h, out_st = kHeads * out.st_h, pool_st = kHeads * c.st_head;
      const uint16_t *src = in.p + t * in.st_t + head0 * in.st_h + i0 * in_st + sub * 8;
      uint16_t *dst = out.p ? out.p + t * out.st_t + head0 * out.st_h + i0 * out_st + sub * 8 : nullptr;
      if (pool) pool += slot + head0 * c.st_head + i0 * pool_st + sub * 8;
#pragma unroll 1
      for (int i = i0; i < i1; i += kRows) {
        uint4 x[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          x[u] = make_uint4(0, 0, 0, 0);
          if (i + u < lim) x[u] = ld_once(src);
          src += in_st;
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          if (i + u >= i1) break;
          const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
          uint64_t y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = unpack2<kHalf>(w[e]);
          float r = 1.f;
          if (norm) {
            const float2 s2 = unpair2(fma2(y[3], y[3], fma2(y[2], y[2], fma2(y[1], y[1], mul2(y[0], y[0])))));
            float s = s2.x + s2.y;
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
            r = rsqrtf(s * (1.f / D) + a.eps);
          }
          const uint64_t r2 = pair2(r, r);
          uint32_t z[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t got = kPairs ? __byte_perm(w[e], 0, 0x1032) : __shfl_sync(kFull, w[e], other);
            uint64_t o = fma2(unpack2<kHalf>(got & keep), B[e], mul2(y[e], A[e]));
            if (norm) o = mul2(o, r2);
            const float2 f = unpair2(o);
            z[e] = pack<kHalf>(f.x, f.y);
          }
          if (i + u < lim) {
            const uint4 zz = make_uint4(z[0], z[1], z[2], z[3]);
            if (dst) *reinterpret_cast<uint4 *>(dst) = zz;
            if (pool) *reinterpret_cast<uint4 *>(pool) = zz;
          }
          if (dst) dst += out_st;
          if (pool) pool += pool_st;
        }
      }
    };
    if (from < iq && a.q_out.p) kind(a.q, a.q_out, a.q_weight, a.Hq, from, min(to, iq), nullptr);
    if (to > iq && from < iq + ik && (a.k_out.p || slot >= 0))
      kind(a.k, a.k_out, a.k_weight, a.Hkv, max(from - iq, 0), min(to - iq, ik), slot >= 0 ? c.k : nullptr);
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
  const int64_t want = ((int64_t)T * iters + kThreads / 32 - 1) / (kThreads / 32), most = (int64_t)kBlocks * sms;
  const dim3 grid((unsigned)(want < most ? want : most));
  const cudaError_t e = half ? (D == 128 ? launch<true, 128>(pairs, grid, c, a, stream) : launch<true, 64>(pairs, grid, c, a, stream))
                             : (D == 128 ? launch<false, 128>(pairs, grid, c, a, stream) : launch<false, 64>(pairs, grid, c, a, stream));
  return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? BASTION_OK : BASTION_ERR_LAUNCH;
}

}  // namespace bastion
