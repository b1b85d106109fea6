// What the attention kernels over the paged cache share: descriptors and issue of
// tcgen05 products, TMA copies of pages, bounded waits, weights as two 16-bit terms.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged.cuh"

namespace bastion {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ uint64_t desc(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint32_t swizzle) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1 << 46;        // descriptor version
  d |= (uint64_t)swizzle << 61;  // 2: 128 bytes, 0: none
  return d;
}

// kind::f16: fp32 accumulators, A and B of one 16-bit type, M = 128, N = n.
template <bool kHalf>
__device__ __forceinline__ constexpr uint32_t idesc(bool a_mn, bool b_mn, int n) {
  return (1u << 4) | (kHalf ? 0u : (1u << 7) | (1u << 10)) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// The instructions that one thread issues are predicated on `one` rather than
// branched around: the issuing warps stay converged, so that descriptors and
// addresses live in uniform registers (a tile's 12 products took 2,100 cycles
// to issue from a branch of one lane).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t x;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(x));
  return x;
}

__device__ __forceinline__ void mma(uint32_t one, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t id,
                                    uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(id), "r"(accum), "r"(one));
}

__device__ __forceinline__ void mma_commit(uint32_t one, uint64_t *bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)),
      "r"(one)
      : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tma_load_4d(uint32_t one, uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2,
                                            int c3, uint32_t bar, uint64_t policy) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %7, 0;\n"
      " @q cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, "
      "{%2, %3, %4, %5}], [%6], %8;\n}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar), "r"(one), "l"(policy)
      : "memory");
}

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Bounded wait that also honours the CTA's abort flag.  The loop is kept out of
// line: the roles' loops compete for the instruction cache.
static __device__ __noinline__ bool wait_slow(uint64_t *bar, uint32_t parity, volatile int *abort, int32_t *status) {
  const uint64_t t0 = global_ns();
  uint32_t spins = 0;
  while (!mbar_try_wait(bar, parity)) {
    if ((++spins & 63u) == 0u) {
      if (*abort) return false;
      if (global_ns() - t0 > 1000000000ull) {
        *abort = 1;
        atomicOr(status, BASTION_STATUS_TIMEOUT);
        return false;
      }
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, volatile int *abort, int32_t *status) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort, status);
}

// p as two 16-bit terms: hi = round(p), lo = round(p - hi), two heads a word.
template <bool kHalf>
__device__ __forceinline__ void split2(float p0, float p1, uint32_t &hi, uint32_t &lo) {
  if (kHalf) {
    const __half2 h = __floats2half2_rn(p0, p1);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(p0 - f.x, p1 - f.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
  } else {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(p1), "f"(p0));
    const float l0 = p0 - bf16lo(hi), l1 = p1 - bf16hi(hi);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(l1), "f"(l0));
  }
}

template <bool kHalf>
__device__ __forceinline__ uint16_t to16(float x) {
  return kHalf ? __half_as_ushort(__float2half_rn(x)) : __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// The driver's tensor-map encoder, looked up once (a function-local static:
// its initialisation is thread-safe, so concurrent first calls are too).
inline PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
  }();
  return fn;
}

// A pool as (D, slot, head, page), or (D, head, slot, page) where the heads lie
// closer together; a box is one page of one head, 64 elements wide.
inline bool make_map(CUtensorMap *m, const uint16_t *base, const Paged &c, bool swap, bool half) {
  auto enc = get_encode();
  if (!enc) return false;
  const cuuint64_t slots = (cuuint64_t)c.page, heads = (cuuint64_t)c.Hkv;
  cuuint64_t dims[4] = {(cuuint64_t)c.D, swap ? heads : slots, swap ? slots : heads, (cuuint64_t)c.n_pages};
  const cuuint64_t ss = (cuuint64_t)c.st_slot * 2, sh = (cuuint64_t)c.st_head * 2;
  cuuint64_t strides[3] = {swap ? sh : ss, swap ? ss : sh, (cuuint64_t)c.st_page * 2};
  cuuint32_t box[4] = {64, swap ? 1u : (cuuint32_t)c.page, swap ? (cuuint32_t)c.page : 1u, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
             const_cast<uint16_t *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace bastion
