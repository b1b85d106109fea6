// Attention of one new token per request over the paged cache.
//
//   s_j = scale q.k_j, out = sum_j exp(s_j - lse) v_j, lse = log sum_j exp(s_j)
//
// Bound by HBM: a token's key and value are read once for the G <= 16 query
// heads of their KV head (2 G flops a byte).  What the design serves is
// an uninterrupted stream of tiles from HBM to every SM:
//
//  * one persistent CTA per SM.  The batch is a list of 128-key tiles, request
//    by request, KV head by KV head (a unit), and every CTA takes an equal
//    contiguous share of it, whatever the lengths; a share is a few segments,
//    each a run of tiles of one unit.  A unit that several CTAs share is joined
//    by the last of them to finish, over the parts in tile order, so that the
//    result does not depend on which one that is;
//  * warp 0 streams key tiles and warp 1 value tiles through rings in shared
//    memory with TMA, one box per page and 64-element column block (128-byte
//    swizzle), across segment boundaries;
//  * the products keep the cache's tiles as the M = 128 operand, so that G
//    heads cost N = 16 columns instead of 128 rows: S^T = K Q^T (M: keys) and
//    O^T += V^T P^T (M: elements of the head; V is read transposed by the
//    descriptor).  Keys and values never pass through registers;
//  * warps 4-7 take the softmax: thread = key, G scores each from TMEM.  The
//    heads' reference maxima are common to the 128 threads; a tile whose scores
//    stay below reference + 2^8 (one barrier vote) goes ahead without a
//    maximum, otherwise the references move and O is rescaled.  Sums stay in
//    the threads until the segment ends;
//  * P is written as a high and a low 16-bit term in separate columns (N = 2 x 8
//    or 2 x 16), which the tensor cores multiply alike, where one bf16 term would
//    add 2^-9 of noise to the output.  bf16: every weight to 2^-17 of itself.
//    Half precision: its low term ends at 2^-24, so that the weights are scaled
//    by 2^6 and are off by at most 2^-31 of the part's largest (and 2^-22 of
//    themselves); those below it are 0 in the product, but not in the sum.
//    P is stored key by key (16 bytes a thread, an MN-major operand without
//    swizzle).
//  * value rows past the sequence's end (a page's unused slots may hold NaN) are
//    zeroed in shared memory; their scores are masked.
//
// With weights, the scores (in base 2) are kept and a second kernel adds
// sum_h exp2(s - lse_h) to each slot's accumulated weight.
//
// Measured, cold caches, 32 query heads on 8 KV heads, D = 128: 64 requests of up to 16,384
// tokens (2.5 GB) 369 us, the copy bandwidth; 8 of 4,096 (134 MB) 29.1 us, 68%; one of
// 131,072 (537 MB) 89 us, 89%; one of 300 (1.2 MB) 7.2 us.  What is left of the small ones is
// latency: a launch (2.2 us), the dependent reads of lengths and page table before the first copy
// (1.5 us), the last tile's chain of products and softmax (1 us) and, where a unit is shared, the
// join (1.4 us).  The accumulated weights add 5 us to 32 requests of 2,065 tokens (53 us) and 12 us to 8 of
// up to 32,768 (153,588 in all, 70 us): the scores, stored once and read back from L2, and the second
// launch, which covers the whole capacity (those 32 requests: 81 us in tables of 32,768 slots).
// With D = 64 the tile's 12 products and the softmax have half the time: 98% all the same (2.6 GB).
//
// Every wait is bounded (~1 s); after one ran out the CTA flags every request of
// which it had tiles left, whose accumulated weights then stay as they were, waits
// for its own copies and products (bounded), frees its TMEM and returns.
#include "paged.cuh"
#include "paged_tc.cuh"
#include "paged_walk.cuh"

namespace bastion {

namespace {

constexpr int kGroup = 24;        // parts joined at a time, at most
constexpr int kPartFloats = 16 * 128 + 32;  // O of up to 16 heads, their references and sums
constexpr int kThreads = 256;
constexpr int kBatch = 4;         // tiles whose table entries are read together
constexpr float kGrow = 8.0f;     // a score may exceed its head's reference by 2^8

struct AttendArgs {
  const uint16_t *q;
  int64_t q_st_b;
  int Hq, G;
  const int32_t *seq_len;
  float scale_log2;
  uint16_t *out;
  float *out32;       // null, or where the outputs go in 32 bits, with lse2: what shared prefixes are joined with
  float *lse;
  const float *acc;
  float *acc_out;
  uint32_t *arrived;  // [2 * kMaxParts + kMaxUnits], zero between calls
  float *parts;       // [2 * kMaxParts, kPartFloats]
  float *lse2;        // [B, Hq] base-2 log of the sum, of the scores in base 2; +inf: given up
  float *scores;      // [B, Hkv, tiles, G, 128], in base 2
  int tiles_cap;
  int swap;           // tensor map dimensions 1 and 2: (head, slot) instead of (slot, head)
  int32_t *status;
};

// --------------------------------------------------------------------------- shared memory

// D elements a head, GP >= G head columns (4, 8 or 16).  The value ring comes first:
// with D = 64 the transposed value operand has 64 rows, and the M = 128
// instruction's other 64 rows read the memory one tile further on; those rows
// of O are never used.
template <int D, int GP>
struct Layout {
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kNP = 2 * GP;                              // high and low columns of P
  static constexpr int kN = kNP < 16 ? 16 : kNP;                  // of the instruction: the rest are zeros
  static constexpr uint32_t kTile = kTileKeys * D * 2;
  static constexpr uint32_t kBlock = kTileKeys * 128;             // 64-element column block of a tile
  static constexpr uint32_t kQ = (D / 64) * 16 * 128;
  static constexpr uint32_t kP = (kN / 8) * kTileKeys * 16;
  static constexpr uint32_t kOffV = 0;
  static constexpr uint32_t kOffK = kStages * kTile;
  static constexpr uint32_t kOffQ = 2 * kStages * kTile;
  static constexpr uint32_t kOffP = kOffQ + 2 * kQ;
  static constexpr uint32_t kOffList = kOffP + 2 * kP;
  static constexpr uint32_t kOffMisc = kOffList + kMaxRequests * 8;
};

struct Misc {
  uint64_t k_full[6], k_empty[6], v_full[6], v_empty[6];
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2], q_full[2], q_empty[2], mma_done;
  uint2 warp_sum[8];
  float xm[4][16], xl[4][16];
  int li0, off0, f0, f1;
  uint32_t last;
  uint32_t tmem;
  int abort;
};

template <int D, int GP>
constexpr uint32_t smem_bytes() {
  constexpr uint32_t n = Layout<D, GP>::kOffMisc + (uint32_t)sizeof(Misc) + 1024;  // + alignment slack
  static_assert(n <= 227 * 1024, "shared memory of one CTA");
  return n;
}

// --------------------------------------------------------------------------- tensor memory

// N consecutive TMEM columns of the thread's lane, as one load or store per 8.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[N]) {
  uint32_t x[N];
  if (N == 4)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(taddr));
#pragma unroll
  for (int i = 0; i + 8 <= N; i += 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3]), "=r"(x[i + 4]), "=r"(x[i + 5]),
                   "=r"(x[i + 6]), "=r"(x[i + 7])
                 : "r"(taddr + (uint32_t)i));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __uint_as_float(x[i]);
}

template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 8)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr + (uint32_t)i),
                 "r"(__float_as_uint(v[i])), "r"(__float_as_uint(v[i + 1])), "r"(__float_as_uint(v[i + 2])),
                 "r"(__float_as_uint(v[i + 3])), "r"(__float_as_uint(v[i + 4])), "r"(__float_as_uint(v[i + 5])),
                 "r"(__float_as_uint(v[i + 6])), "r"(__float_as_uint(v[i + 7]))
                 : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Whether any of the 128 softmax threads says so; a barrier among them.
__device__ __forceinline__ bool vote128(bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(x ? 1u : 0u)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void bar128() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// --------------------------------------------------------------------------- the shares

__device__ __forceinline__ int clamped_len(const Paged &c, const AttendArgs &a, int r) {
  return min(max(a.seq_len[r], 0), c.cap);
}

// Value h of a small array by a thread's own index, without local memory.
template <int N>
__device__ __forceinline__ float pick(const float (&x)[N], int h) {
  float y = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) y = h == i ? x[i] : y;
  return y;
}

// Sums or maxima of N values over the warp; lane l gets that of value l / (32 / N).
template <int N, bool kMax>
__device__ __forceinline__ float warp_all(const float (&x)[N], int lane) {
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = x[i];
  int o = 16;
#pragma unroll
  for (int m = N / 2; m > 0; m >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < m; ++i) {
      const float give = up ? v[i] : v[i + m], keep = up ? v[i + m] : v[i];
      const float got = __shfl_xor_sync(kFull, give, o);
      v[i] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
#pragma unroll
  for (; o > 0; o >>= 1) {
    const float got = __shfl_xor_sync(kFull, v[0], o);
    v[0] = kMax ? fmaxf(v[0], got) : v[0] + got;
  }
  return v[0];
}

// Adds 1 to a counter: what the thread (and, before a barrier, its CTA) wrote is
// visible to whoever sees the sum, and what others wrote before adding to it is to the thread.
__device__ __forceinline__ uint32_t arrive_gpu(uint32_t *p) {
  uint32_t old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(p) : "memory");
  return old;
}

// Flags the requests of what is left of a share, and marks their rows for the
// weights pass.  Out of line, like wait_slow.
__device__ __noinline__ void leave(Walk<true> w, int heads, int32_t *status, float *lse2, int G, int kt) {
  give_up(w, heads, [&](int r, int g) {
    if (kt == 0) atomicOr(&status[r], BASTION_STATUS_TIMEOUT);
    if (lse2 && kt < G) lse2[((size_t)r * heads + g) * G + kt] = INFINITY;
  });
}

template <bool kHalf, int D, int GP>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, Paged c,
                           AttendArgs a) {
  using Lay = Layout<D, GP>;
  constexpr int kStages = Lay::kStages, kNP = Lay::kNP, kN = Lay::kN, kBlocks = D / 64;
  constexpr float kBias = kHalf ? 6.0f : 0.0f;  // weights are scaled by 2^kBias
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem =
      reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Misc &ms = *reinterpret_cast<Misc *>(smem + Lay::kOffMisc);
  int2 *list = reinterpret_cast<int2 *>(smem + Lay::kOffList);
  volatile int *abort = &ms.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_v)) : "memory");
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&ms.k_full[s], 1);
      mbar_init(&ms.k_empty[s], 1);
      mbar_init(&ms.v_full[s], 1);
      mbar_init(&ms.v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ms.s_full[s], 1);
      mbar_init(&ms.s_free[s], 4);
      mbar_init(&ms.p_full[s], 4);
      mbar_init(&ms.pv_done[s], 1);
      mbar_init(&ms.q_full[s], 1);
      mbar_init(&ms.q_empty[s], 1);
    }
    mbar_init(&ms.mma_done, 1);
    ms.abort = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 64;" ::"r"(smem_u32(&ms.tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // the wait first: the prefix launch of paged_prefix.cu, which may follow, counts on it
  griddep_wait();
  griddep_launch_dependents();

  // ------------------------------------------------------------ this CTA's share
  // prefix sums over the requests of (requests with tiles, tiles); a thread has consecutive requests
  const int chunk = (c.B + kThreads - 1) / kThreads, r0 = tid * chunk, r1 = min(c.B, r0 + chunk);
  int cnt = 0, til = 0;
#pragma unroll 1
  for (int b = r0; b < r1; ++b) {
    const int n = a.seq_len[b];
    if ((n < 0 || n > c.cap) && blockIdx.x == 0) atomicOr(&a.status[b], BASTION_STATUS_KV_OVERFLOW);
    const int m = min(max(n, 0), c.cap);
    cnt += m > 0;
    til += (m + kTileKeys - 1) / kTileKeys;
  }
  int cnt_i = cnt, til_i = til;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFull, cnt_i, o), y = __shfl_up_sync(kFull, til_i, o);
    if (lane >= o) {
      cnt_i += x;
      til_i += y;
    }
  }
  if (lane == 31) ms.warp_sum[warp] = make_uint2((unsigned)cnt_i, (unsigned)til_i);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms.tmem;
  int rank = cnt_i - cnt, at = til_i - til, total = 0;
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    const uint2 y = ms.warp_sum[x];
    if (x < warp) {
      rank += (int)y.x;
      at += (int)y.y;
    }
    total += (int)y.y;
  }
  total *= c.Hkv;
  at *= c.Hkv;
  Shares sh;
  sh.n = min((int)gridDim.x, total);
  sh.quot = sh.n > 0 ? total / sh.n : 0;
  sh.big = total - sh.quot * sh.n;
  const int b0 = sh.begin(blockIdx.x), b1 = sh.begin(blockIdx.x + 1);
  const bool busy = (int)blockIdx.x < sh.n;
  if (tid == 0 && busy && (int)blockIdx.x == sh.n - 1) ms.f1 = total;
  if (busy) {
#pragma unroll 1
    for (int b = r0; b < r1; ++b) {
      const int n = clamped_len(c, a, b), t = (n + kTileKeys - 1) / kTileKeys, end = at + t * c.Hkv;
      if (n == 0) continue;
      list[rank] = make_int2(b, n);
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {  // the share's begin and end
        const int f = k ? b1 : b0;
        if (f < at || f >= end) continue;
        // (f - at) % t: the quotient is below Hkv <= 2^16, so that its estimate is off by one at most
        int off = f - at - (int)(__fdividef((float)(f - at), (float)t)) * t;
        off += off < 0 ? t : off >= t ? -t : 0;
        const int to = Shares::moved(f, off, t);
        if (k) {
          ms.f1 = to;
        } else {
          ms.f0 = to;
          ms.li0 = to == end ? rank + 1 : rank;  // the next request's begin
          ms.off0 = to == end ? 0 : to - at;
        }
      }
      ++rank;
      at = end;
    }
  }
  __syncthreads();
  const int f0 = ms.f0;
  Walk<true> w;
  w.start(list, ms.li0, __shfl_sync(kFull, ms.off0, 0), __shfl_sync(kFull, busy ? ms.f1 - f0 : 0, 0));

  if (warp < 2) {
    // ------------------------------------------------------------ TMA: warp 0 keys, warp 1 values
    const CUtensorMap *map = warp == 0 ? &tm_k : &tm_v;
    uint64_t *full = warp == 0 ? ms.k_full : ms.v_full, *empty = warp == 0 ? ms.k_empty : ms.v_empty;
    unsigned char *ring = smem + (warp == 0 ? Lay::kOffK : Lay::kOffV);
    const uint32_t one = elect_one();
    // Table entries are read in batches of kBatch tiles, a batch ahead of their use, so that the
    // reads' latency never holds up the copies.  Lane: page lane % ppt of the batch's tile lane / ppt.
    const int psh = 7 - c.shift, ppt = 1 << psh, batch = min(kBatch, 32 >> psh);
    Walk<false> lw;  // this lane's tile
    lw.start(list, ms.li0, ms.off0, w.left);
    int lead = lane >> psh;
    auto next_entry = [&]() {  // walks on by `lead` tiles and reads there
#pragma unroll 1
      for (int x = 0; x < lead && lw.left > 0; ++x) lw.step(c.Hkv);
      lead = batch;
      const int pg = (lw.t << psh) + (lane & (ppt - 1));
      const bool on = (lane >> psh) < batch && lw.left > 0 && (pg << c.shift) < lw.n;
      const int e = on ? c.table[(size_t)lw.r * c.max_pages + pg] : 0;
      __syncwarp();
      return e;
    };
    int entry = 0, entry_n = next_entry(), in_batch = batch;
    const uint64_t policy = l2_evict_first_policy();  // read once: not at the scores' and parts' expense
    const uint32_t ring32 = smem_u32(ring), full32 = smem_u32(full);
    int slot = 0, phase = 0, issued = 0;
#pragma unroll 1
    for (; w.left > 0; w.step(c.Hkv)) {
      if (in_batch == batch) {
        entry = entry_n;
        if (entry < 0 || entry >= c.n_pages) {  // no page of the pool: page 0 stands in
          atomicOr(&a.status[lw.r], BASTION_STATUS_BAD_PAGE);
          entry = 0;
        }
        entry_n = next_entry();
        in_batch = 0;
      }
      if (!__all_sync(kFull, wait_bar(&empty[slot], phase ^ 1, abort, &a.status[w.r]))) break;
      const int np = (min(kTileKeys, w.n - w.t * kTileKeys) + c.page - 1) >> c.shift;
      if (one) mbar_arrive_expect_tx(&full[slot], (uint32_t)(np << c.shift) * (uint32_t)(D * 2));
      uint32_t dst = ring32 + (uint32_t)slot * Lay::kTile;
      const int c1 = a.swap ? w.g : 0, c2 = a.swap ? 0 : w.g;
#pragma unroll 4
      for (int p = 0; p < np; ++p) {
        const int id = __shfl_sync(kFull, entry, (in_batch << psh) + p);
#pragma unroll
        for (int blk = 0; blk < kBlocks; ++blk)
          tma_load_4d(one, dst + (uint32_t)blk * Lay::kBlock, map, blk * 64, c1, c2, id, full32 + 8u * (uint32_t)slot,
                      policy);
        dst += (uint32_t)(128 << c.shift);
      }
      if (++slot == kStages) {
        slot = 0;
        phase ^= 1;
      }
      ++issued;
      ++in_batch;
    }
    // our last copies have landed (bounded) before the CTA may exit
    if (lane == 0) {
      for (int u = issued > kStages ? issued - kStages : 0; u < issued; ++u)
        mbar_wait_bounded(&full[u % kStages], (uint32_t)(u / kStages) & 1u);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ products
    constexpr uint32_t id_s = idesc<kHalf>(false, false, 16), id_o = idesc<kHalf>(true, true, kN);
    const uint32_t one = elect_one();
    // descriptors of the rings' and buffers' first bytes; addresses are added in units of 16 bytes
    const uint64_t dk = desc(smem_u32(smem + Lay::kOffK), 16, 1024, 2), dq = desc(smem_u32(smem + Lay::kOffQ), 16, 1024, 2);
    const uint64_t dv = desc(smem_u32(smem + Lay::kOffV), Lay::kBlock, 1024, 2);
    const uint64_t dp = desc(smem_u32(smem + Lay::kOffP), 128, kTileKeys * 16, 0);
    const uint32_t o_col = tmem + 32u;
    bool ok = true, prev_first = false;
    int i = 0, seg = 0, ks = 0, kph = 0, vs = 0, vph = 0, prev_r = 0;
    // O += V^T P^T over the 128 keys of tile j
    auto pv = [&](int j, bool fresh, int r) {
      const int s = j & 1;
      if (!__all_sync(kFull, wait_bar(&ms.p_full[s], (uint32_t)(j >> 1) & 1u, abort, &a.status[r]) &&
                                 wait_bar(&ms.v_full[vs], (uint32_t)vph, abort, &a.status[r])))
        return false;
      tc_fence_after();
      const uint64_t dv_t = dv + (uint32_t)vs * (Lay::kTile >> 4), dp_t = dp + (uint32_t)s * (Lay::kP >> 4);
#pragma unroll
      for (int x = 0; x < kTileKeys / 16; ++x)
        mma(one, o_col, dv_t + 128u * x, dp_t + 16u * x, id_o, x > 0 ? 1u : fresh ? 0u : 1u);
      mma_commit(one, &ms.pv_done[s]);
      mma_commit(one, &ms.v_empty[vs]);
      if (++vs == kStages) {
        vs = 0;
        vph ^= 1;
      }
      return true;
    };
    for (; ok && w.left > 0; w.step(c.Hkv), ++i) {
      ok = __all_sync(kFull, (!w.first || wait_bar(&ms.q_full[seg & 1], (uint32_t)(seg >> 1) & 1u, abort, &a.status[w.r])) &&
                                 wait_bar(&ms.s_free[i & 1], ((uint32_t)(i >> 1) & 1u) ^ 1u, abort, &a.status[w.r]) &&
                                 wait_bar(&ms.k_full[ks], (uint32_t)kph, abort, &a.status[w.r]));
      if (!ok) break;
      tc_fence_after();
      const uint64_t dk_t = dk + (uint32_t)ks * (Lay::kTile >> 4), dq_t = dq + (uint32_t)(seg & 1) * (Lay::kQ >> 4);
#pragma unroll
      for (int x = 0; x < D / 16; ++x)
        mma(one, tmem + 16u * (uint32_t)(i & 1), dk_t + (x >> 2) * (Lay::kBlock >> 4) + (x & 3) * 2u,
            dq_t + (x >> 2) * 128u + (x & 3) * 2u, id_s, x > 0);
      mma_commit(one, &ms.s_full[i & 1]);
      mma_commit(one, &ms.k_empty[ks]);
      if (++ks == kStages) {
        ks = 0;
        kph ^= 1;
      }
      if (w.last()) {
        mma_commit(one, &ms.q_empty[seg & 1]);
        ++seg;
      }
      if (i > 0) ok = pv(i - 1, prev_first, prev_r);
      prev_first = w.first;
      prev_r = w.r;
    }
    if (ok && i > 0) pv(i - 1, prev_first, prev_r);
    // every product issued has completed (bounded) before the CTA may free its TMEM
    mma_commit(one, &ms.mma_done);
    mbar_wait_bounded(&ms.mma_done, 0);
  } else if (warp == 3) {
    // ------------------------------------------------------------ queries of each segment; empty requests
    int seg = 0;
    for (; w.left > 0; w.step(c.Hkv)) {
      if (!w.first) continue;
      const uint16_t *q = a.q + w.r * a.q_st_b + (int64_t)w.g * a.G * D;
      uint4 v[D / 16];  // 16 rows of D / 8 vectors, 32 lanes
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        const int id = lane + 32 * x, h = id / (D / 8), k = id % (D / 8);
        v[x] = h < a.G ? *reinterpret_cast<const uint4 *>(q + h * D + k * 8) : make_uint4(0, 0, 0, 0);
      }
      if (!__all_sync(kFull, wait_bar(&ms.q_empty[seg & 1], ((uint32_t)(seg >> 1) & 1u) ^ 1u, abort, &a.status[w.r])))
        break;
      unsigned char *dst = smem + Lay::kOffQ + (seg & 1) * Lay::kQ;
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        const int id = lane + 32 * x, h = id / (D / 8), k = id % (D / 8);
        *reinterpret_cast<uint4 *>(dst + (k >> 3) * 2048 + h * 128 + (((k & 7) ^ (h & 7)) << 4)) = v[x];
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.q_full[seg & 1]);
      ++seg;
    }
    for (int b = blockIdx.x; b < c.B; b += gridDim.x) {
      if (clamped_len(c, a, b) > 0) continue;
      if (a.out32) {
        for (int h = lane; h < a.Hq; h += 32) a.lse2[(size_t)b * a.Hq + h] = -INFINITY;
        continue;
      }
      uint4 *dst = reinterpret_cast<uint4 *>(a.out + (size_t)b * a.Hq * D);
      for (int x = lane; x < a.Hq * D / 8; x += 32) dst[x] = make_uint4(0, 0, 0, 0);
      for (int h = lane; h < a.Hq; h += 32)
        if (a.lse) a.lse[(size_t)b * a.Hq + h] = -INFINITY;
    }
  } else {
    // ------------------------------------------------------------ softmax and joins
    const int quad = warp - 4, kt = quad * 32 + lane;  // key of the tile = TMEM lane = element of O
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    float ref[GP], l[GP];
    if (kN > kNP) {  // the columns of P that no head uses
#pragma unroll
      for (int x = 0; x < 2; ++x)
        *reinterpret_cast<uint4 *>(smem + Lay::kOffP + x * Lay::kP + kTileKeys * 16 + kt * 16) = make_uint4(0, 0, 0, 0);
    }
    bool ok = true;
    int i = 0, t_first = 0, vs = 0, vph = 0;
    for (; w.left > 0; w.step(c.Hkv), ++i) {
      const int s = i & 1;
      int32_t *st = &a.status[w.r];
      if (w.first) {
        t_first = w.t;
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          ref[h] = -INFINITY;
          l[h] = 0.f;
        }
      }
      ok = __all_sync(kFull, ok && wait_bar(&ms.s_full[s], (uint32_t)(i >> 1) & 1u, abort, st));
      float v[GP];
      bool over = false;
      const bool live = w.t * kTileKeys + kt < w.n;
      if (ok) {
        tc_fence_after();
        tmem_ld<GP>(lane_base + 16u * (uint32_t)s, v);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.s_free[s]);
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          v[h] = live ? v[h] * a.scale_log2 : -INFINITY;
          over |= v[h] > ref[h] + (kBias + kGrow);
        }
        if (a.scores && live) {
          float *dst = a.scores + (((size_t)w.r * c.Hkv + w.g) * a.tiles_cap + w.t) * a.G * kTileKeys + kt;
#pragma unroll
          for (int h = 0; h < GP; ++h)
            if (h < a.G) dst[h * kTileKeys] = v[h];
        }
      }
      // a segment's first tile always sets the references
      if (w.first || vote128(over || !ok)) {
        // the tile's maximum of each head; the references that it exceeds move to it
        const float top_h = warp_all<GP, true>(v, lane);
        if ((lane & (32 / GP - 1)) == 0) ms.xm[quad][lane / (32 / GP)] = top_h;
        if (vote128(!ok)) {
          ok = false;
          break;  // all 128 threads
        }
        float alpha[GP];
        bool moved = false;
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          const float m = fmaxf(fmaxf(ms.xm[0][h], ms.xm[1][h]), fmaxf(ms.xm[2][h], ms.xm[3][h]));
          const bool grow = m > ref[h] + (kBias + kGrow);
          const float to = grow ? m - kBias : ref[h];
          alpha[h] = grow ? ex2f(ref[h] - to) : 1.0f;  // 0 for a head that had no finite score: its l and O are 0
          moved |= grow && !w.first;
          ref[h] = to;
          l[h] *= alpha[h];
        }
        if (moved) {  // the same for all 128 threads; not in a segment's first tile
          ok = __all_sync(kFull, wait_bar(&ms.pv_done[(i - 1) & 1], (uint32_t)((i - 1) >> 1) & 1u, abort, st));
          if (ok) {
            tc_fence_after();
            float o[kNP];
            tmem_ld<kNP>(lane_base + 32u, o);
#pragma unroll
            for (int x = 0; x < kNP; ++x) o[x] *= alpha[x & (GP - 1)];
            tmem_st<kNP>(lane_base + 32u, o);
          }
        }
      }
      // weights; P buffer s is free once tile i - 2 is multiplied
      uint32_t hi[GP / 2], lo[GP / 2];
#pragma unroll
      for (int h = 0; h < GP; h += 2) {
        const float p0 = ex2f(v[h] - (ref[h] == -INFINITY ? 0.f : ref[h]));
        const float p1 = ex2f(v[h + 1] - (ref[h + 1] == -INFINITY ? 0.f : ref[h + 1]));
        l[h] += p0;
        l[h + 1] += p1;
        split2<kHalf>(p0, p1, hi[h / 2], lo[h / 2]);
      }
      if (i >= 2) ok = __all_sync(kFull, ok && wait_bar(&ms.pv_done[s], (uint32_t)((i - 2) >> 1) & 1u, abort, st));
      if (ok) {
        unsigned char *pb = smem + Lay::kOffP + s * Lay::kP + kt * 16;
        if (GP == 4) *reinterpret_cast<uint4 *>(pb) = make_uint4(hi[0], hi[1], lo[0], lo[1]);
#pragma unroll
        for (int x = 0; x < GP / 8; ++x) {
          *reinterpret_cast<uint4 *>(pb + x * (kTileKeys * 16)) =
              make_uint4(hi[4 * x], hi[4 * x + 1], hi[4 * x + 2], hi[4 * x + 3]);
          *reinterpret_cast<uint4 *>(pb + (GP / 8 + x) * (kTileKeys * 16)) =
              make_uint4(lo[4 * x], lo[4 * x + 1], lo[4 * x + 2], lo[4 * x + 3]);
        }
      }
      if (w.n - w.t * kTileKeys < kTileKeys) {  // the rows past the end: zeros, whatever the page holds there
        ok = __all_sync(kFull, ok && wait_bar(&ms.v_full[vs], (uint32_t)vph, abort, st));
        if (ok) {  // consecutive threads on consecutive 16 bytes: a row a thread would hit one bank 32 times over
          unsigned char *tile = smem + Lay::kOffV + vs * Lay::kTile;
#pragma unroll 1
          for (int x = (w.n - w.t * kTileKeys) * 128 + kt * 16; x < kTileKeys * 128; x += 128 * 16)
#pragma unroll
            for (int blk = 0; blk < kBlocks; ++blk)
              *reinterpret_cast<uint4 *>(tile + blk * Lay::kBlock + x) = make_uint4(0, 0, 0, 0);
        }
      }
      if (++vs == kStages) {
        vs = 0;
        vph ^= 1;
      }
      if (ok) {
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.p_full[s]);
      }
      if (!w.last()) continue;

      // ---------------------------------------------------------- the segment's end
      const bool whole = t_first == 0 && w.t == w.tiles - 1;
      const int u0 = f0 + i - w.t, u1 = u0 + w.tiles;
      const int c0 = whole ? 0 : sh.first_cta(u0), np = whole ? 1 : sh.last_cta(u1) - c0 + 1;  // its unit's CTAs
      const float part_l = warp_all<GP, false>(l, lane);
      if ((lane & (32 / GP - 1)) == 0) ms.xl[quad][lane / (32 / GP)] = part_l;
      ok = __all_sync(kFull, ok && wait_bar(&ms.pv_done[s], (uint32_t)(i >> 1) & 1u, abort, st));
      if (vote128(!ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float o[GP];
      {
        float both[kNP];
        tmem_ld<kNP>(lane_base + 32u, both);
#pragma unroll
        for (int h = 0; h < GP; ++h) o[h] = both[h] + both[GP + h];
      }
      tc_fence_before();  // the next segment's products overwrite O after this thread's next p_full arrival
#pragma unroll
      for (int h = 0; h < GP; ++h) l[h] = (ms.xl[0][h] + ms.xl[1][h]) + (ms.xl[2][h] + ms.xl[3][h]);
      bool write = whole;
      if (!write) {
        // One of several parts of the unit.  Parts are joined in groups of consecutive
        // CTAs, the groups' results then as parts of their own; each time by whoever arrives
        // last, in the parts' order.  A CTA's first segment has slot 2 * cta, a later one the
        // next; only a unit's first CTA can have begun another unit before.
        auto slot_of = [&](int x) { return x == 0 ? 2 * c0 + 1 : 2 * (c0 + x); };  // of part x
        auto put = [&](int slot) {
          float *part = a.parts + (size_t)slot * kPartFloats;
#pragma unroll
          for (int h = 0; h < GP; ++h)
            if (h < a.G && kt < D) part[h * D + kt] = o[h];
          if (kt < GP) reinterpret_cast<float2 *>(part + 2048)[kt] = make_float2(pick<GP>(ref, kt), pick<GP>(l, kt));
        };
        // up to kGroup parts at once, more in about as many groups as a group has parts (20 parts: 0.9 us
        // less than by 16 and 4; 152 of one unit: 21 us in all, 24 by 48)
        const int size = np <= kGroup ? np : (int)ceilf(sqrtf((float)np));
        const int x = (int)blockIdx.x - c0, groups = (np + size - 1) / size;
        int first = x / size * size, step = 1, count = min(size, np - first), slot = slot_of(x);
        uint32_t *counter = &a.arrived[slot_of(first)];
#pragma unroll 1
        for (;;) {
          put(slot);
          bar128();
          if (kt == 0) {
            const bool is_last = arrive_gpu(counter) == (uint32_t)(count - 1);
            if (is_last) *counter = 0;
            ms.last = is_last;
          }
          bar128();
          if (!ms.last) break;
          // o, l, ref = parts first, first + step, ... joined
          constexpr int kLoads = GP == 16 ? 4 : 32 / GP, kRows = 128 / GP;  // parts whose loads are in flight together
          const int fh = kt & (GP - 1), fy = kt / GP;
          // the parts' references and sums, then their factors; in the P buffers, which no product reads now
          float2(*jml)[GP] = reinterpret_cast<float2(*)[GP]>(smem + Lay::kOffP);
          static_assert(kGroup * GP * 8 <= (kN > kNP ? kTileKeys * 16 : 2 * Lay::kP), "the factors fit the P buffers");
          float in[kLoads][GP];
          auto fetch = [&](int y0) {
#pragma unroll
            for (int y = 0; y < kLoads; ++y) {
              const float *part = a.parts + (size_t)slot_of(first + min(y0 + y, count - 1) * step) * kPartFloats + kt;
#pragma unroll
              for (int h = 0; h < GP; ++h)
                if (h < a.G && kt < D) in[y][h] = __ldcg(part + h * D);
            }
          };
          constexpr int kMl = (kGroup + kRows - 1) / kRows;
          float2 ml[kMl];
#pragma unroll
          for (int k = 0; k < kMl; ++k) {
            const int y = fy + k * kRows;
            ml[k] = y < count ? __ldcg(reinterpret_cast<const float2 *>(
                                           a.parts + (size_t)slot_of(first + y * step) * kPartFloats + 2048) + fh)
                              : make_float2(-INFINITY, 0.f);
          }
          fetch(0);
#pragma unroll
          for (int k = 0; k < kMl; ++k)
            if (fy + k * kRows < kGroup) jml[fy + k * kRows][fh] = ml[k];
          bar128();
          float top = -INFINITY;
#pragma unroll
          for (int y = 0; y < kGroup; ++y) top = fmaxf(top, jml[y][fh].x);
          bar128();
#pragma unroll
          for (int k = 0; k < kMl; ++k) {
            const float f = ml[k].x == -INFINITY ? 0.f : ex2f(ml[k].x - top);
            if (fy + k * kRows < kGroup) jml[fy + k * kRows][fh] = make_float2(f, f * ml[k].y);
          }
          if (fy == 0) ms.xm[0][fh] = top;
          bar128();
#pragma unroll
          for (int h = 0; h < GP; ++h) {
            o[h] = l[h] = 0.f;
            ref[h] = ms.xm[0][h];
          }
          for (int y0 = 0; y0 < count; y0 += kLoads) {
#pragma unroll
            for (int y = 0; y < kLoads; ++y) {
              if (y0 + y >= count) break;
#pragma unroll
              for (int h = 0; h < GP; ++h) {
                const float2 f = jml[y0 + y][h];
                l[h] += f.y;
                if (h < a.G && kt < D) o[h] += f.x * in[y][h];
              }
            }
            if (y0 + kLoads < count) fetch(y0 + kLoads);
          }
          bar128();  // jml and xm are read: the next round or tile may write them
          if (step > 1 || groups == 1) {
            write = true;
            break;
          }
          slot = slot_of(first);  // the group's result takes its first part's place
          first = 0;
          step = size;
          count = groups;
          counter = &a.arrived[2 * kMaxParts + w.r * c.Hkv + w.g];
        }
      }
      if (write) {
        const size_t row = (size_t)w.r * a.Hq + (size_t)w.g * a.G;
#pragma unroll
        for (int h = 0; h < GP; ++h)
          if (h < a.G && kt < D) {
            const float x = l[h] == 0.f ? 0.f : __fdividef(o[h], l[h]);  // no key with a score above -inf: 0
            if (a.out32) a.out32[(row + h) * D + kt] = x;
            else a.out[(row + h) * D + kt] = to16<kHalf>(x);
          }
        if (kt < a.G) {
          const float lh = pick<GP>(l, kt), x = lh == 0.f ? -INFINITY : pick<GP>(ref, kt) + log2f(lh);
          if (a.lse) a.lse[row + kt] = x * kLn2;
          if (a.acc || a.out32) a.lse2[row + kt] = x;
        }
      }
    }
    // a wait ran out, of which only one request has been told
    if (w.left > 0) leave(w, c.Hkv, a.status, a.acc ? a.lse2 : nullptr, a.G, kt);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 64;" ::"r"(tmem));
  }
}

// acc_out = acc + sum over the group's heads of exp2(s - lse2), in head order;
// four keys a thread, 16 bytes of every row that it touches, with the heads'
// loads in flight together and none of them waiting for the length (the score
// rows span the whole capacity).
constexpr int kWeightsThreads = 128;
__global__ void __launch_bounds__(kWeightsThreads) paged_weights_kernel(Paged c, AttendArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int unit = blockIdx.y, r = unit / c.Hkv, g = unit % c.Hkv;
  const int j = 4 * (blockIdx.x * kWeightsThreads + threadIdx.x);
  if (j >= c.cap) return;
  const float *s = a.scores + ((size_t)unit * a.tiles_cap + j / kTileKeys) * a.G * kTileKeys + j % kTileKeys;
  const float *lse2 = a.lse2 + (size_t)r * a.Hq + g * a.G;
  const size_t at = (size_t)unit * c.cap + j;
  const int n = clamped_len(c, a, r);
  const float4 was = *reinterpret_cast<const float4 *>(a.acc + at);
  float w[4] = {};
  for (int h0 = 0; h0 < a.G; h0 += 4) {
    float4 x[4];
    float y[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const bool on = h0 + h < a.G;
      y[h] = on ? lse2[h0 + h] : -INFINITY;
      if (on) x[h] = *reinterpret_cast<const float4 *>(s + (h0 + h) * kTileKeys);
    }
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      if (isinf(y[h])) continue;  // -inf: no such head, or one that sees nothing; +inf: given up
      w[0] += exp2f(x[h].x - y[h]);
      w[1] += exp2f(x[h].y - y[h]);
      w[2] += exp2f(x[h].z - y[h]);
      w[3] += exp2f(x[h].w - y[h]);
    }
  }
  if (j + 4 <= n) {
    *reinterpret_cast<float4 *>(a.acc_out + at) = make_float4(was.x + w[0], was.y + w[1], was.z + w[2], was.w + w[3]);
  } else {
    if (j < n) a.acc_out[at] = was.x + w[0];
    if (j + 1 < n) a.acc_out[at + 1] = was.y + w[1];
    if (j + 2 < n) a.acc_out[at + 2] = was.z + w[2];
  }
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

template <bool kHalf, int D, int GP>
cudaError_t launch_one(const CUtensorMap &mk, const CUtensorMap &mv, int dev, int grid, const Paged &c,
                       const AttendArgs &a, cudaStream_t stream) {
  constexpr uint32_t smem = smem_bytes<D, GP>();
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(paged_attention_kernel<kHalf, D, GP>, (int)smem, dev, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(paged_attention_kernel<kHalf, D, GP>, dim3((unsigned)grid), dim3(kThreads), smem, stream, mk, mv,
                    c, a);
}

template <bool kHalf>
cudaError_t launch_half(const CUtensorMap &mk, const CUtensorMap &mv, int dev, int grid, const Paged &c,
                        const AttendArgs &a, cudaStream_t stream) {
  if (c.D == 128)
    return a.G <= 4   ? launch_one<kHalf, 128, 4>(mk, mv, dev, grid, c, a, stream)
           : a.G <= 8 ? launch_one<kHalf, 128, 8>(mk, mv, dev, grid, c, a, stream)
                      : launch_one<kHalf, 128, 16>(mk, mv, dev, grid, c, a, stream);
  return a.G <= 4   ? launch_one<kHalf, 64, 4>(mk, mv, dev, grid, c, a, stream)
         : a.G <= 8 ? launch_one<kHalf, 64, 8>(mk, mv, dev, grid, c, a, stream)
                    : launch_one<kHalf, 64, 16>(mk, mv, dev, grid, c, a, stream);
}

constexpr size_t kPartsBytes = (size_t)2 * kMaxParts * kPartFloats * sizeof(float);

}  // namespace

size_t paged_attention_workspace_bytes(int B, int Hq, int Hkv, int D, int64_t cap, int weights) {
  (void)Hkv;
  (void)D;
  size_t n = kCounterBytes + up256(kPartsBytes);
  if (weights) {
    n += up256((size_t)B * Hq * sizeof(float));
    n += (size_t)B * Hq * (size_t)((cap + kTileKeys - 1) / kTileKeys) * kTileKeys * sizeof(float);
  }
  return n;
}

namespace {

int launch_any(const Paged &c, bool half, const void *q, int Hq, int64_t q_st_b, const int32_t *seq_len, float scale,
               void *out, float *out32, float *lse2, float *lse, const float *acc, float *acc_out, void *ws,
               int32_t *status, cudaStream_t stream) {
  AttendArgs a;
  a.q = static_cast<const uint16_t *>(q);
  a.q_st_b = q_st_b;
  a.Hq = Hq;
  a.G = Hq / c.Hkv;
  a.seq_len = seq_len;
  a.scale_log2 = scale * kLog2e;
  a.out = static_cast<uint16_t *>(out);
  a.out32 = out32;
  a.lse = lse;
  a.acc = acc;
  a.acc_out = acc_out;
  a.tiles_cap = (c.cap + kTileKeys - 1) / kTileKeys;
  char *at = static_cast<char *>(ws);
  a.arrived = reinterpret_cast<uint32_t *>(at);
  a.parts = reinterpret_cast<float *>(at += kCounterBytes);
  at += up256(kPartsBytes);
  a.lse2 = lse2 ? lse2 : reinterpret_cast<float *>(at);
  a.scores = acc ? reinterpret_cast<float *>(at + up256((size_t)c.B * Hq * 4)) : nullptr;
  a.swap = c.Hkv > 1 && c.st_head < c.st_slot;
  a.status = status;
  CUtensorMap mk, mv;
  if (!make_map(&mk, c.k, c, a.swap, half) || !make_map(&mv, c.v, c, a.swap, half)) return BASTION_ERR_LAUNCH;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return BASTION_ERR_LAUNCH;
  const int64_t most = (int64_t)c.B * c.Hkv * a.tiles_cap;  // tiles, at most
  const int sm_grid = sms < kMaxParts ? sms : kMaxParts, grid = most < sm_grid ? (int)most : sm_grid;
  cudaError_t e = half ? launch_half<true>(mk, mv, dev, grid, c, a, stream) : launch_half<false>(mk, mv, dev, grid, c, a, stream);
  if (e == cudaSuccess && acc)
    e = launch_pdl(paged_weights_kernel,
                   dim3((unsigned)((c.cap + 4 * kWeightsThreads - 1) / (4 * kWeightsThreads)), (unsigned)(c.B * c.Hkv)),
                   dim3(kWeightsThreads), 0, stream, c, a);
  return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? BASTION_OK : BASTION_ERR_LAUNCH;
}

}  // namespace

int launch_paged_attention(const Paged &c, bool half, const void *q, int Hq, int64_t q_st_b, const int32_t *seq_len,
                           float scale, void *out, float *lse, const float *acc, float *acc_out, void *ws,
                           int32_t *status, cudaStream_t stream) {
  return launch_any(c, half, q, Hq, q_st_b, seq_len, scale, out, nullptr, nullptr, lse, acc, acc_out, ws, status, stream);
}

// The outputs in 32 bits (rows of requests without slots are left out) and the
// logarithms of their sums in base 2.
int launch_paged_attention32(const Paged &c, bool half, const void *q, int Hq, int64_t q_st_b, const int32_t *seq_len,
                             float scale, float *out32, float *lse2, void *ws, int32_t *status, cudaStream_t stream) {
  return launch_any(c, half, q, Hq, q_st_b, seq_len, scale, nullptr, out32, lse2, nullptr, nullptr, nullptr, ws, status,
                    stream);
}

}  // namespace bastion
