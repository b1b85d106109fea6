// Attention of one new token per request over its group's shared prefix and its
// own slots.
//
//   out = (sum_prefix exp(s_j) v_j + sum_own exp(s_j) v_j) / (sum_prefix exp(s_j) + sum_own exp(s_j))
//
// Three launches: the own slots, in 32 bits, by the one-token kernel of
// paged_attention.cu or, where they are few, by paged_prefix_own.cu; the prefixes,
// which begin on the SMs that the own slots leave free; and the join of each row's
// parts (paged_prefix_join.cu).
//
// The prefixes.  A group's n requests are n * G query rows of a KV head, which
// read each key and value once per 256 rows: 512 flops a byte at 256 rows of
// D = 128, about where HBM and the tensor cores take equally long, so that
// neither may wait for the other:
//  * one persistent CTA per SM.  A unit is (group, KV head, up to 256 rows); the
//    batch is a list of 128-key tiles, unit by unit, of which every CTA takes an
//    equal contiguous share (paged_units.cuh);
//  * warp 0 streams keys and warp 2 values through one ring in shared memory,
//    warp 3 the queries of the next M tile of 128 rows, with TMA;
//  * warp 1 issues the products, S = Q K^T from shared memory and O += P V with P
//    in tensor memory: P takes the place of its scores.  Visits (a key tile and
//    an M tile) alternate between two softmax warpgroups, which own 128 columns
//    of S and up to 128 of O each, so that one's softmax runs under the other's
//    products.  A unit of two M tiles gives each warpgroup one; a unit of one
//    gives them alternate key tiles, as two parts;
//  * a thread is a row.  The reference maximum moves, and O is rescaled, only
//    where a score exceeds it by 2^8;
//  * P enters the product as a high and a low 16-bit term, as in
//    paged_attention.cu, twice the instructions for weights to 2^-17.
// Rows of a unit are whole requests (floor(128 / G) of them an M tile), so that a
// box of the query tensor is an M tile, whatever G is.
//
// A part is an M tile's unnormalised rows in 32 bits with their references and sums.
// Units that one CTA finishes have places of their own, others slots of the CTAs;
// warp 3 works out from the shares where the join finds each request's.
//
// Measured in graphs, 32/8 heads, D = 128: 64 requests over 16,384 shared tokens (own slots up
// to 512) 55 us, 256 over 32,768 163 us (131 of them products at 85% of the tensor cores' rate;
// a call from Python 168-173), 4 over 300 11.8 us; 61 in 8 groups, 14/2 heads, D = 64, 22.3 us.
//
// Every wait is bounded (~1 s); after one ran out the CTA flags the requests of
// its remaining tiles, waits for its own copies and products (bounded), frees its
// TMEM and returns.
#include "paged_prefix.cuh"
#include "paged_ring.cuh"
#include "paged_tc.cuh"

namespace bastion {

size_t paged_attention_workspace_bytes(int B, int Hq, int Hkv, int D, int64_t cap, int weights);
int launch_paged_attention32(const Paged &c, bool half, const void *q, int Hq, int64_t q_st_b, const int32_t *seq_len,
                             float scale, float *out32, float *lse2, void *ws, int32_t *status, cudaStream_t stream);

namespace {

constexpr int kThreads = 384;
constexpr int kPer = (kMaxRequests + kThreads - 1) / kThreads;  // groups of a thread in the prologue, at most
constexpr int kBatch = 4;      // tiles whose table entries are read together
constexpr float kGrow = 8.0f;  // a score may exceed its row's reference by 2^8

// The tensor cores cut a sum to 32 bits where others round: O comes out too small by
// half a unit of 2^-24 a product instruction on average, 16 instructions a key tile, and
// half of that as it grows (54 tiles: 1.2e-5 of itself; 164 tiles, 800,000 tokens of 8 heads and
// two M tiles: 8.8e-5, a third of half a step of half precision).  So a chain of products has
// at most kChain visits, after which a warpgroup adds O, rounded, to what is in its part's
// place: 2^-15 at most, whatever the length.  256 requests over 32,768 tokens (54 tiles a
// CTA): 172 us without a limit and with 64, 176 with 32 (error 6e-6), 183 with 16 (2.5e-6).
constexpr int kChain = 64;
// Key tile x of a segment, counted from its chain's first.  A unit of one M tile deals its tiles to both warpgroups.
__device__ __forceinline__ int chain_place(int x, int m_tiles) { return x & (kChain * (3 - m_tiles) - 1); }

// --------------------------------------------------------------------------- shared memory

// The value tiles' operand has D = N rows of MN-major blocks, all inside the stage.
template <int D>
struct Layout {
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kBlocks = D / 64;
  static constexpr uint32_t kBlock = kTileKeys * 128;  // a 64-element column block of 128 rows
  static constexpr uint32_t kTile = kBlocks * kBlock;
  static constexpr uint32_t kOffQ = kStages * kTile;   // two M tiles
  static constexpr uint32_t kOffList = kOffQ + 2 * kTile;
  static constexpr uint32_t kOffMisc = kOffList + kMaxRequests * sizeof(UnitEntry);
};

struct Misc {
  uint64_t full[8], empty[8];
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][2], pv_done[2], mma_done;  // p_full: of a warpgroup's upper, lower keys
  uint64_t begun;  // the first keys have landed; completes once
  int2 warp_sum[kThreads / 32];
  int warp_max[kThreads / 32];
  int li0, f0, f1;
  TilePlace from;
  uint32_t tmem;
  int abort;
};

template <int D>
constexpr uint32_t smem_bytes() {
  constexpr uint32_t n = Layout<D>::kOffMisc + (uint32_t)sizeof(Misc) + 1024;  // + alignment slack
  static_assert(n <= 227 * 1024, "shared memory of one CTA");
  return n;
}

// The ring's barriers as the warp that fills it has them (paged_ring.cuh).
struct RingBars {
  Misc &ms;
  volatile int *abort;
  int32_t *status;
  int lane;
  __device__ __forceinline__ bool wait(uint64_t &bar, uint32_t parity) {
    return __all_sync(kFull, wait_bar(&bar, parity, abort, status));
  }
  __device__ __forceinline__ bool wait_full(int stage, uint32_t parity) { return wait(ms.full[stage], parity); }
  __device__ __forceinline__ bool wait_empty(int stage, uint32_t parity) { return wait(ms.empty[stage], parity); }
  __device__ __forceinline__ bool wait_begun() { return wait(ms.begun, 0); }
  __device__ __forceinline__ void arrive_begun() {
    if (lane == 0) mbar_arrive(&ms.begun);
  }
};

// --------------------------------------------------------------------------- tensor memory

// A in tensor memory (two 16-bit elements a column), B in shared memory.
__device__ __forceinline__ void mma_ta(uint32_t one, uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t id,
                                       uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(id), "r"(accum), "r"(one));
}

// 32 columns of the thread's lane; the registers hold them once wait_ld has returned.
__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// N loaded registers, for the compiler: not to be read before this.
template <int N>
__device__ __forceinline__ void wait_ld(uint32_t (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                 "+r"(r[i + 6]), "+r"(r[i + 7]));
}

__device__ __forceinline__ void st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// Eight columns of O times alpha; the stores are complete after wait_st.
__device__ __forceinline__ void move_o(uint32_t taddr, float alpha) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
  wait_ld(r);
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint64_t l2_evict_normal_policy() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// Two products and sums at once: (x0, x1) * m + a.
__device__ __forceinline__ void fma2(float &x0, float &x1, float m, float a0, float a1) {
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %2};\n mov.b64 z, {%3, %4};\n"
      " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}\n"
      : "+f"(x0), "+f"(x1)
      : "f"(m), "f"(a0), "f"(a1));
}
__device__ __forceinline__ void add2(float &a0, float &a1, float b0, float b1) {
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n add.rn.f32x2 a, a, b;\n"
      " mov.b64 {%0, %1}, a;\n}\n"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}

__device__ __forceinline__ float max3f(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The scores of a tile's keys past its end become -inf.
__device__ __noinline__ void mask_scores(uint32_t s_col, int valid) {
#pragma unroll 1
  for (int k = valid / 32; k < kTileKeys / 32; ++k) {
    uint32_t v[32];
    ld32(s_col + 32u * (uint32_t)k, v);
    wait_ld(v);
#pragma unroll
    for (int y = 0; y < 32; ++y) v[y] = 32 * k + y < valid ? v[y] : 0xff800000u;
    st32(s_col + 32u * (uint32_t)k, v);
  }
  wait_st();
}

// Four running maxima over 32 scores more.
__device__ __forceinline__ void top_of(float (&top)[4], const uint32_t (&v)[32]) {
#pragma unroll
  for (int y = 0; y < 32; y += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k) top[k] = max3f(top[k], __uint_as_float(v[y + 2 * k]), __uint_as_float(v[y + 2 * k + 1]));
}

// split2 of paged_tc.cuh with both differences in one instruction.
template <bool kHalf>
__device__ __forceinline__ void split_pair(float p0, float p1, uint32_t &hi, uint32_t &lo) {
  float h0, h1;
  if (kHalf) {
    const __half2 h = __floats2half2_rn(p0, p1);
    const float2 f = __half22float2(h);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    h0 = f.x;
    h1 = f.y;
  } else {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(p1), "f"(p0));
    h0 = bf16lo(hi);
    h1 = bf16hi(hi);
  }
  fma2(h0, h1, -1.f, p0, p1);  // p - h, exactly
  if (kHalf) {
    const __half2 x = __floats2half2_rn(h0, h1);
    lo = *reinterpret_cast<const uint32_t *>(&x);
  } else {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(h1), "f"(h0));
  }
}

template <bool kHalf, int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_prefix_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, Paged c, PrefixArgs a) {
  using Lay = Layout<D>;
  constexpr int kStages = Lay::kStages, kBlocks = Lay::kBlocks;
  using Tiles = Ring<kStages>;
  constexpr float kBias = kHalf ? 6.0f : 0.0f;  // weights are scaled by 2^kBias
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem =
      reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Misc &ms = *reinterpret_cast<Misc *>(smem + Lay::kOffMisc);
  UnitEntry *list = reinterpret_cast<UnitEntry *>(smem + Lay::kOffList);
  volatile int *abort = &ms.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_q)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_v)) : "memory");
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&ms.full[s], 1);
      mbar_init(&ms.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ms.q_full[s], 1);
      mbar_init(&ms.q_empty[s], 1);
      mbar_init(&ms.s_full[s], 1);
      mbar_init(&ms.p_full[s][0], 4);
      mbar_init(&ms.p_full[s][1], 4);
      mbar_init(&ms.pv_done[s], 1);
    }
    mbar_init(&ms.mma_done, 1);
    mbar_init(&ms.begun, 1);
    ms.abort = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&ms.tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // No wait for the launch before: it attends to the own slots, of which nothing is read here, and let this one begin
  // after everything before it was complete (both kernels that do so wait first).  This launch ends after it (below), and
  // the join waits for this one.  But what earlier launches wrote is certain to be in L2 alone: this SM's L1 may hold
  // lines from before, which a wait here would have dropped.  So the groups and their tables are read past L1 (__ldcg),
  // as the copies are by themselves.
  griddep_launch_dependents();

  // ------------------------------------------------------------ this CTA's share
  // A thread has consecutive groups.  A group begins where the ones before it end, at the earliest.
  const int chunk = (a.n_groups + kThreads - 1) / kThreads, g0 = tid * chunk;
  int from[kPer], n_req[kPer], len[kPer];
  int ends = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int g = g0 + i;
    from[i] = n_req[i] = len[i] = 0;
    if (i >= chunk || g >= a.n_groups) continue;
    const int x = __ldcg(a.start + g), y = __ldcg(a.start + g + 1), n = __ldcg(a.len + g);
    if (x >= 0 && x <= y && y <= c.B) {
      from[i] = x;
      n_req[i] = y;  // for now, the end
      len[i] = n;
      ends = max(ends, y);
    } else if (blockIdx.x == 0) {
      atomicOr(&a.status[min(max(x, 0), c.B - 1)], BASTION_STATUS_BAD_GROUP);
    }
  }
  int before = ends;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFull, before, o);
    if (lane >= o) before = max(before, x);
  }
  if (lane == 31) ms.warp_max[warp] = before;
  before = __shfl_up_sync(kFull, before, 1);
  if (lane == 0) before = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms.tmem;
#pragma unroll
  for (int x = 0; x < kThreads / 32; ++x) before = max(before, x < warp ? ms.warp_max[x] : 0);
  int cnt = 0, sum = 0, items[kPer];
  bool two = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int end = n_req[i];
    from[i] = max(from[i], before);
    n_req[i] = max(0, end - from[i]);
    before = max(before, end);
    if (n_req[i] > 0 && (len[i] < 0 || len[i] > a.cap) && blockIdx.x == 0)
      atomicOr(&a.status[from[i]], BASTION_STATUS_KV_OVERFLOW);
    len[i] = min(max(len[i], 0), a.cap);
    items[i] = tiles_of(len[i]) * m_tiles_of(n_req[i], a.nb) * c.Hkv;
    cnt += items[i] > 0;
    sum += items[i];
    two |= items[i] > 0 && n_req[i] > a.nb;
  }
  int cnt_i = cnt, sum_i = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFull, cnt_i, o), y = __shfl_up_sync(kFull, sum_i, o);
    if (lane >= o) {
      cnt_i += x;
      sum_i += y;
    }
  }
  if (lane == 31) ms.warp_sum[warp] = make_int2(cnt_i, sum_i);
  const int widest = __syncthreads_or(two) ? 2 : 1;
  int rank = cnt_i - cnt, at = sum_i - sum, total = 0, groups = 0;
#pragma unroll
  for (int x = 0; x < kThreads / 32; ++x) {
    const int2 y = ms.warp_sum[x];
    if (x < warp) {
      rank += y.x;
      at += y.y;
    }
    groups += y.x;
    total += y.y;
  }
  const UnitShares sh = UnitShares::of((int)gridDim.x, total, widest);
  const int b0 = sh.begin(blockIdx.x), b1 = sh.begin(blockIdx.x + 1);
  const bool busy = (int)blockIdx.x < sh.n;
  if (tid == 0 && busy && (int)blockIdx.x == sh.n - 1) ms.f1 = total;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (items[i] == 0) continue;
    const int end = at + items[i];
    list[rank] = UnitEntry{from[i] | (g0 + i) << 16, n_req[i], len[i], at};
    if (busy && ((b0 >= at && b0 < end) || (b1 >= at && b1 < end))) {
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {  // the share's begin and end
        const int f = k ? b1 : b0;
        if (f < at || f >= end) continue;
        const TilePlace p = TilePlace::boundary(sh, f - at, tiles_of(len[i]), m_tiles_of(n_req[i], a.nb));
        if (k) {
          ms.f1 = at + p.off;
        } else {
          const bool next = p.off == items[i];  // the next group's begin
          ms.f0 = at + p.off;
          ms.li0 = next ? rank + 1 : rank;
          ms.from = next ? TilePlace{0, 0, 0, 0} : p;
        }
      }
    }
    ++rank;
    at = end;
  }
  __syncthreads();
  const int share = __shfl_sync(kFull, busy ? ms.f1 - ms.f0 : 0, 0), li0 = __shfl_sync(kFull, ms.li0, 0);
  const TilePlace from_here = {__shfl_sync(kFull, ms.from.head, 0), __shfl_sync(kFull, ms.from.pair, 0),
                               __shfl_sync(kFull, ms.from.t, 0), 0};
  Units<true> w;
  w.start(list, li0, from_here, share, a.nb);

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------ TMA: warp 0 keys, warp 2 values
    // tile x of the share has its keys in stage 2 x and its values in stage 2 x + 1 of the ring
    const int odd = warp >> 1;
    const CUtensorMap *map = odd ? &tm_v : &tm_k;
    const uint32_t one = elect_one();
    // Table entries are read in batches of kBatch tiles, a batch ahead of their use, so that the
    // reads' latency never holds up the copies.  Lane: page lane % ppt of the batch's tile lane / ppt.
    const int psh = 7 - c.shift, ppt = 1 << psh, batch = min(kBatch, 32 >> psh);
    Units<false> lw;  // this lane's tile
    lw.start(list, li0, from_here, share, a.nb);
    int lead = lane >> psh;
    auto next_entry = [&]() {  // walks on by `lead` tiles and reads there
#pragma unroll 1
      for (int x = 0; x < lead && lw.left > 0; ++x) lw.step(c.Hkv, a.nb);
      lead = batch;
      const int pg = (lw.t << psh) + (lane & (ppt - 1));
      const bool on = (lane >> psh) < batch && lw.left > 0 && (pg << c.shift) < lw.len;
      int e = on ? __ldcg(a.table + (size_t)lw.group * a.max_pages + pg) : 0;
      if (e < 0 || e >= c.n_pages) {  // no page of the pool: page 0 stands in
        atomicOr(&a.status[lw.req], BASTION_STATUS_BAD_PAGE);
        e = 0;
      }
      __syncwarp();
      return e;
    };
    int entry = 0, entry_n = next_entry(), in_batch = batch;
    // a prefix that one unit a head reads: not at the parts' expense; several units: the others find it in L2
    const uint64_t once = l2_evict_first_policy(), again = l2_evict_normal_policy();
    const uint32_t ring32 = smem_u32(smem), full32 = smem_u32(ms.full);
    int issued = 0;
#pragma unroll 1
    for (; w.left > 0; w.step(c.Hkv, a.nb)) {
      if (in_batch == batch) {
        entry = entry_n;
        entry_n = next_entry();
        in_batch = 0;
      }
      const int x = 2 * issued + odd, slot = Tiles::stage(x);
      RingBars bars{ms, abort, &a.status[w.req], lane};
      if (!Tiles::before(bars, x)) break;
      const int np = (min(kTileKeys, w.len - w.t * kTileKeys) + c.page - 1) >> c.shift;
      if (one) mbar_arrive_expect_tx(&ms.full[slot], (uint32_t)(np << c.shift) * (uint32_t)(D * 2));
      uint32_t dst = ring32 + (uint32_t)slot * Lay::kTile;
      const int c1 = a.swap ? w.head : 0, c2 = a.swap ? 0 : w.head;
#pragma unroll 4
      for (int p = 0; p < np; ++p) {
        const int id = __shfl_sync(kFull, entry, (in_batch << psh) + p);
#pragma unroll
        for (int blk = 0; blk < kBlocks; ++blk)
          tma_load_4d(one, dst + (uint32_t)blk * Lay::kBlock, map, blk * 64, c1, c2, id, full32 + 8u * (uint32_t)slot,
                      w.m_tiles > 2 ? again : once);
        dst += (uint32_t)(128 << c.shift);
      }
      ++issued;
      ++in_batch;
    }
    if (odd == 0 && issued > 0 && w.left == 0) {
      RingBars bars{ms, abort, &a.status[w.req], lane};
      Tiles::after_keys(bars, issued);
    }
    // our last copies have landed (bounded) before the CTA may exit
    if (lane == 0) {
      for (int u = max(0, issued - kStages / 2); u < issued; ++u)
        mbar_wait_bounded(&ms.full[Tiles::stage(2 * u + odd)], Tiles::full_parity(2 * u + odd));
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    // Visit i (a key tile and an M tile) belongs to warpgroup i % 2.  S of visit i + 2 goes out right
    // after P V of visit i, whose P it overwrites: products of one thread execute in order.
    constexpr uint32_t id_s = idesc<kHalf>(false, false, kTileKeys), id_o = idesc<kHalf>(false, true, D);
    const uint32_t one = elect_one();
    const uint64_t d_ring = desc(smem_u32(smem), 16, 1024, 2), d_q = desc(smem_u32(smem + Lay::kOffQ), 16, 1024, 2);
    const uint64_t d_v = desc(smem_u32(smem), Lay::kBlock, 1024, 2);
    Units<true> pw = w;
    int i_s = 0, m_s = 0, x_s = 0, q_s = 0;        // of the next S: visit, M tile, key tile, M tiles of segments before
    int i_p = 0, m_p = 0, x_p = 0, seg_p = 0;      // of the next P V: ..., key tile of its segment
    auto scores = [&]() {
      const int wg = i_s & 1, x = 2 * x_s, slot = Tiles::stage(x), q = q_s + m_s, count = w.ms();
      int32_t *st = &a.status[w.req];
      if (!__all_sync(kFull, (!w.first || wait_bar(&ms.q_full[q & 1], (uint32_t)(q >> 1) & 1u, abort, st)) &&
                                 wait_bar(&ms.full[slot], Tiles::full_parity(x), abort, st)))
        return false;
      tc_fence_after();
      const uint64_t dk = d_ring + (uint32_t)slot * (Lay::kTile >> 4), dq = d_q + (uint32_t)(q & 1) * (Lay::kTile >> 4);
#pragma unroll
      for (int y = 0; y < D / 16; ++y) {
        const uint32_t off = (uint32_t)(y >> 2) * (Lay::kBlock >> 4) + (uint32_t)(y & 3) * 2u;
        mma(one, tmem + 128u * (uint32_t)wg, dq + off, dk + off, id_s, y > 0);
      }
      mma_commit(one, &ms.s_full[wg]);
      if (w.last()) mma_commit(one, &ms.q_empty[q & 1]);
      ++i_s;
      if (++m_s == count) {
        mma_commit(one, &ms.empty[slot]);
        m_s = 0;
        ++x_s;
        if (w.last()) q_s += count;
        w.step(c.Hkv, a.nb);
      }
      return true;
    };
    auto values = [&]() {
      const int wg = i_p & 1, x = 2 * x_p + 1, slot = Tiles::stage(x), count = pw.ms();
      int32_t *st = &a.status[pw.req];
      const bool fresh = chain_place(seg_p, count) < 3 - count;  // a chain's first visit of this warpgroup: key tile 0, or 0 and 1
      const uint64_t dv = d_v + (uint32_t)slot * (Lay::kTile >> 4);
      const uint32_t p_col = tmem + 128u * (uint32_t)wg, o_col = tmem + 256u + 128u * (uint32_t)wg;
#pragma unroll
      for (int part = 0; part < 2; ++part) {  // the upper 64 keys, whose weights are formed first, then the lower
        if (!__all_sync(kFull, wait_bar(&ms.p_full[wg][part], (uint32_t)(i_p >> 1) & 1u, abort, st) &&
                                   (part > 0 || wait_bar(&ms.full[slot], Tiles::full_parity(x), abort, st))))
          return false;
        tc_fence_after();
#pragma unroll
        for (int z = 0; z < kTileKeys / 32; ++z) {  // 16 keys: 8 columns of high terms, 16 further on those of low terms
          const int y = z + (part == 0 ? kTileKeys / 32 : 0);
          const uint32_t p = p_col + 32u * (uint32_t)(y >> 1) + 8u * (uint32_t)(y & 1);
          mma_ta(one, o_col, p, dv + 128u * (uint32_t)y, id_o, part + z > 0 ? 1u : fresh ? 0u : 1u);
          mma_ta(one, o_col, p + 16u, dv + 128u * (uint32_t)y, id_o, 1u);
        }
      }
      mma_commit(one, &ms.pv_done[wg]);
      ++i_p;
      if (++m_p == count) {
        mma_commit(one, &ms.empty[slot]);
        m_p = 0;
        ++x_p;
        ++seg_p;
        if (pw.last()) seg_p = 0;
        pw.step(c.Hkv, a.nb);
      }
      return true;
    };
    bool ok = true;
    for (int y = 0; y < 2; ++y) ok = ok && (w.left == 0 || scores());
    while (ok && pw.left > 0) ok = values() && (w.left == 0 || scores());
    // every product issued has completed (bounded) before the CTA may free its TMEM
    mma_commit(one, &ms.mma_done);
    mbar_wait_bounded(&ms.mma_done, 0);
  } else if (warp == 3) {
    // ------------------------------------------------------------ queries of each segment
    const uint32_t one = elect_one();
    const uint64_t policy = l2_evict_first_policy();
    const uint32_t q32 = smem_u32(smem + Lay::kOffQ), full32 = smem_u32(ms.q_full);
    int q = 0;
    for (; w.left > 0; w.step(c.Hkv, a.nb)) {
      if (!w.first) continue;
      bool ok = true;
      for (int m = 0; ok && m < w.ms(); ++m, ++q) {
        const int slot = q & 1;
        ok = __all_sync(kFull, wait_bar(&ms.q_empty[slot], ((uint32_t)(q >> 1) & 1u) ^ 1u, abort, &a.status[w.req]));
        if (!ok) break;
        if (one) mbar_arrive_expect_tx(&ms.q_full[slot], (uint32_t)(a.nb * a.G) * (uint32_t)(D * 2));
#pragma unroll
        for (int blk = 0; blk < kBlocks; ++blk)
          tma_load_4d(one, q32 + (uint32_t)slot * Lay::kTile + (uint32_t)blk * Lay::kBlock, &tm_q, blk * 64, 0, w.head,
                      w.req + (2 * w.pair + m) * a.nb, full32 + 8u * (uint32_t)slot, policy);
      }
      if (!ok) break;
    }
    // where the join finds each request's parts
    for (int x = blockIdx.x * 32 + lane; x < c.B * c.Hkv; x += gridDim.x * 32) {
      const int b = x / c.Hkv, head = x - b * c.Hkv;
      int lo = 0, hi = groups;
      while (hi - lo > 1) {  // the last group that begins at b or before
        const int mid = (lo + hi) >> 1;
        if ((list[mid].who & 0xffff) <= b) lo = mid; else hi = mid;
      }
      PartsRec r = {0, 0, 0, 0, 0, 0, 0, 0};
      if (groups > 0) {
        const UnitEntry l = list[lo];
        const int place = b - (l.who & 0xffff), m = place / a.nb;
        if (place >= 0 && place < l.n) {
          const UnitParts u = UnitParts::of(sh, l.at, tiles_of(l.len), m_tiles_of(l.n, a.nb), head, m);
          r.parts = u.count();
          r.two = u.planes == 2;
          r.whole = u.whole;
          r.place0 = (int)(u.whole ? whole_part(0, head, b - (place - m * a.nb), c, a.G) : cut_part(u.slot(0), u.plane));
          r.place1 = u.whole ? 0 : (int)cut_part(u.slot(1), u.plane);
          r.step = u.whole ? c.Hkv * c.B * a.G : 128;
          r.rows = min(a.nb, l.n - m * a.nb) * a.G;
          r.first = (place - m * a.nb) * a.G;
        }
      }
      a.rec[x] = r;
    }
    if (lane == 0)
      for (int u = max(0, q - 2); u < q; ++u) mbar_wait_bounded(&ms.q_full[u & 1], (uint32_t)(u >> 1) & 1u);
  } else {
    // ------------------------------------------------------------ softmax and parts: a thread is a row
    const int wg = (warp - 4) >> 2, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t s_col = tmem + ((uint32_t)(quad * 32) << 16) + 128u * (uint32_t)wg, o_col = s_col + 256u;
    int visits = 0, x_t = 0;  // this warpgroup's visits; the share's key tiles
    int par = 0, par0 = 0, t0 = 0, rows = 0, m = 0;
    bool any = false, stored = false, ok = true;  // something in O; in the part's place
    float ref = -INFINITY, ref_stored = 0.f, l = 0.f;
    for (; w.left > 0; w.step(c.Hkv, a.nb), ++x_t) {
      const int count = w.ms();
      int32_t *st = &a.status[w.req];
      if (w.first) {
        par0 = par;
        t0 = w.t;
        m = count == 2 ? wg ^ par : 0;
        rows = min(a.nb, w.n - (2 * w.pair + m) * a.nb) * a.G;
        any = stored = false;
        ref = -INFINITY;
        l = 0.f;
      }
      if (count == 2 || par == wg) {
        const int valid = w.len - w.t * kTileKeys;  // keys of the tile, where it is the last
        ok = __all_sync(kFull, wait_bar(&ms.s_full[wg], (uint32_t)visits & 1u, abort, st));
        if (!ok) break;
        tc_fence_after();
        if (valid < kTileKeys && (count == 1 || m == 0)) {  // value rows past the end: zeros, whatever the page holds there
          const int x = 2 * x_t + 1, slot = Tiles::stage(x);
          ok = __all_sync(kFull, wait_bar(&ms.full[slot], Tiles::full_parity(x), abort, st));
          if (!ok) break;
          unsigned char *tile = smem + slot * Lay::kTile;
#pragma unroll 1
          for (int y = valid * 128 + row * 16; y < kTileKeys * 128; y += 128 * 16)
#pragma unroll
            for (int blk = 0; blk < kBlocks; ++blk)
              *reinterpret_cast<uint4 *>(tile + blk * Lay::kBlock + y) = make_uint4(0, 0, 0, 0);
          fence_async_smem();
        }
        const auto hand_over = [&](int part) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ms.p_full[wg][part]);
        };
        if (quad * 32 < rows) {
          // 32 keys at a time, the next ones' load under the work on the last; the upper half of the scores
          // stays in registers from the maximum to the weights
          uint32_t va[32], vb[32], vc[32], vd[32];
          if (valid < kTileKeys) mask_scores(s_col, valid);
          float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          ld32(s_col, va);
          wait_ld(va);
          ld32(s_col + 32u, vb);
          top_of(tops, va);
          wait_ld(vb);
          ld32(s_col + 64u, vc);
          top_of(tops, vb);
          wait_ld(vc);
          ld32(s_col + 96u, vd);
          top_of(tops, vc);
          wait_ld(vd);
          top_of(tops, vd);
          const float top = fmaxf(max3f(tops[0], tops[1], tops[2]), tops[3]) * a.scale_log2;
          const bool grow = top > ref + (kBias + kGrow);
          const float to = grow ? top - kBias : ref, alpha = grow ? ex2f(ref - to) : 1.0f;
          if (any && __any_sync(kFull, grow)) {  // S is there: the products before it, all of this O, are done
#pragma unroll 1
            for (int k = 0; k < D / 8; ++k) move_o(o_col + 8u * (uint32_t)k, alpha);
          }
          ref = to;
          l *= alpha;
          const float base = ref == -INFINITY ? 0.f : -ref;
          float sum0 = 0.f, sum1 = 0.f;
          const auto weights = [&](const uint32_t (&v)[32], int k) {
            uint32_t z[32];
#pragma unroll
            for (int y = 0; y < 32; y += 2) {
              float p0 = __uint_as_float(v[y]), p1 = __uint_as_float(v[y + 1]);
              fma2(p0, p1, a.scale_log2, base, base);
              p0 = ex2f(p0);
              p1 = ex2f(p1);
              add2(sum0, sum1, p0, p1);
              split_pair<kHalf>(p0, p1, z[y / 2], z[16 + y / 2]);
            }
            st32(s_col + 32u * (uint32_t)k, z);
          };
          weights(vc, 2);
          weights(vd, 3);
          ld32(s_col, va);
          wait_st();
          hand_over(0);
          wait_ld(va);
          ld32(s_col + 32u, vb);
          weights(va, 0);
          wait_ld(vb);
          weights(vb, 1);
          l += sum0 + sum1;
          wait_st();
        } else {
          hand_over(0);
        }
        hand_over(1);
        any = true;
        ++visits;
      }
      if (count == 1) par ^= 1;
      const bool last = w.last();
      if (!last && chain_place(w.t - t0 + 1, count) != 0) continue;

      // ---------------------------------------------------------- the end of a chain, or of the segment
      const bool whole = t0 == 0 && w.t + w.left / count >= w.tiles;
      const int plane = count == 2 ? m : wg ^ par0;
      if (any) {
        ok = __all_sync(kFull, wait_bar(&ms.pv_done[wg], (uint32_t)(visits - 1) & 1u, abort, st));
        if (!ok) break;
        tc_fence_after();
      }
      if (quad * 32 < rows) {
        const size_t place = whole ? whole_part(count == 2 ? 0 : plane, w.head, w.req + (2 * w.pair + m) * a.nb, c, a.G)
                                   : cut_part(2 * blockIdx.x + (t0 == 0), plane);
        float *dst = (whole ? a.rows : a.parts) + place * D + row * 4;
        float2 *ml = (whole ? a.rows_ml : a.parts_ml) + place + row;
        if (any) {
          const float before = ref_stored == ref ? 1.f : ex2f(ref_stored - ref);
#pragma unroll 1
          for (int k = 0; k < D / 32; ++k) {
            uint32_t o[32];
            ld32(o_col + 32u * (uint32_t)k, o);
            wait_ld(o);
            if (row < rows) {
              if (stored) {
#pragma unroll
                for (int y = 0; y < 32; y += 4) {
                  const float4 x = *reinterpret_cast<const float4 *>(dst + (size_t)(32 * k + y) * rows);
                  o[y] = __float_as_uint(fmaf(x.x, before, __uint_as_float(o[y])));
                  o[y + 1] = __float_as_uint(fmaf(x.y, before, __uint_as_float(o[y + 1])));
                  o[y + 2] = __float_as_uint(fmaf(x.z, before, __uint_as_float(o[y + 2])));
                  o[y + 3] = __float_as_uint(fmaf(x.w, before, __uint_as_float(o[y + 3])));
                }
              }
#pragma unroll
              for (int y = 0; y < 32; y += 4)
                *reinterpret_cast<uint4 *>(dst + (size_t)(32 * k + y) * rows) = make_uint4(o[y], o[y + 1], o[y + 2], o[y + 3]);
            }
          }
        }
        if (row < rows && last) *ml = make_float2(ref, l);
        tc_fence_before();  // the next chain's products overwrite O after this warp's next arrival
      }
      if (any) ref_stored = ref;
      stored = stored || any;
      any = false;
    }
    // A warp may give up alone, the others' waits ending just in time: it flags every request itself, not its rows' share.
    const Units<true> stop = w;
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      const int row = 32 * k + lane;
      Units<true> w = stop;
      if (!ok) {  // a wait ran out, of which only one request has been told
        for (; w.left > 0; w.step(c.Hkv, a.nb))
          for (int b = w.req + row; b < w.req + w.n; b += 128) atomicOr(&a.status[b], BASTION_STATUS_TIMEOUT);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
  griddep_wait();  // the join, which waits for this launch, reads what the one before wrote
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// Queries as (D, head of the group, KV head, request); a box is an M tile's rows, 64 elements wide.
bool make_q_map(CUtensorMap *m, const void *q, const Paged &c, int Hq, int64_t q_st_b, int nb, bool half) {
  auto enc = get_encode();
  if (!enc) return false;
  const cuuint64_t G = (cuuint64_t)(Hq / c.Hkv), D = (cuuint64_t)c.D;
  cuuint64_t dims[4] = {D, G, (cuuint64_t)c.Hkv, (cuuint64_t)c.B};
  cuuint64_t strides[3] = {D * 2, G * D * 2, (cuuint64_t)(c.B > 1 ? q_st_b : (int64_t)Hq * c.D) * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)G, 1, (cuuint32_t)nb};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(q), dims,
             strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kHalf, int D>
cudaError_t launch_parts(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, int dev, const Paged &c,
                         const PrefixArgs &a, cudaStream_t stream) {
  constexpr uint32_t smem = smem_bytes<D>();
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(paged_prefix_kernel<kHalf, D>, (int)smem, dev, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(paged_prefix_kernel<kHalf, D>, dim3((unsigned)a.n_ctas), dim3(kThreads), smem, stream, mq, mk, mv, c, a);
}

struct Sizes {
  size_t own_ws, own, own_lse, rec, rows, rows_ml, parts, parts_ml;
  size_t all() const { return own_ws + own + own_lse + rec + rows + rows_ml + parts + parts_ml; }
};
Sizes sizes_of(int B, int Hq, int Hkv, int D) {
  const size_t rows = (size_t)B * Hq, parts = (size_t)2 * kMaxParts * 2 * 128;
  Sizes s;
  s.own_ws = up256(paged_attention_workspace_bytes(B, Hq, Hkv, D, 1, 0));
  s.own = up256(rows * D * 4);
  s.own_lse = up256(rows * 4);
  s.rec = up256((size_t)B * Hkv * sizeof(PartsRec));
  s.rows = 2 * rows * D * 4;
  s.rows_ml = up256(2 * rows * 8);
  s.parts = parts * D * 4;
  s.parts_ml = parts * 8;
  return s;
}

}  // namespace

size_t paged_prefix_workspace_bytes(int B, int Hq, int Hkv, int D, int n_groups) {
  (void)n_groups;
  return sizes_of(B, Hq, Hkv, D).all();
}

int launch_paged_prefix(const Paged &c, bool half, const int32_t *prefix_table, int max_prefix_pages,
                        const int32_t *prefix_len, const int32_t *group_start, int n_groups, const void *q, int Hq,
                        int64_t q_st_b, const int32_t *seq_len, float scale, void *out, float *lse, void *ws,
                        int32_t *status, cudaStream_t stream) {
  const Sizes sz = sizes_of(c.B, Hq, c.Hkv, c.D);
  PrefixArgs a;
  a.table = prefix_table;
  a.len = prefix_len;
  a.start = group_start;
  a.n_groups = n_groups;
  a.max_pages = max_prefix_pages;
  a.cap = max_prefix_pages * c.page;
  a.Hq = Hq;
  a.G = Hq / c.Hkv;
  a.nb = 128 / a.G;
  a.scale_log2 = scale * kLog2e;
  a.swap = c.Hkv > 1 && c.st_head < c.st_slot;
  char *at = static_cast<char *>(ws) + sz.own_ws;
  auto take = [&](size_t n) {
    char *p = at;
    at += n;
    return p;
  };
  a.own = reinterpret_cast<float *>(take(sz.own));
  a.own_lse = reinterpret_cast<float *>(take(sz.own_lse));
  a.rec = reinterpret_cast<PartsRec *>(take(sz.rec));
  a.rows = reinterpret_cast<float *>(take(sz.rows));
  a.rows_ml = reinterpret_cast<float2 *>(take(sz.rows_ml));
  a.parts = reinterpret_cast<float *>(take(sz.parts));
  a.parts_ml = reinterpret_cast<float2 *>(take(sz.parts_ml));
  a.out = static_cast<uint16_t *>(out);
  a.lse = lse;
  a.status = status;
  CUtensorMap mq, mk, mv;
  if (!make_q_map(&mq, q, c, Hq, q_st_b, a.nb, half) || !make_map(&mk, c.k, c, a.swap, half) ||
      !make_map(&mv, c.v, c, a.swap, half))
    return BASTION_ERR_LAUNCH;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return BASTION_ERR_LAUNCH;
  a.n_ctas = sms < kMaxParts ? sms : kMaxParts;
  a.q = static_cast<const uint16_t *>(q);
  a.q_st_b = q_st_b;
  a.seq_len = seq_len;
  if (c.cap <= own_slots(c.D)) {
    if (launch_prefix_own(half, sms, c, a, stream) != cudaSuccess) return BASTION_ERR_LAUNCH;
  } else {
    const int rc = launch_paged_attention32(c, half, q, Hq, q_st_b, seq_len, scale, a.own, a.own_lse, ws, status, stream);
    if (rc != BASTION_OK) return rc;
  }
  const bool wide = c.D == 128;
  cudaError_t e = half ? (wide ? launch_parts<true, 128>(mq, mk, mv, dev, c, a, stream) : launch_parts<true, 64>(mq, mk, mv, dev, c, a, stream))
                       : (wide ? launch_parts<false, 128>(mq, mk, mv, dev, c, a, stream) : launch_parts<false, 64>(mq, mk, mv, dev, c, a, stream));
  if (e == cudaSuccess) e = launch_prefix_join(half, sms, c, a, stream);
  return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? BASTION_OK : BASTION_ERR_LAUNCH;
}

}  // namespace bastion
