// Eviction from the paged cache by accumulated attention weight.
//
// One launch; a cluster of 1 to 8 CTAs per (request, KV head).  Slot j's key is
// its weight as an order-preserving 32-bit integer, the protected slots' above
// all weights.  A histogram of the keys' top 12 bits, summed over the cluster,
// gives the bin that holds the budget-th largest key; that bin's keys are
// gathered and ranked against one another (or, when they are many, split by two
// more histograms of 10 bits), which gives the budget-th largest key t
// and how many of the slots that tie with it stay.  One count in slot order
// then gives both lists of the moves: the i-th hole (a slot below budget that
// is not kept) takes the i-th kept slot at or past budget, with
//   K(s) = kept slots before s = #(key > t before s) + min(#(key == t before s), ties that stay)
//   hole index of s < budget: s - K(s);   source index of s >= budget: K(s) - K(budget).
// Sources lie at or past budget and targets below it, so that no move reads
// what another writes.  Weights and positions are read once (the keys stay in
// shared memory) and only the holes' rows move.
//
// Few tokens leaving (32 requests x 8 heads, 2,065 slots cut to 2,048): 10.2 us with the weights in L2
// (11.6 without), a chain of some ten phases with a barrier each, against 1.9 us of traffic; as two
// launches it took 14.2 us.  Prompts cut (8 x 8 heads, up to 32,768 slots to 4,096): 56 us, of which the moves take two
// thirds at 5.5 TB/s (rows of 256 bytes in no order) and the selection the rest; as two
// launches, one CTA a head selecting, 88 us.  11, 12 or 13 bits in the first histogram are alike
// within 3% (12 leaves fewer keys in the bin than 11 and clears faster than 13).  The loops take a
// key a lane and little code: every phase runs once or a few times, and its instructions have to
// be fetched (four keys a lane, unrolled: 5 to 8% slower when few tokens leave, 2% faster on prompts).
#include "paged.cuh"

namespace bastion {

namespace {

constexpr uint32_t kSafe = 0xffffffffu;  // key of a protected slot
constexpr int kBits0 = 12, kBits1 = 10, kBits2 = 10;
constexpr int kBins0 = 1 << kBits0, kBins1 = 1 << kBits1, kBins2 = 1 << kBits2;
constexpr int kHist = kBins0 + kBins1 + kBins2;
constexpr int kCand = 256;       // keys of one bin that are ranked directly
constexpr int kNearMoves = 512;
constexpr int kMaxCluster = 8;
constexpr int kKeysMax = 45056;  // keys a CTA keeps in shared memory
constexpr int kMovesWarp = 8;    // moves a warp has in flight

struct EvictArgs {
  const int32_t *seq_len, *n_seen;
  const float *acc;
  const int32_t *pos;
  int budget, n_sink, n_recent, max_moves;
  int32_t *seq_len_out;
  float *acc_out;
  int32_t *pos_out;
  uint32_t *arrived;  // [kMaxRequests], zero between calls
  int2 *moves;        // [units, max_moves] (source slot, target slot)
  int copy;           // acc_out or pos_out is not its input
  int32_t *status;
};

// Key of slot s < end: larger is kept first.  (At or past the end: of no meaning, and no NaN is reported.)
__device__ __forceinline__ uint32_t slot_key(float w, int pos, int sink, int64_t recent, int s, int end, bool &nan) {
  const bool safe = pos < sink || pos >= recent, bad = w != w;
  nan |= bad && !safe && s < end;
  return safe ? kSafe : ord_f32(bad ? INFINITY : w);  // at most ord(+inf) = 0xff800000
}

struct Misc {
  uint32_t warp_sum[3][32];             // entries of each warp's run of bins, of each pass (others may still read one)
  uint32_t warp_gt[32], warp_eq[32];
  alignas(16) uint32_t count[4];        // this CTA's keys above t, equal to t, and of these below budget
  uint32_t bin, above, in_bin;
  uint32_t n_cand;
};

__device__ __forceinline__ uint4 dsmem_ld_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ uint32_t warp_scan(uint32_t x, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// kKeys: the keys of the CTA's segment stay in shared memory (else they are formed anew for each pass).
template <bool kKeys>
__global__ void __launch_bounds__(1024) paged_evict_kernel(Paged c, EvictArgs a, int cs) {
  extern __shared__ __align__(16) uint32_t smem[];
  uint32_t *hist = smem, *keys = smem + kHist;
  __shared__ Misc ms;
  __shared__ __align__(16) uint32_t cand[kCand];  // the bin's keys: this CTA's, then the cluster's
  __shared__ int2 near_moves[kNearMoves];         // the list of moves where it is short and one CTA's
  griddep_wait();
  griddep_launch_dependents();
  const int unit = blockIdx.x / cs, part = blockIdx.x % cs, r = unit / c.Hkv, g = unit % c.Hkv;
  const int tid = threadIdx.x, T = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = T >> 5;
  const size_t base = (size_t)unit * c.cap;
  const float *acc = a.acc + base;
  const int32_t *pos = a.pos + base;
  float *acc_out = a.acc_out + base;
  int32_t *pos_out = a.pos_out + base;
  // A row of acc and pos is whole vectors of 4 (pages have 8 slots at least).  A lone CTA's first
  // vectors do not depend on the length: they are under way before it is known.
  float4 w[2];
  int4 p[2];
  auto fetch = [&](int v0, int end) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int s = v0 + 4 * (u * T + tid);
      if (s < end) {
        w[u] = *reinterpret_cast<const float4 *>(acc + s);
        p[u] = *reinterpret_cast<const int4 *>(pos + s);
      }
    }
  };
  if (kKeys && cs == 1) fetch(0, c.cap);
  const int n = paged_len(c, a.seq_len, r, a.status);
  const int64_t recent = (int64_t)a.n_seen[r] - a.n_recent;
  for (int i = tid; i < kHist / 4; i += T) reinterpret_cast<uint4 *>(hist)[i] = make_uint4(0, 0, 0, 0);
  if (tid == 0) ms.n_cand = 0;
  if (tid < 4) ms.count[tid] = 0;

  // The lengths may be updated in place: the last of the request's CTAs to have
  // read them writes.  A CTA says so after the barrier behind its threads' reads
  // (whose values they have used by then) and looks at the answer when it is done.
  uint32_t readers = 0;
  auto length_read = [&]() {
    if (tid == 0)
      asm volatile("atom.add.relaxed.gpu.global.u32 %0, [%1], 1;" : "=r"(readers) : "l"(&a.arrived[r]) : "memory");
  };
  auto write_length = [&]() {
    if (tid == 0 && readers == (uint32_t)(c.Hkv * cs - 1)) {
      a.arrived[r] = 0;
      const int raw = a.seq_len[r];
      a.seq_len_out[r] = raw > a.budget ? a.budget : raw;
    }
  };
  // this CTA's segment of the slots, in whole vectors of 4
  const int seg = ((n + cs - 1) / cs + 3) & ~3, s0 = min(n, part * seg), s1 = min(n, s0 + seg), count = s1 - s0;
  auto cluster_sync = [&]() {
    if (cs > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
  };
  // Where acc_out and pos_out are other arrays, the slots below budget are copied (the holes among
  // them are written over by the moves): with the keys, in whole vectors, or here slot by slot.
  auto copy_slots = [&](int from, int to) {
#pragma unroll 2
    for (int s = from + tid; s < to; s += T) {
      acc_out[s] = acc[s];
      pos_out[s] = pos[s];
    }
  };
  if (n <= a.budget) {  // the whole cluster: nothing leaves
    if (a.copy) copy_slots(s0, s1);
    __syncthreads();
    length_read();
    write_length();
    return;
  }

  bool nan = false;
  if (kKeys) {
#pragma unroll 1
    for (int v0 = s0; v0 < s1; v0 += 8 * T) {
      if (cs > 1 || v0 > 0) fetch(v0, s1);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int s = v0 + 4 * (u * T + tid);
        if (s >= s1) continue;
        uint4 k;  // slots past the end are never looked at
        k.x = slot_key(w[u].x, p[u].x, a.n_sink, recent, s, s1, nan);
        k.y = slot_key(w[u].y, p[u].y, a.n_sink, recent, s + 1, s1, nan);
        k.z = slot_key(w[u].z, p[u].z, a.n_sink, recent, s + 2, s1, nan);
        k.w = slot_key(w[u].w, p[u].w, a.n_sink, recent, s + 3, s1, nan);
        *reinterpret_cast<uint4 *>(keys + s - s0) = k;
        if (a.copy && s + 4 <= a.budget) {
          *reinterpret_cast<float4 *>(acc_out + s) = w[u];
          *reinterpret_cast<int4 *>(pos_out + s) = p[u];
        }
      }
    }
  }
  __syncthreads();
  auto key_at = [&](int i) {
    return kKeys ? keys[i] : slot_key(acc[s0 + i], pos[s0 + i], a.n_sink, recent, 0, 1, nan);
  };
#pragma unroll 2
  for (int i0 = 32 * warp; i0 < count; i0 += T) {
    const int i = i0 + lane;
    const bool on = i < count;
    const uint32_t k = on ? key_at(i) : 0u;
    // many protected slots lie side by side: one addition for a warp's
    const uint32_t safe = __ballot_sync(kFull, on && k == kSafe);
    if (on && k != kSafe) atomicAdd(&hist[k >> (32 - kBits0)], 1u);
    if (safe && lane == 0) atomicAdd(&hist[kBins0 - 1], (uint32_t)__popc(safe));
  }
  if (nan) atomicOr(&a.status[r], BASTION_STATUS_NONFINITE);
  length_read();

  // t: the bits found of the budget-th largest key, `shift` more are open; `need` of the keys that
  // begin with t are kept
  uint32_t t = 0, need = (uint32_t)a.budget;
  int shift = 32;
#pragma unroll 1
  for (int pass = 0; pass < 3 && shift > 0; ++pass) {
    const int bits = pass == 0 ? kBits0 : pass == 1 ? kBits1 : kBits2, bins = 1 << bits;
    uint32_t *h = hist + (pass == 0 ? 0 : pass == 1 ? kBins0 : kBins0 + kBins1);
    shift -= bits;
    if (pass > 0) {
#pragma unroll 2
      for (int i = tid; i < count; i += T) {
        const uint32_t k = key_at(i);
        if ((k >> (shift + bits)) == t) atomicAdd(&h[(k >> shift) & (uint32_t)(bins - 1)], 1u);
      }
    }
    __syncthreads();
    // each warp's run of bins, the first warp's topmost: this CTA's entries
    const int run = (bins + 128 * warps - 1) / (128 * warps) * 128, runs = (bins + run - 1) / run;
    uint32_t sum = 0;
    if (warp < runs)
      for (int b = bins - warp * run - 4 * lane - 4; b >= max(bins - (warp + 1) * run, 0); b -= 128) {
        const uint4 x = *reinterpret_cast<const uint4 *>(h + b);
        sum += x.x + x.y + x.z + x.w;
      }
    sum = __reduce_add_sync(kFull, sum);
    if (lane == 0) ms.warp_sum[pass][warp] = sum;
    cluster_sync();
    if (warp == 0) {
      // the run, then the bin, over all CTAs of the cluster
      uint32_t own = lane < runs ? ms.warp_sum[pass][lane] : 0u;
      if (cs > 1)
#pragma unroll
      for (int o = 1; o < kMaxCluster; ++o)
        if (o < cs && lane < runs) own += dsmem_ld_u32(dsmem_addr(&ms.warp_sum[pass][lane], (uint32_t)((part + o) & (cs - 1))));
      uint32_t incl = warp_scan(own, lane);
      const int in_run = __ffs(__ballot_sync(kFull, incl >= need)) - 1;  // need <= all entries
      uint32_t before = __shfl_sync(kFull, incl - own, in_run);
      for (int b0 = bins - in_run * run; b0 > 0; b0 -= 128) {
        const int b = b0 - 4 * lane - 4;
        uint4 x = *reinterpret_cast<const uint4 *>(h + b);
        if (cs > 1)
#pragma unroll
        for (int o = 1; o < kMaxCluster; ++o) {
          const uint4 y = o < cs ? dsmem_ld_v4(dsmem_addr(h + b, (uint32_t)((part + o) & (cs - 1)))) : make_uint4(0, 0, 0, 0);
          x.x += y.x;
          x.y += y.y;
          x.z += y.z;
          x.w += y.w;
        }
        own = x.x + x.y + x.z + x.w;
        incl = warp_scan(own, lane);
        uint32_t above = before + incl - own;
        if (above < need && above + own >= need) {  // one lane
          const uint32_t y[4] = {x.w, x.z, x.y, x.x};
          int at = 0;
#pragma unroll
          for (int q = 0; q < 3; ++q)
            if (at == q && above + y[q] < need) {
              above += y[q];
              ++at;
            }
          ms.bin = (uint32_t)(b + 3 - at);
          ms.above = above;
          ms.in_bin = at == 0 ? y[0] : at == 1 ? y[1] : at == 2 ? y[2] : y[3];
        }
        before += __shfl_sync(kFull, incl, 31);
        if (before >= need) break;
      }
    }
    __syncthreads();
    need -= ms.above;
    t = (t << bits) | ms.bin;
    const uint32_t in_bin = ms.in_bin;
    if (shift > 0 && in_bin <= (uint32_t)kCand) {
      // few keys begin with t: gather them and rank each against all
#pragma unroll 2
      for (int i = tid; i < count; i += T) {
        const uint32_t k = key_at(i);
        if ((k >> shift) == t) cand[atomicAdd(&ms.n_cand, 1u)] = k;
      }
      cluster_sync();
      const int own = (int)ms.n_cand;
      int m = own;
      if (cs > 1) {
        // the other CTAs' keys behind this CTA's own, a warp a CTA; each CTA only ever reads the
        // first n_cand of another, which do not change any more
        const uint32_t peer = (uint32_t)((part + lane) & (cs - 1));
        const uint32_t theirs = lane < cs ? dsmem_ld_u32(dsmem_addr(&ms.n_cand, peer)) : 0u;
        const uint32_t end = warp_scan(theirs, lane);
        m = (int)__shfl_sync(kFull, end, 31);
        if (warp > 0 && warp < cs) {
          const int k = (int)__shfl_sync(kFull, theirs, warp), at = (int)__shfl_sync(kFull, end, warp) - k;
          for (int i = lane; i < k; i += 32)
            cand[at + i] = dsmem_ld_u32(dsmem_addr(cand + i, (uint32_t)((part + warp) & (cs - 1))));
        }
        __syncthreads();
      }
      for (int i = tid; i < m; i += T) {
        const uint32_t k = cand[i];
        uint32_t gt = 0, eq = 0;
#pragma unroll 2
        for (int j = 0; j < m; j += 4) {
          const uint4 x = *reinterpret_cast<const uint4 *>(cand + j);
          gt += (x.x > k) + (j + 1 < m && x.y > k) + (j + 2 < m && x.z > k) + (j + 3 < m && x.w > k);
          eq += (x.x == k) + (j + 1 < m && x.y == k) + (j + 2 < m && x.z == k) + (j + 3 < m && x.w == k);
        }
        if (gt < need && gt + eq >= need) {  // every thread that holds t writes the same
          ms.bin = k;
          ms.above = gt;
        }
      }
      __syncthreads();
      need -= ms.above;
      t = ms.bin;
      shift = 0;
    }
  }

  // t is the budget-th largest key; `need` of the slots that equal it stay.  Each
  // warp counts its own run of the segment, in whole groups of 32.
  const int run = (count + T - 1) / T * 32, w0 = min(count, warp * run), w1 = min(count, w0 + run);
  const int below = a.budget - s0;  // the segment's slots below it are below budget
  uint32_t gt = 0, eq = 0, gt_b = 0, eq_b = 0;
#pragma unroll 2
  for (int i = w0 + lane; i < w1; i += 32) {
    const uint32_t k = key_at(i);
    gt += k > t;
    eq += k == t;
    gt_b += i < below && k > t;
    eq_b += i < below && k == t;
  }
  gt = __reduce_add_sync(kFull, gt);
  eq = __reduce_add_sync(kFull, eq);
  gt_b = __reduce_add_sync(kFull, gt_b);
  eq_b = __reduce_add_sync(kFull, eq_b);
  if (lane == 0) {
    ms.warp_gt[warp] = gt;
    ms.warp_eq[warp] = eq;
    atomicAdd(&ms.count[0], gt);
    atomicAdd(&ms.count[1], eq);
    atomicAdd(&ms.count[2], gt_b);
    atomicAdd(&ms.count[3], eq_b);
  }
  __syncthreads();
  if (cs > 1) cluster_sync();
  uint32_t g0 = __reduce_add_sync(kFull, lane < warp ? ms.warp_gt[lane] : 0u);
  uint32_t e0 = __reduce_add_sync(kFull, lane < warp ? ms.warp_eq[lane] : 0u);
  uint32_t gb = ms.count[2], eb = ms.count[3];
  if (cs > 1) {
#pragma unroll
    for (int o = 1; o < kMaxCluster; ++o) {
      const int rank = (part + o) & (cs - 1);
      const uint4 x = o < cs ? dsmem_ld_v4(dsmem_addr(ms.count, (uint32_t)rank)) : make_uint4(0, 0, 0, 0);
      if (rank < part) {
        g0 += x.x;
        e0 += x.y;
      }
      gb += x.z;
      eb += x.w;
    }
  }
  const uint32_t kb = gb + min(eb, need);  // kept slots below budget
  const int n_moves = a.budget - (int)kb;
  const bool near = cs == 1 && n_moves <= kNearMoves;
  int2 *moves = near ? near_moves : a.moves + (size_t)unit * a.max_moves;
  const uint32_t lt = (1u << lane) - 1u;
#pragma unroll 1
  for (int i = w0 + lane; i - lane < w1; i += 32) {
    const bool on = i < w1;
    const uint32_t k = on ? key_at(i) : 0u;
    const uint32_t mg = __ballot_sync(kFull, on && k > t), me = __ballot_sync(kFull, on && k == t);
    const uint32_t ee = e0 + __popc(me & lt), before = g0 + __popc(mg & lt) + min(ee, need);
    const bool keep = on && (k > t || (k == t && ee < need));
    if (on && i < below) {
      if (!keep) moves[s0 + i - (int)before].y = s0 + i;
    } else if (keep) {
      moves[before - kb].x = s0 + i;
    }
    g0 += __popc(mg);
    e0 += __popc(me);
  }
  // what the keys' vectors left out
  if (a.copy) copy_slots(kKeys ? max(s0, a.budget & ~3) : s0, min(a.budget, s1));
  cluster_sync();  // the list is whole; no CTA reads another's shared memory any more

  // The moves, T of them at a time.  First a thread a move: its pages, its
  // weight and position; then a warp has the rows of kMovesWarp of them in
  // flight, lanes 0-15 on keys and 16-31 on values (16 bytes each; with D = 64
  // half of them).  The resolved rows take the keys' and bins' place.
  longlong2 *rows = reinterpret_cast<longlong2 *>(smem);
  const int half = lane >> 4, sub = lane & 15;
  const bool row_on = sub < c.D / 8;
  uint16_t *pool = half ? c.v : c.k;
#pragma unroll 1
  for (int m0 = part * T; m0 < n_moves; m0 += cs * T) {
    const int left = min(T, n_moves - m0);
    if (tid < left) {
      const int2 mv = near ? near_moves[m0 + tid] : __ldcg(&moves[m0 + tid]);
      const float x = acc[mv.x];
      const int y = pos[mv.x];
      const int ps = paged_page(c, r, mv.x, a.status), pd = paged_page(c, r, mv.y, a.status);
      rows[tid] = ps >= 0 && pd >= 0 ? make_longlong2(paged_row(c, ps, mv.x, g), paged_row(c, pd, mv.y, g))
                                     : make_longlong2(-1, -1);
      acc_out[mv.y] = x;
      pos_out[mv.y] = y;
    }
    __syncthreads();
#pragma unroll 1
    for (int i = warp * kMovesWarp; i < left; i += warps * kMovesWarp) {
      uint4 v[kMovesWarp];
#pragma unroll
      for (int x = 0; x < kMovesWarp; ++x) {
        const int64_t src = i + x < left ? rows[i + x].x : -1;
        if (src >= 0 && row_on) v[x] = *reinterpret_cast<const uint4 *>(pool + src + sub * 8);
      }
#pragma unroll
      for (int x = 0; x < kMovesWarp; ++x) {
        const int64_t dst = i + x < left ? rows[i + x].y : -1;
        if (dst >= 0 && row_on) *reinterpret_cast<uint4 *>(pool + dst + sub * 8) = v[x];
      }
    }
    __syncthreads();
  }
  write_length();
}

}  // namespace

size_t paged_evict_workspace_bytes(int B, int Hkv, int64_t cap) {
  // at most cap / 2 moves: targets lie below budget, sources at or past it
  return kCounterBytes + (size_t)B * Hkv * (size_t)(cap / 2) * sizeof(int2);
}

int launch_paged_evict(const Paged &c, const int32_t *seq_len, const int32_t *n_seen, const float *acc,
                       const int32_t *pos, int budget, int n_sink, int n_recent, int32_t *seq_len_out,
                       float *acc_out, int32_t *pos_out, void *ws, int32_t *status, cudaStream_t stream) {
  const int units = c.B * c.Hkv;
  EvictArgs a;
  a.seq_len = seq_len;
  a.n_seen = n_seen;
  a.acc = acc;
  a.pos = pos;
  a.budget = budget;
  a.n_sink = n_sink;
  a.n_recent = n_recent;
  a.max_moves = c.cap / 2;
  a.seq_len_out = seq_len_out;
  a.acc_out = acc_out;
  a.pos_out = pos_out;
  a.arrived = static_cast<uint32_t *>(ws);
  a.moves = reinterpret_cast<int2 *>(static_cast<char *>(ws) + kCounterBytes);
  a.copy = acc_out != acc || pos_out != pos;
  a.status = status;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return BASTION_ERR_LAUNCH;
  // CTAs of a unit: up to two an SM over all units, each with 2,048 slots at least (32 units of 8,200 slots: 12.3 us
  // so, 14.7 with half as many slots a CTA, 13.9 with twice as many); more where their keys would not fit
  int cs = 1;
  while (cs < 8 && ((units * cs <= sms && c.cap >= 4096 * cs) || c.cap > cs * kKeysMax)) cs *= 2;
  const int seg = ((c.cap + cs - 1) / cs + 3) & ~3;
  const bool in_smem = seg <= kKeysMax;
  const int T = seg <= 8192 ? 512 : 1024;
  const size_t smem = (size_t)kHist * 4 + (in_smem ? (size_t)seg * 4 : 0);
  auto kernel = in_smem ? paged_evict_kernel<true> : paged_evict_kernel<false>;
  static std::atomic<uint64_t> done[2] = {{0}, {0}};
  cudaError_t e = allow_smem(kernel, (int)((kHist + kKeysMax) * 4), dev, done[in_smem]);
  if (e == cudaSuccess)
    e = launch_cluster_pdl(kernel, dim3((unsigned)(units * cs)), dim3((unsigned)T), smem, stream, cs, c, a, cs);
  return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? BASTION_OK : BASTION_ERR_LAUNCH;
}

}  // namespace bastion
