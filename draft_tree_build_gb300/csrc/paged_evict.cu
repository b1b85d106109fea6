// Eviction from the paged cache by accumulated attention weight.
//
// One launch; a cluster of 1 to 8 CTAs per (request, KV head).  Slot j's key is
// its weight as an order-preserving 32-bit integer, the protected slots' above
// all weights.  A radix select (13 + 10 + 9 bits, histograms in shared memory,
// summed over the cluster) finds the budget-th largest key t and how many of
// the slots that tie with it stay.  One count in slot order then gives both
// lists of the moves: the i-th hole (a slot below budget that is not kept)
// takes the i-th kept slot at or past budget, with
//   K(s) = kept slots before s = #(key > t before s) + min(#(key == t before s), ties that stay)
//   hole index of s < budget: s - K(s);   source index of s >= budget: K(s) - K(budget).
// Sources lie at or past budget and targets below it, so that no move reads
// what another writes.  Weights and positions are read once (the keys stay in
// shared memory) and only the holes' rows move.
//
// 13 bits in the first pass because weights crowd into few octaves: 16 bins an
// octave keep the lanes of a warp out of one another's way, 4 (11 bits) made
// the histogram the longest step.
#include "paged.cuh"

namespace bastion {

namespace {

constexpr uint32_t kSafe = 0xffffffffu;  // key of a protected slot
constexpr int kBits0 = 13, kBits1 = 10, kBits2 = 9;
constexpr int kBins0 = 1 << kBits0, kBins1 = 1 << kBits1, kBins2 = 1 << kBits2;
constexpr int kHist = kBins0 + kBins1 + kBins2;
constexpr int kKeysMax = 45056;  // keys a CTA keeps in shared memory
constexpr int kMovesWarp = 8;    // moves a warp has in flight
constexpr int kMaxRequests = 1024;

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

// Key of a slot: larger is kept first.
__device__ __forceinline__ uint32_t slot_key(float w, int pos, int sink, int64_t recent, bool &nan) {
  if (pos < sink || pos >= recent) return kSafe;
  if (w != w) {
    nan = true;
    w = INFINITY;
  }
  return ord_f32(w);  // at most ord(+inf) = 0xff800000
}

struct Misc {
  uint32_t warp_sum[32];
  uint32_t warp_gt[32], warp_eq[32];
  uint32_t count[4];  // this CTA's keys above t, equal to t, and of these below budget
  uint32_t bin, above;
};

__device__ __forceinline__ uint4 dsmem_ld_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// kKeys: the keys of the CTA's segment stay in shared memory (else they are formed anew for each pass).
template <bool kKeys>
__global__ void __launch_bounds__(1024) paged_evict_kernel(Paged c, EvictArgs a, int cs) {
  extern __shared__ __align__(16) uint32_t smem[];
  uint32_t *hist = smem, *keys = smem + kHist;
  __shared__ Misc ms;
  griddep_wait();
  griddep_launch_dependents();
  const int unit = blockIdx.x / cs, part = blockIdx.x % cs, r = unit / c.Hkv, g = unit % c.Hkv;
  const int tid = threadIdx.x, T = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = T >> 5;
  const int n = paged_len(c, a.seq_len, r, a.status);
  const int64_t recent = (int64_t)a.n_seen[r] - a.n_recent;
  const size_t base = (size_t)unit * c.cap;
  const float *acc = a.acc + base;
  const int32_t *pos = a.pos + base;
  float *acc_out = a.acc_out + base;
  int32_t *pos_out = a.pos_out + base;

  // The lengths may be updated in place: the request's last CTA to have read them writes.
  auto leave = [&]() {
    __syncthreads();
    if (tid == 0) {
      __threadfence();
      if (atomicAdd(&a.arrived[r], 1u) == (uint32_t)(c.Hkv * cs - 1)) {
        a.arrived[r] = 0;
        const int raw = a.seq_len[r];
        a.seq_len_out[r] = raw > a.budget ? a.budget : raw;
      }
    }
  };
  if (n <= a.budget) {  // the whole cluster
    if (a.copy)
      for (int s = part * T + tid; s < n; s += cs * T) {
        acc_out[s] = acc[s];
        pos_out[s] = pos[s];
      }
    leave();
    return;
  }

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
  bool nan = false;
  for (int i = tid; i < kHist / 4; i += T) reinterpret_cast<uint4 *>(hist)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  auto key_at = [&](int i) {
    return kKeys ? keys[i] : slot_key(acc[s0 + i], pos[s0 + i], a.n_sink, recent, nan);
  };
  auto enter = [&](uint32_t k, bool on) {
    // many protected slots lie side by side: one addition for a warp's
    const uint32_t safe = __ballot_sync(kFull, on && k == kSafe);
    if (on && k != kSafe) atomicAdd(&hist[k >> (32 - kBits0)], 1u);
    if (safe && lane == 0) atomicAdd(&hist[kBins0 - 1], (uint32_t)__popc(safe));
  };
  if (kKeys) {
    const int vecs = (count + 3) / 4;  // acc and pos rows are padded to whole vectors by the page size
    for (int v0 = 0; v0 < vecs; v0 += 2 * T) {
      float4 w[2];
      int4 p[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int v = v0 + u * T + tid;
        if (v < vecs) {
          w[u] = *reinterpret_cast<const float4 *>(acc + s0 + 4 * v);
          p[u] = *reinterpret_cast<const int4 *>(pos + s0 + 4 * v);
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int v = v0 + u * T + tid;
        const float *wf = reinterpret_cast<const float *>(&w[u]);
        const int *pf = reinterpret_cast<const int *>(&p[u]);
        uint32_t k[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const bool on = v < vecs && 4 * v + x < count;
          k[x] = on ? slot_key(wf[x], pf[x], a.n_sink, recent, nan) : 0u;
          enter(k[x], on);
        }
        if (v < vecs) *reinterpret_cast<uint4 *>(keys + 4 * v) = make_uint4(k[0], k[1], k[2], k[3]);
      }
    }
  } else {
    for (int i0 = 0; i0 < count; i0 += T) enter(i0 + tid < count ? key_at(i0 + tid) : 0u, i0 + tid < count);
  }
  if (nan) atomicOr(&a.status[r], BASTION_STATUS_NONFINITE);

  uint32_t t = 0, need = (uint32_t)a.budget;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass == 0 ? kBits0 : pass == 1 ? kBits1 : kBits2, bins = 1 << bits;
    uint32_t *h = hist + (pass == 0 ? 0 : pass == 1 ? kBins0 : kBins0 + kBins1);
    if (pass > 0) {
      const int shift = pass == 1 ? kBits2 : 0;
      for (int i = tid; i < count; i += T) {
        const uint32_t k = key_at(i);
        if ((k >> (shift + bits)) == t) atomicAdd(&h[(k >> shift) & (uint32_t)(bins - 1)], 1u);
      }
    }
    cluster_sync();
    // the cluster's sums of bins b .. b + 3
    auto bins4 = [&](int b) {
      uint4 x = *reinterpret_cast<const uint4 *>(h + b);
      for (int o = 1; o < cs; ++o) {
        const uint4 y = dsmem_ld_v4(dsmem_addr(h + b, (uint32_t)((part + o) % cs)));
        x.x += y.x;
        x.y += y.y;
        x.z += y.z;
        x.w += y.w;
      }
      return x;
    };
    // each warp sums its run of bins, the first warp the topmost
    const int run = max(bins / warps, 128), top = bins - warp * run;
    uint32_t sum = 0;
    for (int b = top - 4 * lane - 4; b >= top - run && b >= 0; b -= 128) {
      const uint4 x = bins4(b);
      sum += x.x + x.y + x.z + x.w;
    }
    sum = __reduce_add_sync(kFull, sum);
    if (lane == 0) ms.warp_sum[warp] = sum;
    __syncthreads();
    uint32_t before = lane < warps ? ms.warp_sum[lane] : 0u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(kFull, before, o);
      if (lane >= o) before += y;
    }
    before = __shfl_sync(kFull, before, warp) - sum;  // entries above this warp's run
    if (before < need && before + sum >= need) {      // one warp: the bin is in its run
      for (int b0 = top;; b0 -= 128) {
        const int b = b0 - 4 * lane - 4;
        const uint4 x = b >= 0 ? bins4(b) : make_uint4(0, 0, 0, 0);
        uint32_t incl = x.x + x.y + x.z + x.w;
        const uint32_t own = incl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(kFull, incl, o);
          if (lane >= o) incl += y;
        }
        uint32_t above = before + incl - own;
        if (above < need && above + own >= need) {
          const uint32_t y[4] = {x.w, x.z, x.y, x.x};
          int at = b + 3;
#pragma unroll
          for (int q = 0; q < 3; ++q)
            if (at == b + 3 - q && above + y[q] < need) {
              above += y[q];
              --at;
            }
          ms.bin = (uint32_t)at;
          ms.above = above;
        }
        before += __shfl_sync(kFull, incl, 31);
        if (before >= need || b0 <= 128) break;
      }
    }
    __syncthreads();
    need -= ms.above;
    t = (t << bits) | ms.bin;
  }

  // t is the budget-th largest key; `need` of the slots that equal it stay.  Each
  // warp counts its own run of the segment, in whole groups of 32.
  const int run = (count + T - 1) / T * 32, w0 = min(count, warp * run), w1 = min(count, w0 + run);
  const int below = a.budget - s0;  // the segment's slots below it are below budget
  uint32_t gt = 0, eq = 0, gt_b = 0, eq_b = 0;
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
  if (tid < 4) ms.count[tid] = 0;
  __syncthreads();
  if (lane == 0) {
    ms.warp_gt[warp] = gt;
    ms.warp_eq[warp] = eq;
    atomicAdd(&ms.count[0], gt);
    atomicAdd(&ms.count[1], eq);
    atomicAdd(&ms.count[2], gt_b);
    atomicAdd(&ms.count[3], eq_b);
  }
  __syncthreads();
  cluster_sync();
  uint32_t g0 = __reduce_add_sync(kFull, lane < warp ? ms.warp_gt[lane] : 0u);
  uint32_t e0 = __reduce_add_sync(kFull, lane < warp ? ms.warp_eq[lane] : 0u);
  uint32_t gb = ms.count[2], eb = ms.count[3];
  for (int o = 0; o < cs; ++o) {
    if (o == part) continue;
    const uint32_t at = dsmem_addr(ms.count, (uint32_t)o);
    if (o < part) {
      g0 += dsmem_ld_u32(at);
      e0 += dsmem_ld_u32(at + 4);
    }
    gb += dsmem_ld_u32(at + 8);
    eb += dsmem_ld_u32(at + 12);
  }
  const uint32_t kb = gb + min(eb, need);  // kept slots below budget
  int2 *moves = a.moves + (size_t)unit * a.max_moves;
  const uint32_t lt = (1u << lane) - 1u;
  for (int i = w0 + lane; i - lane < w1; i += 32) {
    const bool on = i < w1;
    const uint32_t k = on ? key_at(i) : 0u;
    const uint32_t mg = __ballot_sync(kFull, on && k > t), me = __ballot_sync(kFull, on && k == t);
    const uint32_t ge = g0 + __popc(mg & lt), ee = e0 + __popc(me & lt);
    const bool keep = on && (k > t || (k == t && ee < need));
    const uint32_t before = ge + min(ee, need);
    const int s = s0 + i;
    if (on && i < below) {
      if (!keep) {
        moves[s - (int)before].y = s;
      } else if (a.copy) {
        acc_out[s] = acc[s];
        pos_out[s] = pos[s];
      }
    } else if (keep) {
      moves[before - kb].x = s;
    }
    g0 += __popc(mg);
    e0 += __popc(me);
  }
  cluster_sync();  // the list is whole; no CTA reads another's shared memory any more

  // the moves: a warp has the rows of kMovesWarp of them in flight, lanes 0-15
  // on keys and 16-31 on values (16 bytes each; with D = 64 half of them)
  const int n_moves = a.budget - (int)kb, half = lane >> 4, sub = lane & 15;
  const bool row_on = sub < c.D / 8;
  uint16_t *pool = half ? c.v : c.k;
  for (int m0 = (part * warps + warp) * kMovesWarp; m0 < n_moves; m0 += cs * warps * kMovesWarp) {
    int64_t src = -1, dst = -1;
    if (lane < kMovesWarp && m0 + lane < n_moves) {
      const int2 mv = __ldcg(&moves[m0 + lane]);
      const int ps = paged_page(c, r, mv.x, a.status), pd = paged_page(c, r, mv.y, a.status);
      if (ps >= 0 && pd >= 0) {
        src = paged_row(c, ps, mv.x, g);
        dst = paged_row(c, pd, mv.y, g);
      }
      acc_out[mv.y] = acc[mv.x];
      pos_out[mv.y] = pos[mv.x];
    }
    uint4 v[kMovesWarp];
    int64_t to[kMovesWarp];
#pragma unroll
    for (int x = 0; x < kMovesWarp; ++x) {
      const int64_t from = __shfl_sync(kFull, src, x);
      to[x] = __shfl_sync(kFull, dst, x);
      if (to[x] >= 0 && row_on) v[x] = *reinterpret_cast<const uint4 *>(pool + from + sub * 8);
    }
#pragma unroll
    for (int x = 0; x < kMovesWarp; ++x)
      if (to[x] >= 0 && row_on) *reinterpret_cast<uint4 *>(pool + to[x] + sub * 8) = v[x];
  }
  leave();
}

}  // namespace

size_t paged_evict_workspace_bytes(int B, int Hkv, int64_t cap) {
  // counters, at the same place for every size; at most cap / 2 moves: targets lie below budget, sources past it
  return kMaxRequests * sizeof(uint32_t) + (size_t)B * Hkv * (size_t)(cap / 2) * sizeof(int2);
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
  a.moves = reinterpret_cast<int2 *>(static_cast<char *>(ws) + kMaxRequests * sizeof(uint32_t));
  a.copy = acc_out != acc || pos_out != pos;
  a.status = status;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return BASTION_ERR_LAUNCH;
  // CTAs of a unit: as many as the device has room for at one CTA per SM, with 2,048 slots each at least; more
  // where their keys would not fit
  int cs = 1;
  while (cs < 8 && ((units * cs * 2 <= sms && c.cap >= 4096 * cs) || c.cap > cs * kKeysMax)) cs *= 2;
  const int seg = ((c.cap + cs - 1) / cs + 3) & ~3;
  const bool in_smem = seg <= kKeysMax;
  const int T = seg <= 4096 ? 256 : seg <= 8192 ? 512 : 1024;
  const size_t smem = (size_t)kHist * 4 + (in_smem ? (size_t)seg * 4 : 0);
  auto kernel = in_smem ? paged_evict_kernel<true> : paged_evict_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)((kHist + kKeysMax) * 4));
  if (e == cudaSuccess)
    e = launch_cluster_pdl(kernel, dim3((unsigned)(units * cs)), dim3((unsigned)T), smem, stream, cs, c, a, cs);
  return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? BASTION_OK : BASTION_ERR_LAUNCH;
}

}  // namespace bastion
