// Eviction from the paged cache by accumulated attention weight.
//
// Two launches.  The selection, one CTA per (request, KV head): slot j's key is
// its weight as an order-preserving 32-bit integer (the protected slots' above
// all weights); a radix select finds the budget-th largest key t and how many
// slots that tie with it stay, and one more pass in slot order, with running
// counts, marks the kept slots and lists the moves.  The i-th hole (a slot
// below budget that is not kept) takes the i-th kept slot at or past budget:
//   K(s) = kept slots before s = #(key > t before s) + min(#(key == t before s), ties that stay)
//   hole index of s < budget: s - K(s);   source index of s >= budget: K(s) - K(budget)
// so both lists come from one prefix count.  Then the moves: K and V rows,
// weights and positions.  Sources lie at or past budget and targets below it,
// so no move reads what another writes.
#include "paged.cuh"

namespace bastion {

namespace {

constexpr int kSel = 1024;  // threads of the selection
constexpr int kWarps = kSel / 32;
constexpr uint32_t kSafe = 0xffffffffu;  // key of a protected slot
constexpr int kBins = 2048;

struct EvictArgs {
  const int32_t *seq_len, *n_seen;
  const float *acc;
  const int32_t *pos;
  int budget, n_sink, n_recent, max_moves;
  int32_t *seq_len_out;
  float *acc_out;
  int32_t *pos_out;
  int32_t *n_moves;   // [units]
  int2 *moves;        // [units, max_moves] (source slot, target slot)
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

// Bin that holds the need-th largest entry of a histogram (bins from the top),
// and how many lie in the bins above it.  Every thread gets the answer.
__device__ __forceinline__ void find_bin(const uint32_t *hist, uint32_t need, uint32_t *scratch, int &bin,
                                         uint32_t &above) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t a = hist[kBins - 1 - 2 * tid], b = hist[kBins - 2 - 2 * tid];
  uint32_t x = a + b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  if (warp == 0) {
    uint32_t t = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(kFull, t, o);
      if (lane >= o) t += y;
    }
    scratch[lane] = t;
  }
  __syncthreads();
  const uint32_t incl = x + (warp ? scratch[warp - 1] : 0u), before = incl - a - b;
  if (before < need && incl >= need) {
    if (before + a >= need) {
      scratch[32] = (uint32_t)(kBins - 1 - 2 * tid);
      scratch[33] = before;
    } else {
      scratch[32] = (uint32_t)(kBins - 2 - 2 * tid);
      scratch[33] = before + a;
    }
  }
  __syncthreads();
  bin = (int)scratch[32];
  above = scratch[33];
}

__global__ void __launch_bounds__(kSel) paged_evict_select_kernel(Paged c, EvictArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int unit = blockIdx.x, r = unit / c.Hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = paged_len(c, a.seq_len, r, a.status);
  const size_t base = (size_t)unit * c.cap;
  const float *acc = a.acc + base;
  const int32_t *pos = a.pos + base;
  float *acc_out = a.acc_out + base;
  int32_t *pos_out = a.pos_out + base;
  if (n <= a.budget) {
    if (tid == 0) a.n_moves[unit] = 0;
    for (int s = tid; s < n; s += kSel) {
      acc_out[s] = acc[s];
      pos_out[s] = pos[s];
    }
    return;
  }
  const int64_t recent = (int64_t)a.n_seen[r] - a.n_recent;
  __shared__ uint32_t hist[kBins], scratch[34], s_gt[kWarps], s_eq[kWarps], s_below[2];
  bool nan = false;
  // radix select, 11 + 11 + 10 bits from the top
  uint32_t prefix = 0, need = (uint32_t)a.budget;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    for (int i = tid; i < kBins; i += kSel) hist[i] = 0;
    __syncthreads();
    for (int s = tid; s < n; s += kSel) {
      const uint32_t k = slot_key(acc[s], pos[s], a.n_sink, recent, nan);
      if (pass == 0 || (k >> (shift + bits)) == prefix) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
    }
    __syncthreads();
    int bin;
    uint32_t above;
    find_bin(hist, need, scratch, bin, above);
    need -= above;
    prefix = (prefix << bits) | (uint32_t)bin;
    __syncthreads();
  }
  if (nan) atomicOr(&a.status[r], BASTION_STATUS_NONFINITE);
  const uint32_t t = prefix;  // the budget-th largest key; `need` of the slots that equal it stay
  // each warp counts its own run of slots, in whole groups of 32
  const int run = ((n + kSel - 1) / kSel) * 32, s0 = warp * run, s1 = min(n, s0 + run);
  if (tid < 2) s_below[tid] = 0;
  __syncthreads();
  uint32_t gt = 0, eq = 0, gt_b = 0, eq_b = 0;  // *_b: below budget
  for (int s = s0 + lane; s < s1; s += 32) {
    const uint32_t k = slot_key(acc[s], pos[s], a.n_sink, recent, nan);
    gt += k > t;
    eq += k == t;
    if (s < a.budget) {
      gt_b += k > t;
      eq_b += k == t;
    }
  }
  gt = __reduce_add_sync(kFull, gt);
  eq = __reduce_add_sync(kFull, eq);
  gt_b = __reduce_add_sync(kFull, gt_b);
  eq_b = __reduce_add_sync(kFull, eq_b);
  if (lane == 0) {
    s_gt[warp] = gt;
    s_eq[warp] = eq;
    atomicAdd(&s_below[0], gt_b);
    atomicAdd(&s_below[1], eq_b);
  }
  __syncthreads();
  uint32_t g0 = lane < warp ? s_gt[lane] : 0u, e0 = lane < warp ? s_eq[lane] : 0u;
  g0 = __reduce_add_sync(kFull, g0);
  e0 = __reduce_add_sync(kFull, e0);
  const uint32_t kb = s_below[0] + min(s_below[1], need);  // kept slots below budget
  if (tid == 0) a.n_moves[unit] = a.budget - (int)kb;
  int2 *moves = a.moves + (size_t)unit * a.max_moves;
  const uint32_t lt = (1u << lane) - 1u;
  for (int s = s0 + lane; s - lane < s1; s += 32) {
    const bool on = s < s1;
    float w = 0.f;
    int p = 0;
    uint32_t k = 0;
    if (on) {
      w = acc[s];
      p = pos[s];
      k = slot_key(w, p, a.n_sink, recent, nan);
    }
    const uint32_t mg = __ballot_sync(kFull, on && k > t), me = __ballot_sync(kFull, on && k == t);
    const uint32_t ge = g0 + __popc(mg & lt), ee = e0 + __popc(me & lt);
    const bool keep = on && (k > t || (k == t && ee < need));
    const uint32_t before = ge + min(ee, need);
    if (on && s < a.budget) {
      if (keep) {
        acc_out[s] = w;
        pos_out[s] = p;
      } else {
        moves[s - (int)before].y = s;
      }
    } else if (keep) {
      moves[before - kb].x = s;
    }
    g0 += __popc(mg);
    e0 += __popc(me);
  }
}

// Row vectors of 16 bytes; a move is 2 * D / 8 of them.
__global__ void __launch_bounds__(256) paged_evict_move_kernel(Paged c, EvictArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int unit = blockIdx.y, r = unit / c.Hkv, g = unit % c.Hkv, tid = threadIdx.x;
  if (blockIdx.x == 0 && g == 0 && tid == 0) {
    const int n = a.seq_len[r];
    a.seq_len_out[r] = n > a.budget ? a.budget : n;
  }
  const int n = a.n_moves[unit];
  const int2 *moves = a.moves + (size_t)unit * a.max_moves;
  const int dv = c.D >> 3, sub = tid % dv, per = 256 / dv;  // moves of one sweep of the CTA
  const size_t base = (size_t)unit * c.cap;
  for (int i = blockIdx.x * per + tid / dv; i < n; i += gridDim.x * per) {
    const int2 mv = moves[i];
    const int ps = paged_page(c, r, mv.x, a.status), pd = paged_page(c, r, mv.y, a.status);
    if (ps >= 0 && pd >= 0) {
      const int64_t src = paged_row(c, ps, mv.x, g) + sub * 8, dst = paged_row(c, pd, mv.y, g) + sub * 8;
      const uint4 kk = *reinterpret_cast<const uint4 *>(c.k + src);
      const uint4 vv = *reinterpret_cast<const uint4 *>(c.v + src);
      *reinterpret_cast<uint4 *>(c.k + dst) = kk;
      *reinterpret_cast<uint4 *>(c.v + dst) = vv;
    }
    if (sub == 0) a.acc_out[base + mv.y] = a.acc[base + mv.x];
    if (sub == 1) a.pos_out[base + mv.y] = a.pos[base + mv.x];
  }
}

}  // namespace

size_t paged_evict_workspace_bytes(int B, int Hkv, int64_t cap) {
  // at most cap / 2 moves: targets lie below budget, sources at or past it
  return (((size_t)B * Hkv * sizeof(int32_t) + 255) & ~(size_t)255) + (size_t)B * Hkv * (size_t)(cap / 2) * sizeof(int2);
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
  a.n_moves = static_cast<int32_t *>(ws);
  a.moves = reinterpret_cast<int2 *>(static_cast<char *>(ws) + (((size_t)units * sizeof(int32_t) + 255) & ~(size_t)255));
  a.status = status;
  cudaError_t e = launch_pdl(paged_evict_select_kernel, dim3((unsigned)units), dim3(kSel), 0, stream, c, a);
  if (e == cudaSuccess) {
    const int most = budget < c.cap - budget ? budget : (c.cap > budget ? c.cap - budget : 0);
    const int per = 256 / (c.D / 8);
    int gx = (most + per - 1) / per;
    gx = gx < 1 ? 1 : gx > 64 ? 64 : gx;
    e = launch_pdl(paged_evict_move_kernel, dim3((unsigned)gx, (unsigned)units), dim3(256), 0, stream, c, a);
  }
  return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? BASTION_OK : BASTION_ERR_LAUNCH;
}

}  // namespace bastion
