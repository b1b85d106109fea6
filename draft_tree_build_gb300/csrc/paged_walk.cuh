// How the batch's 128-key tiles are dealt to the CTAs of a paged attention
// launch, and how a CTA walks its share.  Plain index arithmetic, for the host
// as well.
#pragma once

#include <cuda_runtime.h>

namespace bastion {

constexpr int kTileKeys = 128;

// A CTA's tiles, one after the other: tile t of the unit (request r, KV head g).
// kUniform: all lanes of a warp walk together, and the compiler is told so.
template <bool kUniform>
struct Walk {
  const int2 *list;  // the requests that have tiles: number and length
  int li, r, n, tiles, g, t, left;
  bool first;  // the first tile of its segment
  static __host__ __device__ __forceinline__ int uniform(int x) {
#ifdef __CUDA_ARCH__
    if (kUniform) return __shfl_sync(0xffffffffu, x, 0);
#endif
    return x;
  }
  __host__ __device__ __forceinline__ void load() {
    const int2 e = list[li];
    r = uniform(e.x);
    n = uniform(e.y);
    tiles = (n + kTileKeys - 1) / kTileKeys;
  }
  __host__ __device__ __forceinline__ void start(const int2 *l, int index, int off, int count) {
    list = l;
    li = index;
    left = count;
    first = true;
    if (left > 0) {
      load();
      g = off / tiles;
      t = off - g * tiles;
    }
  }
  __host__ __device__ __forceinline__ void step(int heads) {
    first = false;
    --left;
    if (++t == tiles) {
      t = 0;
      first = true;
      if (++g == heads) {
        g = 0;
        ++li;
        if (left > 0) load();
      }
    }
  }
  __host__ __device__ __forceinline__ bool last() const { return t == tiles - 1 || left == 1; }
};

// The batch's tiles in equal shares: `big` CTAs of quot + 1 tiles, then shares
// of quot.  A boundary moves to a unit's begin or end where cutting the unit
// costs more in the join (1.4 us) than it saves: from anywhere in a unit of at
// most kWhole tiles to the nearer end, and from within kSnap tiles of the ends
// of a longer one.  Shares may become empty.  (8 units of 3 tiles: 6.6 us whole,
// 9.9 us cut; 8 of 8 tiles: 8.0 us cut.)
constexpr int kWhole = 4, kSnap = 1;
struct Shares {
  int n, quot, big;
  __host__ __device__ __forceinline__ int begin(int cta) const { return cta * quot + (cta < big ? cta : big); }
  __host__ __device__ __forceinline__ int owner(int f) const {  // the share of tile f, before boundaries move
    const int edge = big * (quot + 1);
    return f < edge ? f / (quot + 1) : big + (f - edge) / quot;
  }
  // Where boundary f moves to; unit of t tiles, off = f - its begin.
  static __host__ __device__ __forceinline__ int moved(int f, int off, int t) {
    if (t <= kWhole) return 2 * off <= t ? f - off : f - off + t;
    return off <= kSnap ? f - off : t - off <= kSnap ? f - off + t : f;
  }
  // The first and last CTA of a cut unit of tiles [u0, u1).
  __host__ __device__ __forceinline__ int first_cta(int u0) const { return owner(u0 + kSnap); }
  __host__ __device__ __forceinline__ int last_cta(int u1) const { return owner(u1 - kSnap - 1); }
};

// Gives up at tile w: every unit from the current segment to the share's end,
// in order.  None of them is written by this CTA, nor by one that shares it,
// which never sees all of its parts arrive.
template <bool kUniform, typename F>
__host__ __device__ __forceinline__ void give_up(Walk<kUniform> &w, int heads, F unit) {
  bool current = true;
#pragma unroll 1
  for (; w.left > 0; w.step(heads)) {
    if (current || w.first) unit(w.r, w.g);
    current = false;
  }
}

}  // namespace bastion
