// How the tiles of a shared-prefix attention are dealt to the CTAs of a launch,
// how a CTA walks its share, and how the join finds a unit's parts.  Plain index
// arithmetic, for the host as well.
#pragma once

#include <cuda_runtime.h>

#include "paged_walk.cuh"

namespace bastion {

// A list entry: a group of requests and its prefix.
struct UnitEntry {
  int32_t who;  // the first request, and the group's number << 16
  int32_t n;    // requests
  int32_t len;  // slots
  int32_t at;   // first work item
};

__host__ __device__ __forceinline__ int imin(int a, int b) { return a < b ? a : b; }
__host__ __device__ __forceinline__ int tiles_of(int len) { return (len + kTileKeys - 1) / kTileKeys; }
__host__ __device__ __forceinline__ int m_tiles_of(int n, int nb) { return (n + nb - 1) / nb; }

// A unit is an entry, a KV head and a pair of M tiles of nb requests (or the odd one left);
// a tile of it is 128 keys, which weigh as many work items as it has M tiles.  The
// items are in order entry, head, pair, tile, and every CTA takes an equal share
// of them.  A boundary moves to the begin of its tile, and, where shares are of
// kWhole tiles or more, to a unit's begin or end where cutting costs more than it
// saves: within a unit of at most kWhole tiles, and within kSnap tiles of the ends
// of a longer one.  (Smaller shares are latency: 24 tiles of 8 units 15.4 us whole, 12.2 cut.)
struct UnitShares {
  int n, quot, big;
  bool fine;  // nothing but tiles holds boundaries
  // widest: the items of the heaviest tile, so that no two boundaries fall into one tile
  static __host__ __device__ __forceinline__ UnitShares of(int ctas, int total, int widest) {
    UnitShares s;
    s.n = total == 0 ? 0 : imin(ctas, total >= widest ? total >> (widest - 1) : 1);
    s.quot = s.n > 0 ? total / s.n : 0;
    s.big = total - s.quot * s.n;
    s.fine = s.quot < kWhole * widest;
    return s;
  }
  __host__ __device__ __forceinline__ int begin(int cta) const { return cta * quot + imin(cta, big); }
  __host__ __device__ __forceinline__ int owner(int item) const {  // before boundaries move
    const int edge = big * (quot + 1);
    return item < edge ? item / (quot + 1) : big + (item - edge) / quot;
  }
  // The tile that a boundary `off` items into a unit moves to.
  __host__ __device__ __forceinline__ int moved(int off, int tiles, int weight) const {
    if (fine) return off >> (weight - 1);
    if (tiles <= kWhole) return 2 * off <= tiles * weight ? 0 : tiles;
    const int t = off >> (weight - 1);
    return t <= kSnap ? 0 : tiles - t <= kSnap ? tiles : t;
  }
  // Whether a unit may be cut, and the CTAs of one that may, items [u0, u1): those with its first and its last tile.
  __host__ __device__ __forceinline__ bool cuts(int tiles) const { return fine || tiles > kWhole; }
  __host__ __device__ __forceinline__ int first_cta(int u0, int weight) const {
    return owner(u0 + (fine ? 1 : kSnap + 1) * weight - 1);
  }
  __host__ __device__ __forceinline__ int last_cta(int u1, int weight) const {
    return owner(u1 - (fine ? 0 : kSnap) * weight - 1);
  }
};

// A tile of an entry, `off` items into it.
struct TilePlace {
  int head, pair, t, off;
  // Where a boundary `off` items into the entry falls.
  static __host__ __device__ __forceinline__ TilePlace boundary(const UnitShares &s, int off, int tiles, int m_tiles) {
    const int per_head = tiles * m_tiles;
    TilePlace p;
    p.head = off / per_head;
    const int rest = off - p.head * per_head;
    p.pair = rest / (2 * tiles);
    const int weight = imin(2, m_tiles - 2 * p.pair);
    p.t = s.moved(rest - p.pair * 2 * tiles, tiles, weight);
    p.off = p.head * per_head + p.pair * 2 * tiles + weight * p.t;
    if (p.t == tiles) {  // the next unit's begin
      p.t = 0;
      if (2 * ++p.pair >= m_tiles) {
        p.pair = 0;
        ++p.head;
      }
    }
    return p;
  }
};

// A CTA's tiles, one after the other.  kUniform: all lanes of a warp walk together,
// and the compiler is told so.
template <bool kUniform>
struct Units {
  const UnitEntry *list;
  int li, group, req, n, len, tiles, m_tiles, head, pair, t, left;
  bool first;  // the first tile of its segment
  static __host__ __device__ __forceinline__ int uniform(int x) {
#ifdef __CUDA_ARCH__
    if (kUniform) return __shfl_sync(0xffffffffu, x, 0);
#endif
    return x;
  }
  __host__ __device__ __forceinline__ void load(int nb) {
    const UnitEntry e = list[li];
    const int who = uniform(e.who);
    group = who >> 16;
    req = who & 0xffff;
    n = uniform(e.n);
    len = uniform(e.len);
    tiles = tiles_of(len);
    m_tiles = m_tiles_of(n, nb);
  }
  __host__ __device__ __forceinline__ int ms() const { return imin(2, m_tiles - 2 * pair); }  // M tiles of the unit
  // From that tile of entry `index` on, `count` items in all.
  __host__ __device__ __forceinline__ void start(const UnitEntry *l, int index, TilePlace from, int count, int nb) {
    list = l;
    li = index;
    left = count;
    first = true;
    head = from.head;
    pair = from.pair;
    t = from.t;
    if (left > 0) load(nb);
  }
  __host__ __device__ __forceinline__ void step(int heads, int nb) {
    first = false;
    left -= ms();
    if (++t == tiles) {
      t = 0;
      first = true;
      if (++pair * 2 >= m_tiles) {
        pair = 0;
        if (++head == heads) {
          head = 0;
          ++li;
          if (left > 0) load(nb);
        }
      }
    }
  }
  __host__ __device__ __forceinline__ bool last() const { return t == tiles - 1 || left == ms(); }
};

// A unit's parts as the join sees them.  Each of its CTAs leaves one for every M
// tile, or two for a unit of one M tile, whose key tiles the two warpgroups take
// in turn.  A unit that one CTA finishes keeps its parts by request, the others
// in the CTAs' slots: the last segment of its first CTA, the first of the others.
struct UnitParts {
  bool whole;
  int cta, ctas, planes, plane;  // the first CTA, how many, parts of each and the first of them
  static __host__ __device__ __forceinline__ UnitParts of(const UnitShares &s, int at, int tiles, int m_tiles, int head,
                                                          int m) {
    const int pair = m >> 1, weight = imin(2, m_tiles - 2 * pair);
    const int u0 = at + (head * m_tiles + 2 * pair) * tiles, u1 = u0 + tiles * weight;
    UnitParts p;
    p.cta = s.cuts(tiles) ? s.first_cta(u0, weight) : 0;
    p.ctas = s.cuts(tiles) ? s.last_cta(u1, weight) - p.cta + 1 : 1;
    p.whole = p.ctas <= 1;
    p.planes = weight == 2 ? 1 : 2;
    p.plane = weight == 2 ? m & 1 : 0;
    return p;
  }
  __host__ __device__ __forceinline__ int count() const { return ctas * planes; }
  __host__ __device__ __forceinline__ int slot(int x) const { return 2 * (cta + x) + (x == 0 ? 1 : 0); }  // of CTA x of them
};

}  // namespace bastion
