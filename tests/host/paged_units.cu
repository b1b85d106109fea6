// Host program: deals random batches of shared prefixes to CTAs as
// the shared-prefix attention kernel does, and looks for every row's parts as its
// join does: each key tile is there once, and no place is written twice.  Prints
// the first difference and returns 1, else 0.
#include <cstdio>
#include <map>
#include <random>
#include <set>
#include <tuple>
#include <vector>

#include "paged_units.cuh"

using namespace bastion;

int main() {
  std::mt19937 rng(1);
  auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
  long cut = 0, whole_units = 0, fine = 0;
  for (int trial = 0; trial < 6000; ++trial) {
    const int heads = pick(1, 4), grid = pick(1, 40), nb = pick(1, 9), longest = pick(0, 3) ? 1200 : 9000;
    const bool single = pick(0, 3) == 0;
    std::vector<UnitEntry> list;
    int total = 0, widest = 1;
    for (int e = pick(1, 10); e > 0; --e) {
      UnitEntry u;
      u.who = e | e << 16;
      u.n = single ? pick(1, nb) : pick(1, 5 * nb);
      u.len = pick(1, longest);
      u.at = total;
      const int m = m_tiles_of(u.n, nb);
      if (m > 1) widest = 2;
      total += tiles_of(u.len) * m * heads;
      list.push_back(u);
    }
    const UnitShares sh = UnitShares::of(grid, total, widest);
    fine += sh.fine;
    auto boundary = [&](int cta, int &li, TilePlace &from) {  // where CTA cta's share begins
      const int f = sh.begin(cta);
      li = (int)list.size();
      from = TilePlace{0, 0, 0, 0};
      if (f == total) return f;
      li = 0;
      while (li + 1 < (int)list.size() && list[li + 1].at <= f) ++li;
      const int tiles = tiles_of(list[li].len), m = m_tiles_of(list[li].n, nb);
      from = TilePlace::boundary(sh, f - list[li].at, tiles, m);
      const int to = list[li].at + from.off;
      if (from.off == tiles * m * heads) {
        ++li;
        from = TilePlace{0, 0, 0, 0};
      }
      return to;
    };
    using Key = std::tuple<int, int, int, int>;  // whole: plane, entry, head, M tile; else -1, slot, plane, 0
    std::map<Key, std::vector<int>> parts;       // the key tiles in it
    for (int cta = 0; cta < sh.n; ++cta) {
      int li, li1;
      TilePlace from, to;
      const int f0 = boundary(cta, li, from), f1 = boundary(cta + 1, li1, to);
      if (f1 < f0) return printf("trial %d: CTA %d ends before it begins\n", trial, cta), 1;
      Units<false> w;
      w.start(list.data(), li, from, f1 - f0, nb);
      int t0 = 0, place = 0, segments = 0;
      std::map<int, std::vector<int>> open;  // plane -> tiles
      for (; w.left > 0; w.step(heads, nb)) {
        if (w.left < 0) return printf("trial %d: CTA %d passes its end\n", trial, cta), 1;
        if (w.first) {
          t0 = w.t;
          place = 0;
          open.clear();
          open[0], open[1];
        }
        if (w.group != w.req || w.tiles != tiles_of(list[w.li].len)) return printf("trial %d: entry\n", trial), 1;
        if (w.ms() == 2) {
          open[0].push_back(w.t);
          open[1].push_back(w.t);
        } else {
          open[place & 1].push_back(w.t);
        }
        ++place;
        if (!w.last()) continue;
        const bool whole = t0 == 0 && w.t == w.tiles - 1;
        for (int plane = 0; plane < 2; ++plane) {
          Key k = whole ? Key(w.ms() == 2 ? 0 : plane, w.li, w.head, 2 * w.pair + (w.ms() == 2 ? plane : 0))
                        : Key(-1, 2 * cta + (t0 == 0), plane, 0);
          if (parts.count(k)) return printf("trial %d: CTA %d writes a place twice\n", trial, cta), 1;
          parts[k] = open[plane];
        }
        ++segments;
      }
      if (w.left != 0) return printf("trial %d: CTA %d passes its end\n", trial, cta), 1;
    }
    for (int e = 0; e < (int)list.size(); ++e)
      for (int h = 0; h < heads; ++h)
        for (int m = 0; m < m_tiles_of(list[e].n, nb); ++m) {
          const int tiles = tiles_of(list[e].len);
          const UnitParts p = UnitParts::of(sh, list[e].at, tiles, m_tiles_of(list[e].n, nb), h, m);
          std::multiset<int> seen;
          for (int x = 0; x < p.ctas; ++x)
            for (int y = 0; y < p.planes; ++y) {
              const Key k = p.whole ? Key(p.planes == 1 ? 0 : y, e, h, m) : Key(-1, p.slot(x), p.plane + y, 0);
              if (!parts.count(k)) return printf("trial %d: entry %d head %d M tile %d: part %d, %d is nowhere\n", trial, e, h, m, x, y), 1;
              seen.insert(parts[k].begin(), parts[k].end());
            }
          (p.whole ? whole_units : cut) += 1;
          bool right = (int)seen.size() == tiles;
          for (int t = 0; t < tiles; ++t) right = right && seen.count(t) == 1;
          if (!right) return printf("trial %d: entry %d head %d M tile %d: %d tiles of %d\n", trial, e, h, m, (int)seen.size(), tiles), 1;
          if (p.count() > 2 * grid) return printf("trial %d: too many parts\n", trial), 1;
        }
  }
  if (cut < 5000 || whole_units < 5000 || fine < 300)
    return printf("%ld %ld %ld\n", cut, whole_units, fine), 1;
  return 0;
}
