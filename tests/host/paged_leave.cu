// Host program: the softmax warps of shared-prefix attention CTAs, each of which stops
// at a tile of its own (a wait that ran out) or not at all, over random batches.  Every
// request with rows that are then not written must have been flagged.  With the
// argument "share" a warp that stops flags its own rows' share of the requests alone,
// which the program has to find wanting.  Prints the first difference and returns
// 1, else 0.
#include <cstdio>
#include <cstring>
#include <random>
#include <set>
#include <vector>

#include "paged_units.cuh"

using namespace bastion;

int main(int argc, char **argv) {
  const bool share = argc > 1 && !strcmp(argv[1], "share");
  std::mt19937 rng(3);
  auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
  long left = 0, alone = 0;
  for (int trial = 0; trial < 3000; ++trial) {
    const int heads = pick(1, 3), grid = pick(1, 20), G = pick(1, 16), nb = 128 / G;
    std::vector<UnitEntry> list;
    int total = 0, widest = 1, req = 0;
    for (int e = 0, n = pick(1, 6); e < n; ++e) {
      UnitEntry u;
      req += pick(0, 2);
      u.n = pick(1, 4 * nb);
      u.who = req | e << 16;
      u.len = pick(1, pick(0, 2) ? 700 : 5000);
      u.at = total;
      const int m = m_tiles_of(u.n, nb);
      if (m > 1) widest = 2;
      total += tiles_of(u.len) * m * heads;
      req += u.n;
      list.push_back(u);
    }
    const UnitShares sh = UnitShares::of(grid, total, widest);
    auto boundary = [&](int cta, int &li, TilePlace &from) {
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
    const int cta = pick(0, sh.n - 1);
    int li, li1;
    TilePlace from, to;
    const int f0 = boundary(cta, li, from), f1 = boundary(cta + 1, li1, to);
    std::set<int> unwritten, told;
    int steps = 0;
    {
      Units<false> w;
      w.start(list.data(), li, from, f1 - f0, nb);
      for (; w.left > 0; w.step(heads, nb)) ++steps;
    }
    const int stopping = pick(0, 2) ? 0xff : 1 << pick(0, 7);  // which warps may stop
    for (int warp = 0; warp < 8; ++warp) {
      const int wg = warp >> 2, quad = warp & 3;
      const int stop = steps > 0 && (stopping >> warp & 1) ? pick(0, steps - 1) : steps;
      Units<false> w;
      w.start(list.data(), li, from, f1 - f0, nb);
      int par = 0, m = 0, at = 0;
      // as the kernel has it: parts are written at a segment's end, by both warpgroups, rows of this quad
      for (; w.left > 0 && at < stop; w.step(heads, nb), ++at) {
        if (w.first) m = w.ms() == 2 ? wg ^ par : 0;
        if (w.ms() == 1) par ^= 1;
      }
      const Units<false> here = w;
      bool current = !w.first;  // the segment that it is in the middle of keeps its M tile
      for (; w.left > 0; w.step(heads, nb)) {
        if (w.first) {
          m = w.ms() == 2 ? wg ^ par : 0;
          current = true;
        }
        if (current) {
          const int rows = imin(nb, w.n - (2 * w.pair + m) * nb) * G;
          for (int row = quad * 32; row < quad * 32 + 32 && row < rows; ++row) {
            unwritten.insert(w.req + (2 * w.pair + m) * nb + row / G);
            ++left;
          }
          current = false;
        }
        if (w.ms() == 1) par ^= 1;
      }
      if (here.left == 0) continue;
      alone += stopping != 0xff;
      for (int k = share ? quad : 0; k < (share ? quad + 1 : 4); ++k)
        for (int lane = 0; lane < 32; ++lane) {
          const int row = 32 * k + lane;
          for (Units<false> v = here; v.left > 0; v.step(heads, nb))
            for (int b = v.req + row; b < v.req + v.n; b += 128) told.insert(b);
        }
    }
    for (int b : unwritten)
      if (!told.count(b)) return printf("trial %d: CTA %d leaves rows of request %d, which nobody is told\n", trial, cta, b), 1;
    for (int b : told)  // and of the batch alone
      if (b < 0 || b >= req) return printf("trial %d: request %d of %d\n", trial, b, req), 1;
  }
  if (left < 10000 || alone < 300) return printf("%ld %ld\n", left, alone), 1;
  return 0;
}
