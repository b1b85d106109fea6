// Host program: deals random batches to CTAs as the paged attention kernel
// does, lets some CTAs give up at a random tile, and compares the units that
// they report with the units that then lack a part.  Prints the first
// difference and returns 1, else 0.
#include <cstdio>
#include <random>
#include <set>
#include <utility>
#include <vector>

#include "paged_walk.cuh"

using namespace bastion;

int main() {
  std::mt19937 rng(1);
  auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
  long cut = 0, reported = 0;
  for (int trial = 0; trial < 4000; ++trial) {
    const int B = pick(1, 12), heads = pick(1, 5), grid = pick(1, 40), longest = pick(0, 3) ? 1200 : 9000;
    std::vector<int2> list;
    std::vector<int> first_tile;  // of each request in the list
    int total = 0;
    for (int r = 0; r < B; ++r) {
      const int n = pick(0, 4) ? pick(1, longest) : 0;
      if (n == 0) continue;
      list.push_back(make_int2(r, n));
      first_tile.push_back(total);
      total += (n + kTileKeys - 1) / kTileKeys * heads;
    }
    if (total == 0) continue;
    Shares sh;
    sh.n = grid < total ? grid : total;
    sh.quot = total / sh.n;
    sh.big = total - sh.quot * sh.n;
    auto boundary = [&](int cta, int &li, int &off) {  // where CTA cta's share begins
      const int f = sh.begin(cta);
      li = (int)list.size();
      off = 0;
      if (f == total) return f;
      li = 0;
      while (li + 1 < (int)list.size() && first_tile[li + 1] <= f) ++li;
      const int t = (list[li].y + kTileKeys - 1) / kTileKeys, end = first_tile[li] + t * heads;
      const int to = Shares::moved(f, (f - first_tile[li]) % t, t);
      off = to - first_tile[li];
      if (to == end) {
        ++li;
        off = 0;
      }
      return to;
    };
    using Unit = std::pair<int, int>;  // request, head
    std::vector<std::vector<int>> got(B, std::vector<int>(heads, 0));  // tiles of segments that came to their end
    std::set<Unit> given_up;
    for (int cta = 0; cta < sh.n; ++cta) {
      int li, off, li1, off1;
      const int f0 = boundary(cta, li, off), f1 = boundary(cta + 1, li1, off1), count = f1 - f0;
      Walk<false> w;
      w.start(list.data(), li, off, count);
      int at = count > 0 && pick(0, 3) == 0 ? pick(0, count - 1) : count, done = 0, open = 0;
      for (; w.left > 0 && done < at; w.step(heads), ++done) {
        ++open;
        if (!w.last()) continue;
        got[w.r][w.g] += open;
        open = 0;
      }
      give_up(w, heads, [&](int r, int g) { given_up.insert(Unit(r, g)); });
      if (w.left != 0) return printf("trial %d: CTA %d stops before its end\n", trial, cta), 1;
    }
    for (const int2 &e : list)
      for (int g = 0; g < heads; ++g) {
        const int t = (e.y + kTileKeys - 1) / kTileKeys;
        const bool whole = got[e.x][g] == t, said = given_up.count(Unit(e.x, g)) != 0;
        if (whole == said || got[e.x][g] > t)
          return printf("trial %d: request %d head %d: %d of %d tiles, reported %d\n", trial, e.x, g, got[e.x][g], t, said), 1;
        cut += !whole;
      }
    reported += (long)given_up.size();
  }
  if (cut != reported || cut < 1000) return printf("%ld units cut, %ld reported\n", cut, reported), 1;
  return 0;
}
