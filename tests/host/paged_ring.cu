// Host program: the warps of a shared-prefix attention CTA as threads that wait on
// barriers with phases and parities as the GPU's have, in the order of
// paged_ring.cuh, each held up in turn before its first step.  Every share has to
// come to its end, and no copy may land in a stage that is still read.  With the
// argument "shared" the value warp waits for the first phase of the keys' own
// barrier instead, which the model has to find stuck.  Prints the first difference
// and returns 1, else 0.
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <cstring>
#include <functional>
#include <mutex>
#include <thread>
#include <vector>

#include "paged_ring.cuh"

using namespace bastion;

namespace {

std::mutex mu;
std::condition_variable cv;
bool stuck = false;  // a wait has run out
int limit_ms = 20000, wrong = 0;

struct Bar {
  int count = 1, arrived = 0;
  unsigned phase = 0;  // phases complete
  void arrive() {
    std::lock_guard<std::mutex> l(mu);
    if (++arrived == count) {
      arrived = 0;
      ++phase;
    }
    cv.notify_all();
  }
  // The phase with this parity has completed: what the hardware can tell of it.
  bool wait(unsigned parity) {
    std::unique_lock<std::mutex> l(mu);
    const bool ok = cv.wait_for(l, std::chrono::milliseconds(limit_ms), [&] { return stuck || (phase & 1u) != parity; });
    if (!ok) stuck = true;
    cv.notify_all();
    return !stuck;
  }
};

template <int kStages>
struct Cta {
  Bar full[kStages], empty[kStages], begun, s_full[2], p_full[2];
  int holds[kStages];  // the place whose tile a stage holds
  bool shared;         // the mistake
  struct Bars {
    Cta &c;
    bool wait_full(int stage, unsigned parity) { return c.full[stage].wait(parity); }
    bool wait_empty(int stage, unsigned parity) { return c.empty[stage].wait(parity); }
    bool wait_begun() { return c.shared ? c.full[0].wait(0) : c.begun.wait(0); }
    void arrive_begun() { c.begun.arrive(); }
  };
  void look(int x) {  // a product reads place x
    std::lock_guard<std::mutex> l(mu);
    if (holds[Ring<kStages>::stage(x)] != x) ++wrong;
  }
  void fill(int odd, int tiles) {
    Bars b{*this};
    int issued = 0;
    for (; issued < tiles; ++issued) {
      const int x = 2 * issued + odd, at = Ring<kStages>::stage(x);
      if (!Ring<kStages>::before(b, x)) break;
      {
        std::lock_guard<std::mutex> l(mu);
        holds[at] = x;
      }
      full[at].arrive();
    }
    if (odd == 0 && issued > 0 && issued == tiles) Ring<kStages>::after_keys(b, issued);
  }
  void products(int tiles) {  // scores two tiles ahead of the values
    int s = 0;
    auto scores = [&] {
      const int x = 2 * s, at = Ring<kStages>::stage(x);
      if (!full[at].wait(Ring<kStages>::full_parity(x))) return false;
      look(x);
      s_full[s & 1].arrive();
      empty[at].arrive();
      ++s;
      return true;
    };
    bool ok = true;
    for (int y = 0; y < 2; ++y) ok = ok && (s == tiles || scores());
    for (int p = 0; ok && p < tiles; ++p) {
      const int x = 2 * p + 1, at = Ring<kStages>::stage(x);
      ok = p_full[p & 1].wait((unsigned)(p >> 1) & 1u) && full[at].wait(Ring<kStages>::full_parity(x));
      if (!ok) break;
      look(x);
      empty[at].arrive();
      ok = s == tiles || scores();
    }
  }
  void weights(int wg, int tiles) {
    for (int i = wg, n = 0; i < tiles; i += 2, ++n) {
      if (!s_full[wg].wait((unsigned)n & 1u)) return;
      p_full[wg].arrive();
    }
  }
};

template <int kStages>
bool run(int tiles, int late, bool shared) {  // the thread `late` begins when the others have nothing left to do
  Cta<kStages> c;
  c.shared = shared;
  stuck = false;
  wrong = 0;
  for (int &x : c.holds) x = -1;
  const std::vector<std::function<void()>> roles = {[&] { c.fill(0, tiles); }, [&] { c.fill(1, tiles); }, [&] { c.products(tiles); },
                                                    [&] { c.weights(0, tiles); }, [&] { c.weights(1, tiles); }};
  std::vector<std::thread> threads;
  for (int i = 0; i < (int)roles.size(); ++i)
    threads.emplace_back([&, i] {
      if (i == late) std::this_thread::sleep_for(std::chrono::milliseconds(15));
      roles[i]();
    });
  for (auto &t : threads) t.join();
  if (wrong) printf("%d stages, %d tiles, thread %d late: %d tiles read that were not there\n", kStages, tiles, late, wrong);
  else if (stuck) printf("%d stages, %d tiles, thread %d late: stuck\n", kStages, tiles, late);
  return !stuck && !wrong;
}

}  // namespace

int main(int argc, char **argv) {
  bool ok = true;
  if (argc > 1 && !strcmp(argv[1], "shared")) {
    limit_ms = 1000;
    for (int tiles = 2; tiles <= 5; ++tiles) {
      ok &= run<4>(tiles, 1, true);
      ok &= run<8>(tiles, 1, true);
    }
    return ok ? 0 : 1;
  }
  for (int tiles = 1; tiles <= 20; ++tiles)
    for (int late = -1; late < 5; ++late) {
      ok &= run<4>(tiles, late, false);
      ok &= run<8>(tiles, late, false);
    }
  return ok ? 0 : 1;
}
