// Host-side check of the key tiles' ring in the few-rows attention kernel
// (cache_common.cuh: ring_clear, ring_arm, ring_armed), built and run on the CPU by
// tests/test_cache_host.py.  Plays the block's warps, barriers and copies step by
// step in random orders, some warps much slower than others, over shared memory that
// holds what an earlier block left, and verifies that a warp never takes a stage
// before its tile is there and that every tile is taken.  With the argument "keep"
// the words are not cleared: the play then has to see a tile taken too early.
// Prints "OK", or what went wrong.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <vector>

#include "../sparse_hstu_attention_b200/csrc/cache_common.cuh"

using namespace hstu;

constexpr int kW = 8, kStages = 12;

struct Block {
  volatile int armed[kStages];
  int done[kStages] = {};   // phases of the stage's barrier that are complete
  int tile[kStages];        // tile the stage holds
  std::vector<int> flying;  // tiles whose copies are in flight
  // a parity wait passes unless the phase under way has that parity
  bool parity_wait(int s, int parity) const { return (done[s] & 1) != parity; }
};

// One warp, a step at a time: its first loads, then wait, take, load.
struct Warp {
  int w, nt, k, step = 0;
  std::vector<int> first;
  Warp(int w_, int nt_) : w(w_), nt(nt_), k(w_) {
    if (w < nt) first.push_back(w);
    if (w + kW < kStages && w + kW < nt) first.push_back(w + kW);
  }
  bool ended() const { return first.empty() && k >= nt && step == 0; }
  // 0: went on or waited; 1: took a stage that does not hold its tile
  int go(Block& b, int* taken) {
    const bool start = !first.empty();
    if (start || step >= 2) {  // a load: the word, then the copies
      const int t = start ? first.front() : k + kStages;
      const int word = start ? 0 : 2;
      if (step == word) {
        ring_arm(b.armed, t, kStages);
        ++step;
        return 0;
      }
      b.flying.push_back(t);
      step = 0;
      if (start) first.erase(first.begin());
      else k += kW;
      return 0;
    }
    if (k >= nt) return 0;
    const int s = k % kStages;
    if (step == 0) {
      step = ring_armed(b.armed, k, kStages);
      return 0;
    }
    if (!b.parity_wait(s, k / kStages & 1)) return 0;
    if (b.tile[s] != k) return 1;
    ++*taken;
    step = k + kStages < nt ? 2 : 0;
    if (step == 0) k += kW;
    return 0;
  }
};

int main(int argc, char** argv) {
  const int plays = argc > 1 ? atoi(argv[1]) : 2000;
  const bool keep = argc > 2 && !strcmp(argv[2], "keep");
  std::mt19937 g(11);
  auto u = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(g); };
  int early = 0;
  for (int p = 0; p < plays; ++p) {
    const int nt = u(0, 4) ? u(0, 80) : u(10, 14);
    Block b;
    for (int s = 0; s < kStages; ++s) {
      b.armed[s] = u(-2, 7);
      b.tile[s] = -1;
    }
    if (!keep) ring_clear(b.armed, kStages);
    std::vector<Warp> warps;
    int odds[kW], sum = 0, taken = 0, bad = 0;
    for (int w = 0; w < kW; ++w) {
      warps.emplace_back(w, nt);
      sum += odds[w] = u(0, 3) ? u(20, 100) : 1;
    }
    const int copy_odds = u(5, 200);
    long steps = 0;
    for (bool left = true; left && !bad; ++steps) {
      if (steps > 2000000) {
        printf("stuck: nt=%d taken=%d\n", nt, taken);
        return 1;
      }
      int x = u(0, sum + copy_odds - 1);
      if (x < copy_odds) {  // a copy lands
        if (!b.flying.empty()) {
          const int i = u(0, (int)b.flying.size() - 1), t = b.flying[i];
          b.flying.erase(b.flying.begin() + i);
          b.tile[t % kStages] = t;
          ++b.done[t % kStages];
        }
      } else {
        x -= copy_odds;
        int w = 0;
        while (x >= odds[w]) x -= odds[w++];
        bad = warps[w].go(b, &taken);
      }
      left = !b.flying.empty();
      for (auto& w : warps) left = left || !w.ended();
    }
    early += bad;
    if (!bad && taken != nt) {
      printf("%d of %d tiles taken\n", taken, nt);
      return 1;
    }
  }
  if (keep ? early == 0 : early != 0) {
    printf("%d of %d plays took a tile too early\n", early, plays);
    return 1;
  }
  printf("OK\n");
  return 0;
}
