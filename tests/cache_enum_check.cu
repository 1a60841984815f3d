// Host-side check of the history cache's masks and key tiles
// (cache_common.cuh), built and run on the CPU by tests/test_cache_host.py.
// For random sequences it brute-forces the mask and verifies that a row's
// intervals are exactly its visible keys, that the key tiles of a tile of rows
// hold every visible pair, each once and below the sequence's last tile, and
// that a tile called full is visible to every row.  Prints "OK".
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "../sparse_hstu_attention_b200/csrc/cache_common.cuh"

using namespace hstu;

static bool vis(int r, int j, int h, int Lh, int K1, int K2e) {
  if (j < 0 || j >= Lh) return false;
  if (r < h) {
    const int i = Lh - h + r;
    return j <= i && (i - j < K1 || j < K2e);
  }
  return Lh - j < K1 || j < K2e;
}

template <int TK>
static int check(int n, int h, int Lh, int K1, int K2e, int BM) {
  for (int r = 0; r < n; ++r) {
    const CacheRow c = cache_row(r, h, Lh, K1, K2e);
    for (int j = 0; j < Lh + 70; ++j)
      if (vis(r, j, h, Lh, K1, K2e) != (j < c.pre || (j >= c.lo && j < c.hi))) return 1;
  }
  for (int r0 = 0; r0 < n; r0 += BM) {
    const int r1 = r0 + BM < n ? r0 + BM : n;
    const CacheTiles t = cache_tiles<TK>(r0, r1, h, Lh, K1, K2e);
    const CacheFull f = cache_full(r0, r1, h, Lh, K1, K2e);
    std::vector<int> seen((Lh + TK - 1) / TK + 1, 0);
    for (int e = 0; e < t.n; ++e) {
      const int k = t.at(e);
      if (k < 0 || k * TK >= Lh || seen[k]++) return 2;
    }
    for (int k = 0; k * TK < Lh; ++k)
      for (int r = r0; r < r1; ++r)
        for (int j = k * TK; j < (k + 1) * TK; ++j) {
          const bool v = vis(r, j, h, Lh, K1, K2e);
          if (v && !seen[k]) return 3;
          if (!v && f(k * TK, TK)) return 4;
        }
  }
  return 0;
}

int main(int argc, char** argv) {
  std::mt19937 g(7);
  auto u = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(g); };
  const int cases = argc > 1 ? atoi(argv[1]) : 300;
  for (int c = 0; c < cases; ++c) {
    const int Lh = u(0, 3) ? u(0, 500) : u(0, 3);
    const int h = u(0, Lh < 80 ? Lh : 80), n = h + u(0, 60);
    const int K1 = u(0, 3) ? u(0, 300) : u(0, 1) ? 0x7fffffff : 0;
    const int K2e = u(0, 2) ? u(0, 150) : u(0, 1) ? 0x7fffffff : 0;
    int e = check<64>(n, h, Lh, K1, K2e, 16);
    if (!e) e = check<64>(n, h, Lh, K1, K2e, 128);
    if (!e) e = check<128>(n, h, Lh, K1, K2e, 128);
    if (e) {
      printf("mismatch %d: n=%d h=%d Lh=%d K1=%d K2e=%d\n", e, n, h, Lh, K1, K2e);
      return 1;
    }
  }
  printf("OK\n");
  return 0;
}
