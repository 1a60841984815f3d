// Shared definitions of the paged 4-bit history cache (include/hstu_cache.h):
// kernel arguments, the page layout and the keys a tile of new rows sees.
#pragma once

#include "../../include/hstu_cache.h"
#include "sla_common.cuh"

namespace hstu {

// Device pointers and sizes of a cache's tables.
struct CacheTab {
  int32_t* status;
  int32_t* free_count;
  int32_t* lengths;
  int32_t* free_pages;
  int32_t* bt;
  int B, M, P;
  int ps, lps;  // page size and its log2
};

__device__ __forceinline__ int cache_status(const CacheTab& t) {
  return *((volatile const int32_t*)t.status);
}
__device__ __forceinline__ void cache_fail(const CacheTab& t, int code) {
  atomicCAS(t.status, 0, code);
}

// SMs of a B200; the launch rules count blocks by it.  (Another number would make a
// rule's choice less apt, not wrong.)
constexpr int kSMs = 148;

// Byte offsets inside one head's block of a page.
template <int D>
struct PageLayout {
  int v, kp, vp, bytes;
  __host__ __device__ __forceinline__ explicit PageLayout(int ps)
      : v(ps * (D / 2)), kp(ps * D), vp(ps * D + 4 * ps), bytes(ps * (D + 8)) {}
};

// Place of token r within its group of four V bytes: 0, 2, 1, 3.
__host__ __device__ __forceinline__ int v_place(int r) {
  return (r & ~3) | ((r & 1) << 1) | ((r >> 1) & 1);
}

struct CacheRowArgs {
  CacheTab t;
  int H;
  int64_t T;
  const int64_t* slots;
  uint8_t* pages;
  int64_t page_stride;
  bf16* k;
  bf16* v;
  int64_t k_rs, v_rs;
};

struct CacheAttnArgs {
  CacheTab t;
  int H, max_new;
  int64_t T;
  const int32_t* offs;
  const int32_t* nts;
  int K1, K2e;
  float alpha, inv_n;
  const bf16* q;
  const bf16* k;
  const bf16* v;
  int64_t q_rs, k_rs, v_rs;
  const uint8_t* pages;
  int64_t page_stride;
  bf16* out;
  int64_t o_rs;
};

// One sequence of an attend call: its rows, cached length and history rows.
struct CacheSeq {
  int s0, n, h, Lh;  // first row, rows, of them history rows, cached tokens
};

// Sequence b's numbers as they stand in memory, and their check: false (and
// status set) if they are out of range.
struct CacheSeqRaw {
  int o0, o1, nt, Lh;
};
__device__ __forceinline__ CacheSeqRaw cache_seq_load(const CacheAttnArgs& a, int b) {
  CacheSeqRaw r;
  r.o0 = a.offs[b];
  r.o1 = a.offs[b + 1];
  r.nt = a.nts ? a.nts[b] : 0;
  r.Lh = a.t.lengths[b];
  return r;
}
__device__ __forceinline__ bool cache_seq_check(const CacheAttnArgs& a, const CacheSeqRaw& r,
                                                CacheSeq* s) {
  s->s0 = r.o0;
  s->n = r.o1 - r.o0;
  s->h = s->n - r.nt;
  s->Lh = r.Lh;
  const bool ok = r.o0 >= 0 && r.o1 >= r.o0 && (int64_t)r.o1 <= a.T && r.nt >= 0 &&
                  r.nt <= s->n && s->n <= a.max_new && r.Lh >= s->h && r.Lh <= a.t.M * a.t.ps;
  if (!ok) cache_fail(a.t, HSTU_SLA_ERR_BAD_INPUT);
  return ok;
}
__device__ __forceinline__ bool cache_seq(const CacheAttnArgs& a, int b, CacheSeq* s) {
  return cache_seq_check(a, cache_seq_load(a, b), s);
}

// Cached keys that row r of a sequence sees: [0, pre) and [lo, hi) (either may
// be empty).  With i the row's position (Lh for a candidate, whose window ends
// there) the window is [i - K1 + 1, i], cut at Lh - 1.
struct CacheRow {
  int pre, lo, hi;
};
__host__ __device__ __forceinline__ CacheRow cache_row(int r, int h, int Lh, int K1, int K2e) {
  const int i = r < h ? Lh - h + r : Lh;
  CacheRow c;
  c.hi = imin(i + 1, Lh);
  c.pre = imin(K2e, c.hi);
  c.lo = imax(0, i - K1 + 1);  // K1 = 0: i + 1, an empty window
  return c;
}

// Key tiles (64 keys each) that rows [r0, r1) see: the first n_pre tiles and
// the tiles [band, band + n - n_pre), n of them in all.
struct CacheTiles {
  int n_pre, band, n;
  __host__ __device__ __forceinline__ int at(int e) const {
    return e < n_pre ? e : band + e - n_pre;
  }
};
template <int TK>
__host__ __device__ __forceinline__ CacheTiles cache_tiles(int r0, int r1, int h, int Lh, int K1,
                                                           int K2e) {
  const CacheRow a = cache_row(r0, h, Lh, K1, K2e);      // the lowest window
  const CacheRow z = cache_row(r1 - 1, h, Lh, K1, K2e);  // the highest ends
  CacheTiles t;
  t.n_pre = (z.pre + TK - 1) / TK;
  const int blo = imax(a.lo / TK, t.n_pre), bhi = a.lo < z.hi ? (z.hi + TK - 1) / TK : 0;
  t.band = blo;
  t.n = t.n_pre + imax(0, bhi - blo);
  return t;
}

// Whether rows [r0, r1) all see the whole key tile [j0, j0 + TK), so that its
// mask need not be evaluated.
struct CacheFull {
  int pre, lo, hi;
  __host__ __device__ __forceinline__ bool operator()(int j0, int TK) const {
    return j0 + TK <= hi && (j0 + TK <= pre || j0 >= lo);
  }
};
__host__ __device__ __forceinline__ CacheFull cache_full(int r0, int r1, int h, int Lh, int K1,
                                                         int K2e) {
  const CacheRow a = cache_row(r0, h, Lh, K1, K2e);
  CacheFull f;
  f.pre = a.pre;
  f.hi = a.hi;
  f.lo = cache_row(r1 - 1, h, Lh, K1, K2e).lo;
  return f;
}

// A block's key tiles k = 0, 1, ... go round a ring of `stages` stages, tile k as
// phase k / stages of its stage's barrier.  A wait on that barrier names only the
// phase's parity, and so also passes while the phase before is still in flight; on a
// barrier that nothing was loaded to yet, the wait for phase 1 does.  So a word per
// stage says which phase it is armed for, none to begin with, and a warp waits for
// phase 1 and up only once that is the phase.  ring_clear comes before a barrier of
// the block that all its loads and waits come after.
__host__ __device__ __forceinline__ void ring_clear(volatile int* armed, int stages) {
  for (int s = 0; s < stages; ++s) armed[s] = -1;
}
__host__ __device__ __forceinline__ void ring_arm(volatile int* armed, int k, int stages) {
  armed[k % stages] = k / stages;
}
__host__ __device__ __forceinline__ bool ring_armed(const volatile int* armed, int k,
                                                    int stages) {
  return k < stages || armed[k % stages] == k / stages;
}

// A kernel launched by launch_early starts before the one ahead of it in the
// stream has ended, and waits for that here.
__device__ __forceinline__ void wait_for_the_last_kernel() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename... P, typename... A>
cudaError_t launch_early(void (*kern)(P...), unsigned grid, unsigned threads, cudaStream_t st,
                         A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Units of a call: B H row tiles (held where it stays beyond any grid, and within 64
// bits).
inline int64_t cache_units(const CacheAttnArgs& a, int rows) {
  const int64_t bh = (int64_t)a.t.B * a.H, most = (int64_t)1 << 33;
  return (bh < most ? bh : most) * ((a.max_new + (int64_t)rows - 1) / rows);
}

cudaError_t launch_cache_plan(const CacheTab& t, const int32_t* offs, const int32_t* nts,
                              const int32_t* release, int64_t T, int64_t* slots, void* ws,
                              cudaStream_t st);
cudaError_t launch_cache_slot_map(const CacheTab& t, const int32_t* offs, int64_t T,
                                  int64_t* slots, cudaStream_t st);
cudaError_t launch_cache_append(const CacheRowArgs& a, int d, cudaStream_t st);
cudaError_t launch_cache_read(const CacheRowArgs& a, int d, cudaStream_t st);
size_t cache_attend_ws_bytes(const CacheAttnArgs& a, int d);
cudaError_t launch_cache_attend(const CacheAttnArgs& a, int d, void* ws, cudaStream_t st);

// Many rows per sequence (cache_attn_tc.cu).
size_t cache_tc_ws_bytes(const CacheAttnArgs& a, int d);
cudaError_t launch_cache_tc(const CacheAttnArgs& a, int d, void* ws, cudaStream_t st);

}  // namespace hstu
