// SLA HSTU attention of a few new rows per sequence over the 4-bit history
// cache (include/hstu_cache.h): one event per user, or a few rows.
//
//   out_i = (1/N) sum_j M(i,j) SiLU(alpha q_i . k_j) v_j,   k_j, v_j = m + s c
//
// The codes go to the tensor cores as whole numbers and the (s, m) pairs are
// applied to the scores and the probabilities, where they are one per key:
//   q . k_j = s_j (q . c_j) + m_j sum(q)
//   out     = sum_j (P_ij s_j) c_j + sum_j P_ij m_j.
// A nibble c in bits 0..3 of a 16-bit half is the f16 number c 2^-24 as it
// stands, and one in bits 4..7 is 16 c 2^-24 (both subnormal, exact, and taken
// at full rate by the matrix instructions): one and per pair of values, one
// shift per word.  The factors 16 go into q (its dims of those nibbles enter
// divided by 16) and into the output's factor.
//
// Roundings to fewer bits than fp32: q enters as f16 times a power of two that
// puts the row's largest |q| into [2^14, 2^15): bf16's 8 bits fit f16's 11, so
// this is exact down to 2^-27 of that largest.  P s enters as f16 times a power
// of two per row, taken from the row's first tile and lowered if a later tile
// would overflow (the sums are then scaled down with it): 11 bits, and what is
// more than 2^18 below that tile's largest is held to 2^-29 of it.  Masked pairs
// are selected to zero before any product, so nothing in a masked place reaches
// a row.
//
// A unit is one (sequence, head, 8 rows); its key tiles of 64 tokens are split
// over S blocks and there over the warps.  A block streams its tiles through a
// ring of bulk copies (one per page: a head's codes and pairs of a page are
// contiguous); a warp takes a whole tile and keeps everything in registers: S
// as [keys][rows] and O as [dims][rows], P turned in between by one register
// transpose per 8 x 8.  SiLU attention has no softmax, so partial results only
// add: warps through shared memory, blocks through the workspace and a second
// kernel, in a fixed order.
//
// Which key a matrix row stands for is free, so it is chosen for the loads:
// rows g and g + 8 of score tile u are tokens 16 (g / 2) + 4 u + g mod 2 and two
// further on; a thread's K bytes (its quarter of d) and V bytes (16 tokens of a
// dim pair) are then single 16-byte loads, without bank conflicts.
//
// Bound: HBM for long histories (d + 8 bytes per token and head); instructions
// come next.  64 sequences x 4 heads of 128 over 8K-16K tokens, one row: 80 us,
// 5.2 TB/s.  Under a window of 512 tokens the same batch takes 9.0 us, and one
// sequence of 300 tokens 4.3: the latency of table, page id, page and products.
// (The one-row kernel of d = 128 keeps 16 bytes a thread in local memory.)
#include <cuda_fp16.h>

#include "cache_common.cuh"
#include "sm100.cuh"

namespace hstu {

namespace {

using namespace sm100;

constexpr int kW = 8, kThreads = 32 * kW, kRows = 8, kTK = 64, kStages = 12;

template <int D>
struct StepCfg {
  // a stage holds the tile's 1, 2 or 4 page blocks, each page_size * 2 bytes
  // further apart when there are several, so that a warp's V loads from them
  // fall into different banks
  static constexpr int STG = kTK * (D + 8) + 128;
  static constexpr int PITCH = D + 8;               // floats between rows of a result
  static constexpr int OFF_REST = kStages * STG;    // [warp][8]
  static constexpr int OFF_SELF = OFF_REST + kW * kRows * 4;
  static constexpr int OFF_BAR = OFF_SELF + kRows * 4;
  static constexpr int OFF_ARMED = OFF_BAR + kStages * 8;  // phase a stage is armed for
  static constexpr int SMEM = OFF_ARMED + kStages * 4;
  static_assert(kStages * STG >= kW * kRows * PITCH * 4, "the warps' results fit the ring");
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// Bounded wait: false after kWaitLimitNs (status set).
__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, const CacheTab& t) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer() - t0 > kWaitLimitNs) {
      cache_fail(t, HSTU_SLA_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

// Waits, as long at most, until tile k's stage is armed for it.
__device__ __forceinline__ bool bounded_armed(const volatile int* armed, int k,
                                              const CacheTab& t) {
  if (ring_armed(armed, k, kStages)) return true;
  const uint64_t t0 = globaltimer();
  while (!ring_armed(armed, k, kStages)) {
    if (globaltimer() - t0 > kWaitLimitNs) {
      cache_fail(t, HSTU_SLA_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float x, float y) {
  const __half2 v = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;  // nibbles n, n + 4 as f16 codes

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <int N>
__device__ __forceinline__ void lds(uint32_t (&r)[N], uint32_t addr) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr));
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r[0]) : "r"(addr));
}

// Tiles of one block of a unit with n of them: at least one per warp.
__device__ __forceinline__ int block_tiles(int n, int S) { return imax(kW, (n + S - 1) / S); }

// A candidate's own pair, SiLU(alpha q_i . k_i), of rows r0 + warp, ...
template <int D>
__device__ __forceinline__ void self_pairs(const CacheAttnArgs& a, const CacheSeq& sq, int h,
                                           int r0, int nr, float* self) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r = warp; r < nr; r += kW) {
    float p = 0.f;
    if (r0 + r >= sq.h) {
      const int64_t row = sq.s0 + r0 + r;
      float x = 0.f;
      for (int e = lane; e < D; e += 32)
        x = fmaf(__bfloat162float(a.q[row * a.q_rs + h * D + e]),
                 __bfloat162float(a.k[row * a.k_rs + h * D + e]), x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      x *= a.alpha;
      p = x / (1.f + __expf(-x));
    }
    if (lane == 0) self[r] = p;
  }
}

// Dims c, c + 1 of row r: the sum over keys, the own pair, 1/N, bf16.
__device__ __forceinline__ void store_pair(const CacheAttnArgs& a, const CacheSeq& sq, int col,
                                           int r, float2 x, float self) {
  const int64_t row = sq.s0 + r;
  if (r >= sq.h) {
    const uint32_t v2 = *reinterpret_cast<const uint32_t*>(a.v + row * a.v_rs + col);
    x.x = fmaf(self, bf_lo(v2), x.x);
    x.y = fmaf(self, bf_hi(v2), x.y);
  }
  *reinterpret_cast<uint32_t*>(a.out + row * a.o_rs + col) =
      pack_bf16x2(x.x * a.inv_n, x.y * a.inv_n);
}

// parts: fp32 [unit][S][8][D], the blocks' sums (S > 1 only).
// ONE: one row a unit.  All 8 columns of the scores then hold that row, so that
// lane t of four takes only the tokens of score tile u = t, a quarter of the
// pointwise work, and gives their P to column 2t of the second product; the
// columns are added at the end.
template <int D, bool ONE>
__global__ void __launch_bounds__(kThreads, 2)
    cache_step_kernel(const __grid_constant__ CacheAttnArgs a, int S, int row_tiles,
                      float* __restrict__ parts) {
  using C = StepCfg<D>;
  constexpr int WD = D / 32;  // words of a thread's K quarter
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int split = (int)blockIdx.x % S;
  const int unit = (int)blockIdx.x / S;
  const int bh = unit / row_tiles, r0 = (unit % row_tiles) * kRows;
  const int b = bh / a.H, h = bh % a.H;

  const int status = cache_status(a.t);
  CacheSeq sq;
  if (!cache_seq(a, b, &sq) || r0 >= sq.n) return;
  const int nr = ONE ? 1 : imin(kRows, sq.n - r0);
  const CacheTiles tl = cache_tiles<kTK>(r0, r0 + nr, sq.h, sq.Lh, a.K1, a.K2e);
  const int bl = block_tiles(tl.n, S);
  const int e0 = imin(split * bl, tl.n), nt = imin(bl, tl.n - e0);  // this block's tiles
  if (split > 0 && nt <= 0) return;

  const int ps = a.t.ps, lps = a.t.lps, ppt = kTK >> lps;  // pages a tile
  const PageLayout<D> lay(ps);
  const int pitch = lay.bytes + (ps < kTK ? 2 * ps : 0);
  const uint32_t ring = smem_addr(smem), bar = ring + C::OFF_BAR;
  volatile int* armed = reinterpret_cast<volatile int*>(smem + C::OFF_ARMED);
  if (threadIdx.x == 0) {
    ring_clear(armed, kStages);
    for (int s = 0; s < kStages; ++s) mbar_init(bar + 8 * s, 1);
    fence_barrier_init();
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }

  // The block's tiles k = 0, 1, ... use stage k mod kStages; warp k mod kW
  // consumes tile k and then loads tile k + kStages into the stage it freed.
  // The first kStages tiles are loaded by the warps in turn, so a warp loads
  // tiles warp, warp + kW (if below kStages), then its own + kStages.
  // Page ids of what a warp loads are held 32 at a time, one a lane: its first
  // two tiles', then those of the tiles it loads later, entry i ppt + p being page
  // p of tile kStages + warp + i kW; the next 32 are read when the last are begun.
  const int32_t* bt = a.t.bt + (int64_t)b * a.t.M;
  const int pages = (sq.Lh + ps - 1) >> lps;
  auto page_id = [&](int k, int p) -> int {
    if (k >= nt) return 0;
    const int i = tl.at(e0 + k) * ppt + p;
    if (i >= pages) return 0;
    const int x = bt[i];
    if (x >= 0 && x < a.t.P) return x;
    cache_fail(a.t, HSTU_SLA_ERR_BAD_INPUT);
    return 0;
  };
  const int lpp = 6 - lps;  // log2 of ppt
  auto load = [&](int k, int ids, int at) {  // by the warp; ids: lanes at, at + 1, ...
    const int id = __shfl_sync(0xffffffffu, ids, (at + lane) & 31);
    const uint32_t dst = ring + (k % kStages) * C::STG, bk = bar + 8 * (k % kStages);
    const int np = imin(ppt, pages - tl.at(e0 + k) * ppt);
    if (lane == 0) {
      mbar_expect_tx(bk, (uint32_t)(np * lay.bytes));
      __threadfence_block();
      ring_arm(armed, k, kStages);
    }
    __syncwarp();
    if (lane < np)
      bulk_load(dst + lane * pitch, a.pages + id * a.page_stride + (int64_t)h * lay.bytes,
                (uint32_t)lay.bytes, bk);
  };
  {
    const int k = warp + (lane >> lpp) * kW;  // lanes of tiles warp and warp + kW
    const int id = k < kStages ? page_id(k, lane & (ppt - 1)) : 0;
    // barriers and phase words are initialised; one status for the whole block, whose
    // warps may have read different ones, so that they part ways together
    if (__syncthreads_or(status != 0)) return;
    if (warp < nt) load(warp, id, 0);
    if (warp + kW < kStages && warp + kW < nt) load(warp + kW, id, ppt);
  }
  auto later_ids = [&](int i0) {
    const int i = i0 + lane;
    return page_id(kStages + warp + (i >> lpp) * kW, i & (ppt - 1));
  };
  int ids = later_ids(0), ids_next = later_ids(32);

  // Q fragments of row g: this thread's quarter of its dims, in the order of a
  // K word's pairs, every second one divided by 16.  sum(q) alpha / 2, and the
  // factor that makes the matrix product alpha / 2 q . c.
  uint32_t qf[2 * WD][2];
  float sum0, sum1, f0, f1;  // of rows 2t, 2t + 1
  {
    uint32_t x[WD][4];
    uint32_t most = 0;
    float sum = 0.f;
    const bf16* q0 = a.q + (int64_t)(sq.s0 + r0 + (ONE ? 0 : g)) * a.q_rs + h * D + t * (D / 4);
#pragma unroll
    for (int w = 0; w < WD; ++w) {
      uint4 y = make_uint4(0, 0, 0, 0);
      if (ONE || g < nr) y = *reinterpret_cast<const uint4*>(q0 + 8 * w);
      x[w][0] = y.x; x[w][1] = y.y; x[w][2] = y.z; x[w][3] = y.w;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sum += bf_lo(x[w][e]) + bf_hi(x[w][e]);
        most = umax(most, umax(x[w][e] & 0x7fffu, (x[w][e] >> 16) & 0x7fffu));
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      most = umax(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
    // 2^(14 - e) for a largest value in [2^e, 2^(e + 1)); rows of zeros and of
    // values below 2^-112 take 2^126
    const int e = imax((int)(most >> 7) - 127, -112);
    const float up = __int_as_float((141 - e) << 23), down = __int_as_float((113 + e) << 23);
    const float f = down * (0.5f * a.alpha * 16777216.f);
    sum *= 0.5f * a.alpha;
    if (most >= 0x7f80u) sum = __int_as_float(0x7fc00000);  // a NaN or infinity: a NaN row
#pragma unroll
    for (int w = 0; w < WD; ++w)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float z = i & 1 ? up * 0.0625f : up;
        qf[2 * w + (i >> 1)][i & 1] = pack_f16(bf_lo(x[w][i]) * z, bf_hi(x[w][i]) * z);
      }
    sum0 = __shfl_sync(0xffffffffu, sum, 8 * t);
    sum1 = __shfl_sync(0xffffffffu, sum, 8 * t + 4);
    f0 = __shfl_sync(0xffffffffu, f, 8 * t);
    f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
  }
  const CacheRow cr0 = cache_row(r0 + imin(2 * t, nr - 1), sq.h, sq.Lh, a.K1, a.K2e);
  const CacheRow cr1 = cache_row(r0 + imin(2 * t + 1, nr - 1), sq.h, sq.Lh, a.K1, a.K2e);
  const CacheFull whole = cache_full(r0, r0 + nr, sq.h, sq.Lh, a.K1, a.K2e);

  // o[i]: dims 16 i + 2 g (+ 1 in [2], [3], times 16) of rows 2t ([0], [2]) and
  // 2t + 1, times 2^-24 and the row's scale
  float o[D / 16][4];
#pragma unroll
  for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float rest0 = 0.f, rest1 = 0.f;    // sum P m of rows 2t, 2t + 1 (this thread's keys)
  float sc0 = 0x1p100f, sc1 = sc0;   // the rows' scales: the first P lowers them

  const int pt = (16 * t) >> lps, in = (16 * t) & (ps - 1);    // page and place of tokens 16 t
  const int pg = (16 * (g >> 1)) >> lps, ing = (16 * (g >> 1)) & (ps - 1);  // and 16 (g / 2)
  const uint32_t koff = pg * pitch + (ing + (g & 1)) * (D / 2) + t * (D / 8);
  const uint32_t poff = pg * pitch + lay.kp + 4 * (ing + (g & 1));
  const uint32_t voff = pt * pitch + lay.v + in + g * ps;
  const int jg = 16 * (g >> 1) + (g & 1);
  // Phase k / kStages - 1 of tile k's stage is another warp's tile, perhaps not
  // landed yet: so the stage's word first (ring_armed).
  auto landed = [&](int k) -> bool {
    bool done = bounded_armed(armed, k, a.t);
    done = done && bounded_wait(bar + 8 * (k % kStages), k / kStages & 1, a.t);
    return __all_sync(0xffffffffu, done);
  };
  bool ok = true;
  int k = warp, n_done = 0;
  for (; k < nt; k += kW, ++n_done) {
    ok = landed(k);
    if (!ok) break;
    const int j0 = tl.at(e0 + k) * kTK;
    const uint32_t stg = ring + (k % kStages) * C::STG;
    const bool full = whole(j0, kTK);
    // P s of rows 2t, 2t + 1 at tokens j0 + jg + 4u (+ 2); ONE: of the row at u = t
    constexpr int NU = ONE ? 1 : 4;
    float p0[NU][2], p1[NU][2];
    auto pointwise = [&](int u, int iu, const float (&st)[4]) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t kp[1], vp[1];
        lds<1>(kp, stg + poff + 16 * u + 8 * e);
        lds<1>(vp, stg + poff + (lay.vp - lay.kp) + 16 * u + 8 * e);
        const float ks = bf_lo(kp[0]), km = bf_hi(kp[0]), vs = bf_lo(vp[0]), vm = bf_hi(vp[0]);
        const int j = j0 + jg + 4 * u + 2 * e;
        float x = fmaf(st[2 * e] * f0, ks, km * sum0);
        float p = fmaf(x, tanh_approx(x), x), m = p * vm;
        p0[iu][e] = p * vs;
        if (!full) {
          const bool see = j < cr0.pre || (j >= cr0.lo && j < cr0.hi);
          p0[iu][e] = see ? p0[iu][e] : 0.f;
          m = see ? m : 0.f;
        }
        rest0 += m;
        p1[iu][e] = 0.f;
        if constexpr (!ONE) {
          x = fmaf(st[2 * e + 1] * f1, ks, km * sum1);
          p = fmaf(x, tanh_approx(x), x);
          m = p * vm;
          p1[iu][e] = p * vs;
          if (!full) {
            const bool see = j < cr1.pre || (j >= cr1.lo && j < cr1.hi);
            p1[iu][e] = see ? p1[iu][e] : 0.f;
            m = see ? m : 0.f;
          }
          rest1 += m;
        }
      }
    };
    float mine[4] = {0.f, 0.f, 0.f, 0.f};  // ONE: the scores of u = t
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float st[4] = {0.f, 0.f, 0.f, 0.f};
      uint32_t ka[WD], kb[WD];
      lds<WD>(ka, stg + koff + 4 * u * (D / 2));
      lds<WD>(kb, stg + koff + (4 * u + 2) * (D / 2));
#pragma unroll
      for (int w = 0; w < WD; ++w) {
        mma_f16(st, ka[w] & kLow, kb[w] & kLow, ka[w] & kHigh, kb[w] & kHigh, qf[2 * w][0],
                qf[2 * w][1]);
        const uint32_t x = ka[w] >> 8, y = kb[w] >> 8;
        mma_f16(st, x & kLow, y & kLow, x & kHigh, y & kHigh, qf[2 * w + 1][0],
                qf[2 * w + 1][1]);
      }
      if constexpr (ONE) {
        mine[0] = u == t ? st[0] : mine[0];
        mine[2] = u == t ? st[2] : mine[2];
      } else {
        pointwise(u, u, st);
      }
    }
    if constexpr (ONE) pointwise(t, 0, mine);
    uint32_t pk[4][2];
    uint32_t big = 0;
    auto pack = [&]() {
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if constexpr (ONE) {
            const uint32_t x = u == 0 ? pack_f16(p0[0][e] * sc0, 0.f) : pk[0][e];
            pk[u][e] = x;
          } else {
            pk[u][e] = pack_f16(p0[u][e] * sc0, p1[u][e] * sc1);
          }
          if (!ONE || u == 0) big = __vmaxu2(big, pk[u][e] & 0x7fff7fffu);
        }
    };
    pack();
    if (__any_sync(0xffffffffu, (big & 0xffffu) >= 0x7c00u || big >= 0x7c000000u)) {
      // P s beyond f16 with this scale (or the row's first): put its largest
      // into [2^4, 2^5)
      float m0 = 0.f, m1 = 0.f;
#pragma unroll
      for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m0 = fmaxf(m0, fabsf(p0[u][e]));
          m1 = fmaxf(m1, fabsf(p1[u][e]));
        }
#pragma unroll
      for (int x = ONE ? 1 : 4; x < 32; x <<= 1) {
        m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, x));
        m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, x));
      }
      // 2^(4 - e): the exponent field of m is e + 127
      auto scale = [](float m, float old) {
        const int e = (int)(__float_as_uint(m) >> 23);
        return e == 0 ? old : fminf(old, __int_as_float(imin(imax(258 - e, 4), 227) << 23));
      };
      const float n0 = scale(m0, sc0), n1 = scale(m1, sc1);
      const float d0 = n0 / sc0, d1 = n1 / sc1;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        o[i][0] *= d0;
        o[i][2] *= d0;
        o[i][1] *= d1;
        o[i][3] *= d1;
      }
      sc0 = n0;
      sc1 = n1;
      pack();
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int e = 0; e < 2; ++e) pk[u][e] = transpose8x8(!ONE || u == t ? pk[u][e] : 0u);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint32_t vw[4];
      lds<4>(vw, stg + voff + 8 * i * ps);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        // low nibbles: dim 2 (8 i + g); high: the next.  Bytes are tokens 0, 2, 1, 3.
        const uint32_t x = vw[u] >> 8;
        mma_f16(o[i], vw[u] & kLow, vw[u] & kHigh, x & kLow, x & kHigh, pk[u][0], pk[u][1]);
      }
    }
    __syncwarp();
    if (k + kStages < nt) {
      const int at = n_done << lpp;
      if (at > 0 && (at & 31) == 0) {
        ids = ids_next;
        ids_next = later_ids(at + 32);
      }
      load(k + kStages, ids, at & 31);
    }
  }
  // If a wait gave up, the copies in flight land before the ring is used again
  // or the block ends: of every stage, the phase that was armed last.
  if (!__syncthreads_and(ok)) {
    if (threadIdx.x < kStages) {
      drain_wait(bar + 8 * threadIdx.x, 0);
      drain_wait(bar + 8 * threadIdx.x, 1);
    }
    __syncthreads();
  }

  // The warp's result, [8][PITCH] fp32, and its rows' rest.
  if constexpr (ONE) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int x = 1; x < 4; x <<= 1) {
        o[i][0] += __shfl_xor_sync(0xffffffffu, o[i][0], x);
        o[i][2] += __shfl_xor_sync(0xffffffffu, o[i][2], x);
      }
  }
#pragma unroll
  for (int x = ONE ? 1 : 4; x < 32; x <<= 1) {
    rest0 += __shfl_xor_sync(0xffffffffu, rest0, x);
    rest1 += __shfl_xor_sync(0xffffffffu, rest1, x);
  }
  float* rests = reinterpret_cast<float*>(smem + C::OFF_REST);
  float* self = reinterpret_cast<float*>(smem + C::OFF_SELF);
  float* sums = reinterpret_cast<float*>(smem);
  if (g == 0) {
    rests[warp * kRows + 2 * t] = rest0;
    rests[warp * kRows + 2 * t + 1] = rest1;
  }
  {
    const float i0 = 1.f / sc0, i1 = 1.f / sc1;  // exact: powers of two
    float* w = sums + (warp * kRows + 2 * t) * C::PITCH + 2 * g;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      if (2 * t < nr)
        *reinterpret_cast<float2*>(w + 16 * i) =
            make_float2(o[i][0] * 0x1p24f * i0, o[i][2] * 0x1p20f * i0);
      if (2 * t + 1 < nr)
        *reinterpret_cast<float2*>(w + C::PITCH + 16 * i) =
            make_float2(o[i][1] * 0x1p24f * i1, o[i][3] * 0x1p20f * i1);
    }
  }
  if (S == 1) self_pairs<D>(a, sq, h, r0, nr, self);
  __syncthreads();
  for (int e = threadIdx.x * 2; e < nr * D; e += 2 * kThreads) {
    const int r = e / D, c = e % D;
    float2 x = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      const float2 y =
          *reinterpret_cast<const float2*>(sums + (w * kRows + r) * C::PITCH + c);
      x.x += y.x + rests[w * kRows + r];
      x.y += y.y + rests[w * kRows + r];
    }
    if (S == 1)
      store_pair(a, sq, h * D + c, r0 + r, x, self[r]);
    else
      *reinterpret_cast<float2*>(parts + (int64_t)blockIdx.x * (kRows * D) + e) = x;
  }
}

// The blocks' sums of a unit, in order.
template <int D>
__global__ void __launch_bounds__(kThreads)
    cache_join_kernel(const __grid_constant__ CacheAttnArgs a, int S, int row_tiles,
                      const float* __restrict__ parts) {
  __shared__ float self[kRows];
  wait_for_the_last_kernel();
  const int unit = blockIdx.x, bh = unit / row_tiles, r0 = (unit % row_tiles) * kRows;
  const int b = bh / a.H, h = bh % a.H;
  CacheSeq sq;
  const int status = cache_status(a.t);
  if (!cache_seq(a, b, &sq) || r0 >= sq.n) return;
  const int nr = imin(kRows, sq.n - r0);
  const CacheTiles tl = cache_tiles<kTK>(r0, r0 + nr, sq.h, sq.Lh, a.K1, a.K2e);
  const int used = imax(1, cdiv(tl.n, block_tiles(tl.n, S)));
  self_pairs<D>(a, sq, h, r0, nr, self);
  if (__syncthreads_or(status != 0)) return;
  for (int e = threadIdx.x * 2; e < nr * D; e += 2 * kThreads) {
    const float* p = parts + (int64_t)unit * S * (kRows * D) + e;
    float2 x = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < used; ++i, p += kRows * D) {
      const float2 y = *reinterpret_cast<const float2*>(p);
      x.x += y.x;
      x.y += y.y;
    }
    store_pair(a, sq, h * D + e % D, r0 + e / D, x, self[e / D]);
  }
}

// A thread a sequence: the checks of a call that has no rows to compute.
__global__ void __launch_bounds__(kThreads)
    cache_check_kernel(const __grid_constant__ CacheAttnArgs a) {
  const int b = (int)(blockIdx.x * kThreads + threadIdx.x);
  CacheSeq sq;
  if (b < a.t.B) cache_seq(a, b, &sq);
}

// Blocks a unit.  Two blocks fit an SM.  A unit is split until the GPU is full
// once, and further, down to 8 tiles a warp, until it is full eight times, so
// that the last blocks to finish cost little of the whole (64 sequences x 4
// heads of 8K-16K tokens, d = 128, one row: 88 us unsplit, 81 in 4, 88 in 8;
// 10-tile windows of the same batch: 9 us unsplit, 15 in 2).  The tiles are those that
// the window and the tables' capacity allow, since the lengths are on the device: over
// tables for 16K tokens one request that sees all its 300 tokens takes 5.9 us, 4.5 over
// tables of its own size; under a window there is no difference.
int step_splits(int64_t units, int64_t tiles) {
  const int64_t slots = 2 * kSMs;
  int64_t fill = (slots + units - 1) / units;
  fill = fill < tiles / kW ? fill : tiles / kW;
  int64_t even = tiles / (8 * kW);
  even = even < slots * 8 / units ? even : slots * 8 / units;
  const int64_t S = fill > even ? fill : even;
  return S < 1 ? 1 : (int)S;
}

struct StepPlan {
  int row_tiles, S;
  int64_t units;
};

// Most keys a row tile can meet.
int most_keys(const CacheAttnArgs& a) {
  const int64_t w = (int64_t)a.K1 + a.K2e + kRows, c = (int64_t)a.t.M * a.t.ps;
  return (int)(w < c ? w : c);
}

StepPlan step_plan(const CacheAttnArgs& a) {
  StepPlan p;
  p.row_tiles = (int)((a.max_new + (int64_t)kRows - 1) / kRows);
  p.units = cache_units(a, kRows);
  p.S = p.units > 0 ? step_splits(p.units, most_keys(a) / kTK + 2) : 1;
  return p;
}

template <int D>
cudaError_t launch_step(const CacheAttnArgs& a, float* parts, cudaStream_t st) {
  using C = StepCfg<D>;
  auto kern = a.max_new == 1 ? cache_step_kernel<D, true> : cache_step_kernel<D, false>;
  const StepPlan p = step_plan(a);
  if (p.units * p.S > 0x7fffffff) return cudaErrorNotSupported;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)(p.units * p.S), kThreads, C::SMEM, st>>>(a, p.S, p.row_tiles, parts);
  const cudaError_t launched = cudaGetLastError();
  if (launched != cudaSuccess || p.S == 1) return launched;
  return launch_early(cache_join_kernel<D>, (unsigned)p.units, kThreads, st, a, p.S, p.row_tiles,
                      (const float*)parts);
}

}  // namespace

// Which kernel a call takes: the one above up to 16 rows a sequence, and while its
// 8-row units fit the GPU at once up to 64 (32 if there are more than 4096 keys);
// beyond that the tiles of 128 rows on tcgen05.  Measured, above / tcgen05, us:
//   64 sequences x 4 heads of 128, 512-token window: 12 / 23 at 4 rows, 23 / 23 at 16,
//   39 / 24 at 32; 24 x 8 of 32, 256 tokens: 12 / 13 at 16, 17 / 14 at 32;
//   9 x 4 of 128, 512 tokens: 10 / 18 at 32, 13 / 18 at 64; over 8K tokens 33 / 35 at
//   16, 43 / 39 at 32, 66 / 41 at 64; 16 x 4 of 128 over 16K: 98 / 124 at 24, 114 /
//   127 at 32.
bool few_rows(const CacheAttnArgs& a) {
  const int64_t units = cache_units(a, kRows);
  return a.max_new <= 16 ||
         (units <= 2 * kSMs && a.max_new <= (most_keys(a) <= 4096 ? 64 : 32));
}

size_t cache_attend_ws_bytes(const CacheAttnArgs& a, int d) {
  if (!few_rows(a)) return cache_tc_ws_bytes(a, d);
  const StepPlan p = step_plan(a);
  return p.S == 1 ? 0 : align256((size_t)p.units * p.S * kRows * d * sizeof(float));
}

cudaError_t launch_cache_attend(const CacheAttnArgs& a, int d, void* ws, cudaStream_t st) {
  if (a.max_new == 0) {  // or no rows at all
    const unsigned blocks = (unsigned)(((int64_t)a.t.B + kThreads - 1) / kThreads);
    cache_check_kernel<<<blocks, kThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  if (!few_rows(a)) return launch_cache_tc(a, d, ws, st);
  float* parts = static_cast<float*>(ws);
  if (d == 32) return launch_step<32>(a, parts, st);
  if (d == 64) return launch_step<64>(a, parts, st);
  return launch_step<128>(a, parts, st);
}

}  // namespace hstu
