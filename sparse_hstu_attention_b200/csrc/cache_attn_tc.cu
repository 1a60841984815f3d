// SLA HSTU attention of many new rows per sequence over the 4-bit history cache
// (include/hstu_cache.h) on the 5th-generation tensor cores: candidate sets,
// chunks of history.
//
// The algebra is cache_attn.cu's: with k_j = m + s c and v_j = m' + s' c',
//   x_ij = alpha (s_j (q_i . c_j) + m_j sum(q_i)),  P = SiLU(x),
//   out_i = (1/N) (sum_j (P_ij s'_j) c'_j + sum_j P_ij m'_j  [+ own pair]),
// so what a masked place holds never enters a product: its P is selected to
// zero, its codes are finite.  K codes are the f16 subnormals c 2^-24 and
// 16 c 2^-24 there (q in f16, scaled by a power of two per row, its dims of the
// high nibbles divided by 16); V codes are bf16 whole numbers, because P s' is
// a bf16 operand: a row's P may span more than f16's range and the sums O stay
// in TMEM, where rescaling them would cost a pass.  That rounding of P s' to
// bf16 (2^-9 of itself) is the only one of more than 2^-12.
//
// A block is one (sequence, head, 128 rows), 8 warps, and two blocks share an
// SM: S = Q C^T (M = 128, N = 128 keys, K = d) and O += P C' (N = d, K = 128)
// by tcgen05 into 128 + d TMEM columns, and all warps do the same things in
// turn, so that one block's products run under the other's arithmetic:
//   V codes of tile n  -> shared memory     while S of tile n runs
//   wait S; P = SiLU(x) masked, P s' -> TMEM over the scores; issue O += P C'
//   K codes of tile n+1 -> shared memory    while that runs; issue S of n + 1
// Codes come straight from the pages into registers, 16 bytes a thread, one
// step before they are unpacked; the unpacked operands are K-major 128-byte
// swizzled tiles (V transposed: its bytes lie along the tokens).  Scores are
// read from TMEM as 16 x 256-bit fragments, so a thread has 4 rows and a quarter
// of the columns and the per-key pairs are one 16-byte load per two columns and
// four rows.
//
// Bound: issue slots of the pointwise part (about 5 a score), then the tensor
// cores and shared memory.
#include "cache_common.cuh"
#include "sm100.cuh"

namespace hstu {

namespace {

using namespace sm100;

constexpr int kThreads = 256, kBM = 128, kBN = 128;
constexpr int kIdTiles = 32;  // tiles whose page ids are held at a time
constexpr uint32_t kColS = 0, kColO = 128, kTmemCols = 256;

template <int D>
struct TcCfg {
  static constexpr int SWK = D >= 64 ? 128 : 64;       // bytes of a K / Q row in a box
  static constexpr int BOXK = 128 * SWK;               // 128 rows of SWK bytes
  static constexpr int NBK = D * 2 / SWK;              // boxes of a K / Q tile
  static constexpr int TILE_K = NBK * BOXK;
  static constexpr int BOXV = D * 128;                 // D rows of 64 tokens
  static constexpr int OFF_Q = 0, OFF_K = TILE_K, OFF_V = 2 * TILE_K;
  static constexpr int OFF_PAR = OFF_V + 2 * BOXV;     // 2 x [64 column pairs][8] floats
  static constexpr int OFF_F = OFF_PAR + 2 * 64 * 32;  // per row: factor, sum(q), own pair
  static constexpr int OFF_REST = OFF_F + 3 * 128 * 4;  // [2][128]
  static constexpr int OFF_IDS = OFF_REST + 2 * 128 * 4;  // [2][kIdTiles * 8] page ids
  static constexpr int OFF_BAR = OFF_IDS + 2 * kIdTiles * 8 * 4;
  static constexpr int NEED = OFF_BAR + 32 + 1024;     // + alignment slack
  // two blocks an SM, no more: their TMEM columns are all there are
  static constexpr int SMEM = NEED > 80 * 1024 ? NEED : 80 * 1024;
  static constexpr uint32_t SWZK = SWK == 128 ? kSwizzle128B : kSwizzle64B;
  static constexpr int CHK = D / 32;                   // 16-byte chunks of a K code row, per lane group
};

// kind::f16 with f16 A / B (format 0) and f32 accumulator, both K-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// 16 lanes x 32 columns: regs 4i .. 4i + 3 are row g, columns 8i + 2t, + 1, and
// row g + 8, the same columns.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// 16 lanes x 16 columns: regs 2i, 2i + 1 are rows g and g + 8, column 4i + t.
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_f16x2(float x, float y) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t sub16_bf16x2(uint32_t x) {  // 16 + c -> c, exact
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0xc180c180u));
  return r;
}

// Bounded wait for the phase of parity `parity`: false after kWaitLimitNs.
__device__ __forceinline__ bool phase_wait(uint32_t bar, uint32_t parity, const CacheTab& t) {
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

// parts: fp32 [block][128][D], the blocks' sums (S > 1 only).
template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    cache_tc_kernel(const __grid_constant__ CacheAttnArgs a, int S, int row_tiles,
                    float* __restrict__ parts) {
  using C = TcCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const sm = smem_raw + (base - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int split = (int)blockIdx.x % S, unit = (int)blockIdx.x / S;
  const int bh = unit / row_tiles, r0 = (unit % row_tiles) * kBM;
  const int b = bh / a.H, h = bh % a.H;

  CacheSeq sq;
  if (!cache_seq(a, b, &sq) || r0 >= sq.n) return;
  // (one status for the whole block, so that its threads part ways together)
  if (__syncthreads_or(cache_status(a.t) != 0)) return;
  const int nr = imin(kBM, sq.n - r0);
  const CacheTiles tl = cache_tiles<kBN>(r0, r0 + nr, sq.h, sq.Lh, a.K1, a.K2e);
  const int bl = (tl.n + S - 1) / S;
  const int e0 = imin(split * bl, tl.n), nt = imin(bl, tl.n - e0);
  if (split > 0 && nt <= 0) return;

  const uint32_t sQ = base + C::OFF_Q, sK = base + C::OFF_K, sV = base + C::OFF_V;
  const uint32_t bar_s = base + C::OFF_BAR, bar_o = bar_s + 8;
  uint32_t* const slot = reinterpret_cast<uint32_t*>(sm + C::OFF_BAR + 16);
  float* const row_f = reinterpret_cast<float*>(sm + C::OFF_F);
  float* const row_sum = row_f + 128;
  float* const row_self = row_f + 256;
  float* const rests = reinterpret_cast<float*>(sm + C::OFF_REST);
  int* const ids = reinterpret_cast<int*>(sm + C::OFF_IDS);

  if (warp == 0) {
    tmem_alloc(smem_addr(slot), kTmemCols);
    tmem_relinquish();
  }
  if (tid == 32) {
    mbar_init(bar_s, 1);
    mbar_init(bar_o, 1);
    fence_barrier_init();
  }

  const int ps = a.t.ps, lps = a.t.lps, lpt = 7 - lps;  // 2^lpt pages a tile
  const PageLayout<D> lay(ps);
  const int pages = (sq.Lh + ps - 1) >> lps;
  const int32_t* const bt = a.t.bt + (int64_t)b * a.t.M;
  const uint8_t* const head = a.pages + (int64_t)h * lay.bytes;

  // Page ids of the tiles [32 c, 32 c + 32): -1 past the cached tokens.
  auto load_ids = [&](int c) {
    const int n = c * kIdTiles + (tid >> lpt);
    if (tid >= kIdTiles << lpt) return;
    int id = -1;
    if (n < nt) {
      const int i = (tl.at(e0 + n) << lpt) + (tid & ((1 << lpt) - 1));
      if (i < pages) {
        id = bt[i];
        if (id < 0 || id >= a.t.P) {
          cache_fail(a.t, HSTU_SLA_ERR_BAD_INPUT);
          id = -1;
        }
      }
    }
    ids[(c & 1) * (kIdTiles * 8) + tid] = id;
  };
  // Block of the page that holds token `tok` of tile n, or null.
  auto page_of = [&](int n, int tok) -> const uint8_t* {
    const int id = ids[((n / kIdTiles) & 1) * (kIdTiles * 8) + ((n % kIdTiles) << lpt) + (tok >> lps)];
    return id < 0 ? nullptr : head + id * a.page_stride;
  };
  load_ids(0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;

  // K codes: lane takes token 8 (..) + lane % 8 and D / 8 of its bytes.
  uint32_t kc[2][4], vc[2][4], kpar = 0, vpar = 0;
  auto load_k = [&](int n) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int tok = x * 64 + warp * 8 + (lane & 7);
      const uint8_t* p = page_of(n, tok);
#pragma unroll
      for (int w = 0; w < 4; ++w) kc[x][w] = 0;
      if (p) {
        p += (tok & (ps - 1)) * (D / 2) + (lane >> 3) * (D / 8);
        if constexpr (D == 128) {
          const uint4 y = *reinterpret_cast<const uint4*>(p);
          kc[x][0] = y.x; kc[x][1] = y.y; kc[x][2] = y.z; kc[x][3] = y.w;
        } else if constexpr (D == 64) {
          const uint2 y = *reinterpret_cast<const uint2*>(p);
          kc[x][0] = y.x; kc[x][1] = y.y;
        } else {
          kc[x][0] = *reinterpret_cast<const uint32_t*>(p);
        }
      }
    }
    kpar = vpar = 0;
    if (tid < kBN) {
      const uint8_t* p = page_of(n, tid);
      if (p) {
        kpar = *reinterpret_cast<const uint32_t*>(p + lay.kp + 4 * (tid & (ps - 1)));
        vpar = *reinterpret_cast<const uint32_t*>(p + lay.vp + 4 * (tid & (ps - 1)));
      }
    }
  };
  // f16 codes into the K tile; the pairs of token tid as floats, column pairs
  // together: s s m m, s' s' m' m'.
  auto store_k = [&](int n) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int tok = x * 64 + warp * 8 + (lane & 7);
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        const int byte = (lane >> 3) * (D / 2) + w * 16;  // of the token's f16 row
        const uint32_t c = (byte % C::SWK) >> 4;
        const uint32_t sw = C::SWK == 128 ? (uint32_t)(tok & 7) : (uint32_t)((tok >> 1) & 3);
        const uint32_t y = kc[x][w], z = y >> 8;
        st_shared_v4(sK + byte / C::SWK * C::BOXK + tok * C::SWK + ((c ^ sw) << 4),
                     y & 0x000f000fu, y & 0x00f000f0u, z & 0x000f000fu, z & 0x00f000f0u);
      }
    }
    if (tid < kBN) {
      float* p = reinterpret_cast<float*>(sm + C::OFF_PAR + (n & 1) * 2048) + (tid >> 1) * 8 +
                 (tid & 1);
      p[0] = bf_lo(kpar);
      p[2] = bf_hi(kpar);
      p[4] = bf_lo(vpar);
      p[6] = bf_hi(vpar);
    }
  };
  // V codes: lane takes dim pair i and 16 tokens, in each half of the tile.
  constexpr int VI = D / 2 / 8;  // warps a half of the tile needs
  auto load_v = [&](int n) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int job = x * 8 + warp, half = job / VI, i = (job % VI) * 8 + (lane & 7);
      const int tok = half * 64 + 16 * (lane >> 3);
#pragma unroll
      for (int w = 0; w < 4; ++w) vc[x][w] = 0;
      if (half < 2) {
        const uint8_t* p = page_of(n, tok);
        if (p) {
          const uint4 y = *reinterpret_cast<const uint4*>(p + lay.v + i * ps + (tok & (ps - 1)));
          vc[x][0] = y.x; vc[x][1] = y.y; vc[x][2] = y.z; vc[x][3] = y.w;
        }
      }
    }
  };
  // bf16 codes into the V tile, rows = dims.  Lanes 0-3 of eight store the even
  // dim first and lanes 4-7 the odd one, which keeps the eight in eight
  // different 16-byte columns of the swizzle.
  auto store_v = [&]() {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int job = x * 8 + warp, half = job / VI, i = (job % VI) * 8 + (lane & 7);
      if (half < 2) {
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
          const int odd = pass ^ ((lane >> 2) & 1), row = 2 * i + odd;
          const uint32_t at = sV + half * C::BOXV + row * 128;
          const uint32_t sh = (4 * odd + 29) & 31;  // nibble to bits 3..6: right by 4 odd - 3
          uint32_t r[8];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t y = __funnelshift_r(vc[x][w], vc[x][w], sh);
            const uint32_t z = __funnelshift_r(vc[x][w], vc[x][w], (sh + 8) & 31);
            r[2 * w] = sub16_bf16x2((y & 0x00780078u) | 0x41804180u);
            r[2 * w + 1] = sub16_bf16x2((z & 0x00780078u) | 0x41804180u);
          }
          const uint32_t c = 2 * (lane >> 3);
          st_shared_v4(at + ((c ^ (row & 7)) << 4), r[0], r[1], r[2], r[3]);
          st_shared_v4(at + (((c + 1) ^ (row & 7)) << 4), r[4], r[5], r[6], r[7]);
        }
      }
    }
  };

  if (nt > 0) {
    load_k(0);
    load_v(0);
  }
  // Q: two threads a row, half of its dims each.
  {
    const int r = tid >> 1, half = tid & 1;
    constexpr int W = D / 4;  // words of a half row
    uint32_t x[W];
    float sum = 0.f, own = 0.f;
    uint32_t most = 0;
    const int64_t row = sq.s0 + r0 + r;
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      uint4 y = make_uint4(0, 0, 0, 0);
      if (r < nr)
        y = *reinterpret_cast<const uint4*>(a.q + row * a.q_rs + h * D + half * (D / 2) + 2 * i);
      x[i] = y.x; x[i + 1] = y.y; x[i + 2] = y.z; x[i + 3] = y.w;
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
      sum += bf_lo(x[i]) + bf_hi(x[i]);
      most = umax(most, umax(x[i] & 0x7fffu, (x[i] >> 16) & 0x7fffu));
    }
    if (r < nr && r0 + r >= sq.h) {
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const uint4 y =
            *reinterpret_cast<const uint4*>(a.k + row * a.k_rs + h * D + half * (D / 2) + 2 * i);
        own = fmaf(bf_lo(x[i]), bf_lo(y.x), fmaf(bf_hi(x[i]), bf_hi(y.x), own));
        own = fmaf(bf_lo(x[i + 1]), bf_lo(y.y), fmaf(bf_hi(x[i + 1]), bf_hi(y.y), own));
        own = fmaf(bf_lo(x[i + 2]), bf_lo(y.z), fmaf(bf_hi(x[i + 2]), bf_hi(y.z), own));
        own = fmaf(bf_lo(x[i + 3]), bf_lo(y.w), fmaf(bf_hi(x[i + 3]), bf_hi(y.w), own));
      }
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    own += __shfl_xor_sync(0xffffffffu, own, 1);
    most = umax(most, __shfl_xor_sync(0xffffffffu, most, 1));
    // as in cache_attn.cu: the row's largest |q| to [2^14, 2^15)
    const int e = imax((int)(most >> 7) - 127, -112);
    const float up = __int_as_float((141 - e) << 23), down = __int_as_float((113 + e) << 23);
    if (half == 0) {
      row_f[r] = down * (0.5f * a.alpha * 16777216.f);
      row_sum[r] = most >= 0x7f80u ? __int_as_float(0x7fc00000) : sum * (0.5f * a.alpha);
      const float z = own * a.alpha;
      row_self[r] = r < nr && r0 + r >= sq.h ? z / (1.f + __expf(-z)) : 0.f;
    }
    const uint32_t sw = C::SWK == 128 ? (uint32_t)(r & 7) : (uint32_t)((r >> 1) & 3);
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const int byte = half * D + 4 * i;
      uint32_t y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float z = j & 1 ? up * 0.0625f : up;
        y[j] = pack_f16x2(bf_lo(x[i + j]) * z, bf_hi(x[i + j]) * z);
      }
      st_shared_v4(sQ + byte / C::SWK * C::BOXK + r * C::SWK +
                       ((((uint32_t)(byte % C::SWK) >> 4) ^ sw) << 4),
                   y[0], y[1], y[2], y[3]);
    }
  }

  const uint64_t dQ = smem_desc(sQ, 16, 8 * C::SWK, C::SWZK);
  const uint64_t dK = smem_desc(sK, 16, 8 * C::SWK, C::SWZK);
  const uint64_t dV = smem_desc(sV, 16, 1024, kSwizzle128B);
  constexpr uint32_t IS = idesc_f16(kBM, kBN), IO = idesc_bf16(kBM, D, false, false);
  // By warp 0, converged; always the same lane issues.
  auto issue_s = [&]() {
    tc_fence_after();
    if (elect_one()) {
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t off = (uint32_t)(((ks * 32) / C::SWK) * C::BOXK + (ks * 32) % C::SWK) >> 4;
        mma_ss(tmem + kColS, dQ + off, dK + off, IS, ks > 0 ? 1u : 0u);
      }
      tc_commit(bar_s);
    }
    __syncwarp();
  };
  auto issue_o = [&](bool first) {
    tc_fence_after();
    if (elect_one()) {
#pragma unroll
      for (int ks = 0; ks < kBN / 16; ++ks)
        mma_ts(tmem + kColO, tmem + kColS + (ks >> 1) * 32 + (ks & 1) * 8,
               dV + ((uint32_t)((ks >> 2) * C::BOXV + (ks & 3) * 32) >> 4), IO,
               ks > 0 || !first ? 1u : 0u);
      tc_commit(bar_o);
    }
    __syncwarp();
  };

  // Rows of this thread: 32 (warp % 4) + g + 8 i; its columns: of its warp's
  // half, those 2t, 2t + 1 of each eight.
  const int quad = warp & 3, chalf = warp >> 2;
  const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
  const CacheFull whole = cache_full(r0, r0 + nr, sq.h, sq.Lh, a.K1, a.K2e);
  uint64_t rest[4] = {0, 0, 0, 0};  // packed pairs of fp32 sums of P m'
  bool ok = true;

  if (nt > 0) {
    store_k(0);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) issue_s();
    const float f[4] = {row_f[quad * 32 + g], row_f[quad * 32 + g + 8], row_f[quad * 32 + g + 16],
                        row_f[quad * 32 + g + 24]};
    const float qs[4] = {row_sum[quad * 32 + g], row_sum[quad * 32 + g + 8],
                         row_sum[quad * 32 + g + 16], row_sum[quad * 32 + g + 24]};
    int n = 0;
    for (; n < nt; ++n) {
      // V of this tile, once the last tile's product has read its own
      if (n > 0) ok = phase_wait(bar_o, (n - 1) & 1, a.t);
      if (ok) {
        store_v();
        fence_proxy_async_smem();
        if (n + 1 < nt) load_k(n + 1);
        if ((n & (kIdTiles - 1)) == 8 && n + kIdTiles - 8 < nt) load_ids(n / kIdTiles + 1);
        ok = phase_wait(bar_s, n & 1, a.t);
      }
      if (!__syncthreads_and(ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const int j0 = tl.at(e0 + n) * kBN;
      const bool full = whole(j0, kBN);
      const float4* par =
          reinterpret_cast<const float4*>(sm + C::OFF_PAR + (n & 1) * 2048) + chalf * 64;
#pragma unroll
      for (int cg = 0; cg < 2; ++cg) {  // 32 columns each
        const uint32_t at = lanes + kColS + chalf * 64 + cg * 32;
        uint32_t s0[16], s1[16];
        tmem_ld_frag(at, s0);
        tmem_ld_frag(at + (16u << 16), s1);
        tmem_ld_wait2(s0, s1);
        uint32_t bits[4] = {0, 0, 0, 0};
        if (!full) {
          // this thread's columns of the 32, per row
          const int jc = j0 + chalf * 64 + cg * 32;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const CacheRow c = cache_row(r0 + imin(quad * 32 + g + 8 * i, nr - 1), sq.h, sq.Lh,
                                         a.K1, a.K2e);
            bits[i] = (range_bits(0, c.pre, jc) | range_bits(c.lo, c.hi, jc)) >> (2 * t);
          }
        }
        uint32_t p0[8], p1[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // 8 columns each
          const float4 kp = par[(cg * 16 + 4 * i + t) * 2];      // s s m m
          const float4 vp = par[(cg * 16 + 4 * i + t) * 2 + 1];  // of V
          const uint64_t ks = f2(__float_as_uint(kp.x), __float_as_uint(kp.y));
          const uint64_t km = f2(__float_as_uint(kp.z), __float_as_uint(kp.w));
          const uint64_t vs = f2(__float_as_uint(vp.x), __float_as_uint(vp.y));
          const uint64_t vm = f2(__float_as_uint(vp.z), __float_as_uint(vp.w));
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint32_t* s = (r < 2 ? s0 : s1) + 4 * i + 2 * (r & 1);
            const uint64_t x =
                f2_fma(f2_mul(f2(s[0], s[1]), f2s(f[r])), ks, f2_mul(km, f2s(qs[r])));
            const uint64_t p = f2_fma(x, f2_tanh(x), x);
            uint64_t pm = f2_mul(p, vm);
            uint32_t pv = f2_bf16(f2_mul(p, vs));
            if (!full) {
              const bool a0 = bits[r] >> (8 * i) & 1u, a1 = bits[r] >> (8 * i + 1) & 1u;
              pv &= (a0 ? 0xffffu : 0u) | (a1 ? 0xffff0000u : 0u);
              pm = f2(a0 ? (uint32_t)pm : 0u, a1 ? (uint32_t)(pm >> 32) : 0u);
            }
            rest[r] = f2_add(rest[r], pm);
            (r < 2 ? p0 : p1)[2 * i + (r & 1)] = pv;
          }
        }
        tmem_st_frag(at, p0);
        tmem_st_frag(at + (16u << 16), p1);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncthreads();
      if (warp == 0) issue_o(n == 0);
      if (n + 1 < nt) {
        store_k(n + 1);
        load_v(n + 1);
        fence_proxy_async_smem();
        __syncthreads();
        if (warp == 0) issue_s();
      }
    }
    // the last product; if a wait gave up, whatever was issued
    if (ok) {
      ok = phase_wait(bar_o, (nt - 1) & 1, a.t);
    } else {
      drain_wait(bar_s, n & 1);
      if (n > 0) drain_wait(bar_o, (n - 1) & 1);
    }
  }
  // rests: a row's four lanes, then the two column halves
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    float x = f2_lo(rest[r]) + f2_hi(rest[r]);
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    if (t == 0) rests[chalf * 128 + quad * 32 + g + 8 * r] = x;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  // Epilogue: lane = row, each column half by its warps, 16 dims at a time.
  {
    const int r = quad * 32 + lane;
    const float rs = rests[r] + rests[128 + r], own = row_self[r];
    const int64_t row = sq.s0 + r0 + r;
    constexpr int CW = D / 2;  // dims of this warp
#pragma unroll
    for (int c = 0; c < CW; c += 16) {
      const int d0 = chalf * CW + c;
      uint32_t o[16];
      if (nt > 0) {
        tmem_ld16(lanes + kColO + d0, o);
        tmem_ld_wait(o);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = 0;
      }
      if (r < nr && S > 1) {
        float4* dst = reinterpret_cast<float4*>(parts + ((int64_t)blockIdx.x * kBM + r) * D + d0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          dst[i] = make_float4(__uint_as_float(o[4 * i]) + rs, __uint_as_float(o[4 * i + 1]) + rs,
                               __uint_as_float(o[4 * i + 2]) + rs,
                               __uint_as_float(o[4 * i + 3]) + rs);
      } else if (r < nr) {
        uint32_t v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        const bool is_cand = r0 + r >= sq.h;
        if (is_cand) {
          const uint4* vp = reinterpret_cast<const uint4*>(a.v + row * a.v_rs + h * D + d0);
          const uint4 y = vp[0], z = vp[1];
          v[0] = y.x; v[1] = y.y; v[2] = y.z; v[3] = y.w;
          v[4] = z.x; v[5] = z.y; v[6] = z.z; v[7] = z.w;
        }
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float x = __uint_as_float(o[2 * i]) + rs, y = __uint_as_float(o[2 * i + 1]) + rs;
          if (is_cand) {
            x = fmaf(own, bf_lo(v[i]), x);
            y = fmaf(own, bf_hi(v[i]), y);
          }
          w[i] = pack_bf16x2(x * a.inv_n, y * a.inv_n);
        }
        uint4* dst = reinterpret_cast<uint4*>(a.out + row * a.o_rs + h * D + d0);
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// The blocks' sums of a unit, in order; the own pair, 1/N, bf16.  A warp takes
// a row at a time.
template <int D>
__global__ void __launch_bounds__(kThreads)
    cache_tc_join_kernel(const __grid_constant__ CacheAttnArgs a, int S, int row_tiles,
                         const float* __restrict__ parts) {
  constexpr int PL = D / 32;  // dims a lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x / 4, bh = unit / row_tiles, r0 = (unit % row_tiles) * kBM;
  const int b = bh / a.H, h = bh % a.H;
  CacheSeq sq;
  if (!cache_seq(a, b, &sq) || r0 >= sq.n || cache_status(a.t) != 0) return;
  const int nr = imin(kBM, sq.n - r0);
  const CacheTiles tl = cache_tiles<kBN>(r0, r0 + nr, sq.h, sq.Lh, a.K1, a.K2e);
  const int bl = (tl.n + S - 1) / S;
  const int used = bl > 0 ? (tl.n + bl - 1) / bl : 1;
  const int end = imin(nr, (int)(blockIdx.x % 4 + 1) * 32);
  for (int r = (int)(blockIdx.x % 4) * 32 + warp; r < end; r += 8) {
    float x[PL], y[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) x[i] = 0.f;
    for (int s = 0; s < used; ++s) {
      const float* p = parts + (((int64_t)unit * S + s) * kBM + r) * D + lane * PL;
      if constexpr (PL == 4) {
        const float4 z = *reinterpret_cast<const float4*>(p);
        y[0] = z.x; y[1] = z.y; y[2] = z.z; y[3] = z.w;
      } else if constexpr (PL == 2) {
        const float2 z = *reinterpret_cast<const float2*>(p);
        y[0] = z.x; y[1] = z.y;
      } else {
        y[0] = *p;
      }
#pragma unroll
      for (int i = 0; i < PL; ++i) x[i] += y[i];
    }
    const int64_t row = sq.s0 + r0 + r;
    const int col = h * D + lane * PL;
    if (r0 + r >= sq.h) {
      float own = 0.f;
#pragma unroll
      for (int i = 0; i < PL; ++i)
        own = fmaf(__bfloat162float(a.q[row * a.q_rs + col + i]),
                   __bfloat162float(a.k[row * a.k_rs + col + i]), own);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) own += __shfl_xor_sync(0xffffffffu, own, o);
      own *= a.alpha;
      own = own / (1.f + __expf(-own));
#pragma unroll
      for (int i = 0; i < PL; ++i)
        x[i] = fmaf(own, __bfloat162float(a.v[row * a.v_rs + col + i]), x[i]);
    }
#pragma unroll
    for (int i = 0; i < PL; ++i) a.out[row * a.o_rs + col + i] = __float2bfloat16(x[i] * a.inv_n);
  }
}

struct TcPlan {
  int row_tiles, S;
  int64_t units;
};

// Two blocks fit an SM; a unit is split until they are all taken, down to two
// tiles a block.
TcPlan tc_plan(const CacheAttnArgs& a) {
  TcPlan p;
  p.row_tiles = (a.max_new + kBM - 1) / kBM;
  p.units = (int64_t)a.t.B * a.H * p.row_tiles;
  const int64_t w = (int64_t)a.K1 + a.K2e + kBM, c = (int64_t)a.t.M * a.t.ps;
  const int64_t tiles = (w < c ? w : c) / kBN + 2;
  int64_t S = p.units > 0 ? (2 * 148 + p.units - 1) / p.units : 1;
  S = S < tiles / 2 ? S : tiles / 2;
  p.S = S < 1 ? 1 : (int)S;
  return p;
}

template <int D>
cudaError_t launch_tc(const CacheAttnArgs& a, float* parts, cudaStream_t st) {
  using C = TcCfg<D>;
  const cudaError_t e = cudaFuncSetAttribute(
      cache_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const TcPlan p = tc_plan(a);
  if (p.units * p.S > 0x7fffffff || p.units * 4 > 0x7fffffff) return cudaErrorInvalidValue;
  cache_tc_kernel<D><<<(unsigned)(p.units * p.S), kThreads, C::SMEM, st>>>(a, p.S, p.row_tiles,
                                                                         parts);
  if (p.S > 1)
    cache_tc_join_kernel<D><<<(unsigned)(p.units * 4), kThreads, 0, st>>>(a, p.S, p.row_tiles,
                                                                         parts);
  return cudaGetLastError();
}

}  // namespace

size_t cache_tc_ws_bytes(const CacheAttnArgs& a, int d) {
  const TcPlan p = tc_plan(a);
  return p.S == 1 ? 256 : align256((size_t)p.units * p.S * kBM * d * sizeof(float));
}

cudaError_t launch_cache_tc(const CacheAttnArgs& a, int d, void* ws, cudaStream_t st) {
  float* parts = static_cast<float*>(ws);
  if (d == 32) return launch_tc<32>(a, parts, st);
  if (d == 64) return launch_tc<64>(a, parts, st);
  return launch_tc<128>(a, parts, st);
}

}  // namespace hstu
