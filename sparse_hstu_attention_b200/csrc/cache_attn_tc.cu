// SLA HSTU attention of many new rows per sequence over the 4-bit history cache
// (include/hstu_cache.h) on the 5th-generation tensor cores: candidate sets,
// chunks of history.
//
// The algebra is cache_attn.cu's: with k_j = m + s c and v_j = m' + s' c',
//   x_ij = alpha (s_j (q_i . c_j) + m_j sum(q_i)),  P = SiLU(x),
//   out_i = (1/N) (sum_j (P_ij s'_j) c'_j + sum_j P_ij m'_j  [+ own pair]),
// so what a masked place holds never enters a product: its P is selected to
// zero, its codes are finite.  K codes are the f16 subnormals c 2^-24 and
// 16 c 2^-24 there; V codes are the bf16 numbers c / 64, because P s' is a bf16
// operand: a row's P may span more than f16's range, and the sums O stay in
// TMEM, where rescaling them would cost a pass.  That rounding of P s' to bf16
// (up to 2^-8 of itself) is the coarsest, then tanh's instruction (about 2^-11); over 640
// visible keys of SiLU'd rows they add 3e-4 of the output to bf16's own 1.65e-3, both
// root mean squares.  q enters as f16 times
// 2^4, its dims of the high nibbles divided by 16: exact for rows whose largest
// |q| lies in [2^-6, 2^11), down to 2^-12 of that largest; if a block has
// another row, its rows are scaled by a power of two each, and the scores back.
//
// A block is one (sequence, head, 128 rows), possibly a part of its keys, 8
// warps, and two blocks share an SM: S = Q C^T (M = 128, N = 128 keys, K = d)
// and O += P C' (N = d, K = 128) by tcgen05 into 128 + d TMEM columns.  All warps
// do the same things in turn, and one block's products, loads and output run
// under the other's arithmetic:
//   V codes of tile n  -> shared memory     while S of tile n runs
//   wait S; P = SiLU(x) masked, P s' -> TMEM over the scores; issue O += P C'
//   K codes of tile n+1 -> shared memory    while that runs; issue S of n + 1
// Codes come straight from the pages into registers, 16 bytes a thread, a tile
// before they are unpacked; the unpacked operands are K-major 128-byte swizzled
// tiles (V transposed: its bytes lie along the tokens).  Scores are read from
// TMEM as 16 x 256-bit fragments: a thread has 4 rows and a quarter of the
// columns, so the per-key pairs are one 16-byte load per two columns and four
// rows.  The loop over 16-column pieces is unrolled by two: by four it is 3% quicker
// at d = 64, 1% slower at d = 128 and spills there; rolled up, 1 to 4% slower.
//
// Tiles at an edge of the masks are done in 16-column pieces of 32 rows each: whole
// ones as inside, ones that no row sees as zeros, and only the others with masks (700
// rows over a 1024-token window: 84 us without, 74 so).
//
// Bound: latency and issue slots.  A 128 x 128 tile takes some 5500 warp instructions
// at d = 128, half of them on the scores and a third on unpacking, and 1.52 us of an
// SM (48% of the slots; 1.2 us at d = 64); the special-function unit's part (one tanh
// a score) is 0.55 us, the products' as long.  Two blocks of 8 warps with 128
// registers are what an SM holds.  64 sequences x 4 heads x 512 candidates under a
// 512-token window: 92 us; 4 x 4 x 1000 over up to 16K tokens: 123 us; 16 x 8 heads of
// 64, 716 rows over a 1024-token window: 74 us.
#include <type_traits>

#include "cache_common.cuh"
#include "sm100.cuh"

namespace hstu {

namespace {

using namespace sm100;

constexpr int kThreads = 256, kBM = 128, kBN = 128;
constexpr int kIdTiles = 32;  // tiles whose page blocks are held at a time
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
  static constexpr int OFF_ROW = OFF_PAR + 2 * 64 * 32;  // per row: factor, sum(q), own pair
  static constexpr int OFF_REST = OFF_ROW + 3 * 128 * 4;  // [2][128]
  static constexpr int OFF_IDS = OFF_REST + 2 * 128 * 4;  // [2][kIdTiles * 8] page blocks
  static constexpr int OFF_BAR = OFF_IDS + 2 * kIdTiles * 8 * 8;
  static constexpr int NEED = OFF_BAR + 32 + 1024;     // + alignment slack
  // two blocks an SM, no more: their TMEM columns are all there are
  static constexpr int SMEM = NEED > 80 * 1024 ? NEED : 80 * 1024;
  static_assert(SMEM <= 113 * 1024, "two blocks an SM");
  static constexpr uint32_t SWZK = SWK == 128 ? kSwizzle128B : kSwizzle64B;
};

// kind::f16 with f16 A / B (format 0) and f32 accumulator, both K-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// 16 lanes x 16 columns: regs 4i .. 4i + 3 are row g, columns 8i + 2t, + 1, and
// row g + 8, the same columns.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}
// Waits for two of them.
__device__ __forceinline__ void tmem_ld_frag_wait(uint32_t (&r)[8], uint32_t (&s)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(s[0]), "+r"(s[1]), "+r"(s[2]), "+r"(s[3]),
                 "+r"(s[4]), "+r"(s[5]), "+r"(s[6]), "+r"(s[7])
               :
               : "memory");
}
// 16 lanes x 8 columns: regs 2i, 2i + 1 are rows g and g + 8, column 4i + t.
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_f16x2(float x, float y) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// Bounded wait for the phase of parity `parity`: false after kWaitLimitNs.  A
// try may sleep for up to 10 us, so that waiting warps leave the issue slots to
// the others.
__device__ __forceinline__ bool try_wait_long(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(10000u)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool phase_wait(uint32_t bar, uint32_t parity, const CacheTab& t) {
  if (try_wait_long(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (!try_wait_long(bar, parity)) {
    if (globaltimer() - t0 > kWaitLimitNs) {
      cache_fail(t, HSTU_SLA_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool some) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(some ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "r"(a)
               : "memory");
  return x;
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

  const int status = cache_status(a.t);
  CacheSeq sq;
  if (!cache_seq(a, b, &sq) || r0 >= sq.n) return;
  // (one status for the whole block, so that its threads part ways together)
  if (__syncthreads_or(status != 0)) return;
  const int nr = imin(kBM, sq.n - r0);
  const CacheTiles tl = cache_tiles<kBN>(r0, r0 + nr, sq.h, sq.Lh, a.K1, a.K2e);
  const int bl = (tl.n + S - 1) / S;
  const int e0 = imin(split * bl, tl.n), nt = imin(bl, tl.n - e0);
  if (split > 0 && nt <= 0) return;

  const uint32_t sQ = base + C::OFF_Q, sK = base + C::OFF_K, sV = base + C::OFF_V;
  const uint32_t bar_s = base + C::OFF_BAR, bar_o = bar_s + 8;
  uint32_t* const slot = reinterpret_cast<uint32_t*>(sm + C::OFF_BAR + 16);
  float* const rd = reinterpret_cast<float*>(sm + C::OFF_ROW);
  float* const rests = reinterpret_cast<float*>(sm + C::OFF_REST);
  const uint8_t** const blocks = reinterpret_cast<const uint8_t**>(sm + C::OFF_IDS);

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

  // This head's block of the pages of tiles [32 c, 32 c + 32), an entry a thread: its
  // id, and its address into the table.  Places past the cached tokens get page 0's:
  // what is read there is masked.
  auto read_id = [&](int c) -> int {
    const int n = c * kIdTiles + (tid >> lpt);
    if (tid >= kIdTiles << lpt || n >= nt) return 0;
    const int i = (tl.at(e0 + n) << lpt) + (tid & ((1 << lpt) - 1));
    return i < pages ? bt[i] : 0;
  };
  auto put_id = [&](int c, int id) {
    if (tid >= kIdTiles << lpt) return;
    if (id < 0 || id >= a.t.P) {
      cache_fail(a.t, HSTU_SLA_ERR_BAD_INPUT);
      id = 0;
    }
    blocks[(c & 1) * (kIdTiles * 8) + tid] = head + id * a.page_stride;
  };
  // Table entry of the first page of tile n.
  auto entry = [&](int n) -> const uint8_t* const* {
    return blocks + ((n / kIdTiles) & 1) * (kIdTiles * 8) + ((n % kIdTiles) << lpt);
  };
  const int id0 = read_id(0);
  // The rows of q and the candidates' k as they are into the Q and K tiles, D / 8
  // lanes a row; the candidates' v on its way to L2 (0.4 us of 92).
  const int cand = sq.h - r0;  // first candidate row of the block
  auto row_at = [&](int r, int c) -> uint32_t {  // 16-byte piece c of row r
    const uint32_t sw = C::SWK == 128 ? (uint32_t)(r & 7) : (uint32_t)((r >> 1) & 3);
    const int byte = 16 * c;
    return byte / C::SWK * C::BOXK + r * C::SWK +
           ((((uint32_t)(byte % C::SWK) >> 4) ^ sw) << 4);
  };
  {
    constexpr int LPR = D / 8, RPI = 32 / LPR;
    const int ch = lane % LPR, rw = warp * 16 + lane / LPR;
    const int64_t row0 = sq.s0 + r0;
#pragma unroll
    for (int i = 0; i < 16 / RPI; ++i) {
      const int r = rw + i * RPI;
      const bool in = r < nr;
      cp_async16(sQ + row_at(r, ch), in ? a.q + (row0 + r) * a.q_rs + h * D + ch * 8 : a.q, in);
      if (in && r >= cand)
        cp_async16(sK + row_at(r, ch), a.k + (row0 + r) * a.k_rs + h * D + ch * 8, true);
    }
    const int r = tid >> 1;
    if (S == 1 && r >= cand && r < nr)
      prefetch_l2(a.v + (row0 + r) * a.v_rs + h * D + (tid & 1) * (D / 2));
  }
  put_id(0, id0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;

  const float fac = 0.5f * a.alpha * 1048576.f;  // codes 2^-24, q 2^4
  // K codes: lane takes token 8 (..) + lane % 8 and D / 8 of its bytes, of the
  // tile's first 64 tokens and of the others (the same place, other pages).
  uint32_t kc[2][4], vc[2][4], kpar = 0, vpar = 0;
  const int ktok = warp * 8 + (lane & 7), kq = lane >> 3;
  const int k_page = ktok >> lps, k_off = (ktok & (ps - 1)) * (D / 2) + kq * (D / 8);
  const int par_page = tid >> lps, par_off = lay.kp + 4 * (tid & (ps - 1));
  auto load_k = [&](int n) {
    const uint8_t* const* e = entry(n);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint8_t* p = e[k_page + (x ? 64 >> lps : 0)] + k_off;
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
    if (tid < kBN) {
      const uint8_t* p = e[par_page] + par_off;
      kpar = *reinterpret_cast<const uint32_t*>(p);
      vpar = *reinterpret_cast<const uint32_t*>(p + 4 * ps);
    }
  };
  // f16 codes into the K tile; the pairs of token tid as floats, column pairs
  // together: s s m m, s' s' m' m'.
  uint32_t k_at;  // where the lane's first 16 bytes go (the next: xor 16, 32, 48)
  {
    const int byte = kq * (D / 2);  // of the token's f16 row
    const uint32_t sw = C::SWK == 128 ? (uint32_t)(ktok & 7) : (uint32_t)((ktok >> 1) & 3);
    k_at = sK + byte / C::SWK * C::BOXK + ktok * C::SWK + ((((byte % C::SWK) >> 4) ^ sw) << 4);
  }
  const uint32_t par_at = (uint32_t)(tid >> 1) * 32 + (tid & 1) * 4;
  auto store_k = [&](int n) {
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        const uint32_t y = kc[x][w], z = y >> 8;
        st_shared_v4((k_at ^ (w << 4)) + x * 64 * C::SWK, y & 0x000f000fu, y & 0x00f000f0u,
                     z & 0x000f000fu, z & 0x00f000f0u);
      }
    if (tid < kBN) {
      float* p = reinterpret_cast<float*>(sm + C::OFF_PAR + (n & 1) * 2048 + par_at);
      p[0] = bf_lo(kpar) * fac;
      p[2] = bf_hi(kpar);
      p[4] = bf_lo(vpar) * 64.f;
      p[6] = bf_hi(vpar);
    }
  };
  // V codes: lane takes a dim pair and 16 tokens: D / 16 warps cover 64 tokens,
  // so at d = 128 a warp has its place in either half of the tile, and at less
  // the first D / 8 warps have one.
  constexpr int VI = D / 16, VX = D == 128 ? 2 : 1;
  const bool v_warp = D == 128 || warp < 2 * VI;
  const int v_half = D == 128 ? 0 : warp / VI, v_i = (warp % VI) * 8 + (lane & 7);
  const int v_tok = v_half * 64 + 16 * (lane >> 3);
  const int v_page = v_tok >> lps, v_off = lay.v + v_i * ps + (v_tok & (ps - 1));
  auto load_v = [&](int n) {
    const uint8_t* const* e = entry(n);
    if (!v_warp) return;
#pragma unroll
    for (int x = 0; x < VX; ++x) {
      const uint4 y =
          *reinterpret_cast<const uint4*>(e[v_page + (x ? 64 >> lps : 0)] + v_off);
      vc[x][0] = y.x; vc[x][1] = y.y; vc[x][2] = y.z; vc[x][3] = y.w;
    }
  };
  // bf16 codes / 64 into the V tile, rows = dims.  Lanes 0-3 of eight store the even
  // dim first and lanes 4-7 the odd one, which keeps the eight in eight
  // different 16-byte columns of the swizzle.
  const uint32_t v_odd = (lane >> 2) & 1;
  const uint32_t v_row = 2 * v_i + v_odd;
  const uint32_t v_at = sV + v_half * C::BOXV + v_row * 128 + (((2 * (lane >> 3)) ^ (v_row & 7)) << 4);
  // A nibble in bits 0..3 of a half is the bf16 number c 2^-133, in bits 4..7
  // c 2^-129 (c < 8 subnormal, above normal, one line): times 2^127 or 2^123
  // both are c / 64, exactly.
  const uint32_t v_mask[2] = {v_odd ? 0x00f000f0u : 0x000f000fu,
                              v_odd ? 0x000f000fu : 0x00f000f0u};
  const uint32_t v_mul[2] = {v_odd ? 0x7d007d00u : 0x7f007f00u,
                             v_odd ? 0x7f007f00u : 0x7d007d00u};
  auto store_v = [&]() {
    if (!v_warp) return;
#pragma unroll
    for (int x = 0; x < VX; ++x)
#pragma unroll
      for (int pass = 0; pass < 2; ++pass) {
        // the other dim of the pair: row ^ 1, and so its chunks' places ^ 1
        const uint32_t at = (pass ? v_at ^ 144u : v_at) + x * C::BOXV;
        uint32_t r[8];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          r[2 * w] = mul_bf16x2(vc[x][w] & v_mask[pass], v_mul[pass]);
          r[2 * w + 1] = mul_bf16x2((vc[x][w] >> 8) & v_mask[pass], v_mul[pass]);
        }
        st_shared_v4(at, r[0], r[1], r[2], r[3]);
        st_shared_v4(at ^ 16u, r[4], r[5], r[6], r[7]);
      }
  };

  if (nt > 0) {
    load_k(0);
    load_v(0);
  }
  cp_async_wait();
  __syncthreads();
  // q into f16, in place: two lanes a row.
  bool common;
  {
    constexpr int NP = D / 16;  // pieces a lane
    const int r = warp * 16 + (lane & 15), c0 = (lane >> 4) * NP;
    // 16 bytes of f16: q times up; the dims of high nibbles over 16
    auto put_q = [&](int c, const uint4& y, float up) {
      const float hi = up * 0.0625f;
      st_shared_v4(sQ + row_at(r, c), pack_f16x2(bf_lo(y.x) * up, bf_hi(y.x) * up),
                   pack_f16x2(bf_lo(y.y) * hi, bf_hi(y.y) * hi),
                   pack_f16x2(bf_lo(y.z) * up, bf_hi(y.z) * up),
                   pack_f16x2(bf_lo(y.w) * hi, bf_hi(y.w) * hi));
    };
    const bool is_cand = r >= cand && r < nr;
    float sum = 0.f, own = 0.f;
    uint32_t most = 0;
#pragma unroll 4
    for (int i = 0; i < NP; ++i) {
      const uint4 q = ld_shared_v4(sQ + row_at(r, c0 + i));
      uint4 k = make_uint4(0, 0, 0, 0);
      if (is_cand) k = ld_shared_v4(sK + row_at(r, c0 + i));
      const uint32_t w[4] = {q.x, q.y, q.z, q.w}, z[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sum += bf_lo(w[j]) + bf_hi(w[j]);
        own = fmaf(bf_lo(w[j]), bf_lo(z[j]), fmaf(bf_hi(w[j]), bf_hi(z[j]), own));
        most = umax(most, umax(w[j] & 0x7fffu, (w[j] >> 16) & 0x7fffu));
      }
      put_q(c0 + i, q, 16.f);
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
    own += __shfl_xor_sync(0xffffffffu, own, 16);
    most = umax(most, __shfl_xor_sync(0xffffffffu, most, 16));
    // most in [2^-6, 2^11), or a row of zeros: 2^4 will do; else the row's largest
    // goes to [2^14, 2^15) (values below 2^-112: times 2^126)
    const bool fits = most == 0 || (most >= 121u << 7 && most < 138u << 7);
    const int e = imax((int)(most >> 7) - 127, -112);
    const float scale = __int_as_float(imin(117 + e, 254) << 23);  // 2^(e - 10)
    if (lane < 16) {
      rd[r] = scale;
      rd[128 + r] = most >= 0x7f80u ? __int_as_float(0x7fc00000) : sum * (0.5f * a.alpha);
      const float y = own * a.alpha;
      rd[256 + r] = is_cand ? __fdividef(y, 1.f + __expf(-y)) : 0.f;
    }
    common = __syncthreads_and(fits);
    if (!common) {  // 2^(14 - e) for each row
      const bf16* const qp = a.q + (int64_t)(sq.s0 + r0 + r) * a.q_rs + h * D;
#pragma unroll 1
      for (int i = 0; i < NP; ++i) {
        uint4 y = make_uint4(0, 0, 0, 0);
        if (r < nr) y = *reinterpret_cast<const uint4*>(qp + 8 * (c0 + i));
        put_q(c0 + i, y, 16.f / scale);
      }
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
  // rows [q0, q1) are this warp's
  const int q0 = r0 + quad * 32, q1 = imin(q0 + 32, r0 + nr);
  const CacheFull whole = cache_full(q0, q1, sq.h, sq.Lh, a.K1, a.K2e);
  uint64_t rest[4] = {0, 0, 0, 0};  // packed pairs of fp32 sums of P m'
  bool ok = true;
  int n = 0;

  if (nt > 0) {
    store_k(0);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) issue_s();
    const uint64_t qs[4] = {f2s(rd[128 + quad * 32 + g]), f2s(rd[128 + quad * 32 + g + 8]),
                            f2s(rd[128 + quad * 32 + g + 16]),
                            f2s(rd[128 + quad * 32 + g + 24])};
    for (; n < nt; ++n) {
      // V of this tile, once the last tile's product has read its own
      if (n > 0) ok = phase_wait(bar_o, (n - 1) & 1, a.t);
      if (ok) {
        store_v();
        fence_proxy_async_smem();
        if (n + 1 < nt) {
          load_k(n + 1);
          load_v(n + 1);
        }
        if ((n & (kIdTiles - 1)) == 8 && n + kIdTiles - 8 < nt)
          put_id(n / kIdTiles + 1, read_id(n / kIdTiles + 1));
        ok = phase_wait(bar_s, n & 1, a.t);
      }
      if (!__syncthreads_and(ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const int j0 = tl.at(e0 + n) * kBN;
      const ulonglong2* par =
          reinterpret_cast<const ulonglong2*>(sm + C::OFF_PAR + (n & 1) * 2048) + chalf * 64;
      // 16 columns.  FAST: every pair visible, one factor for all rows (in the steps s)
      auto piece = [&](auto fast, int cg) {
        constexpr bool FAST = decltype(fast)::value;
        const uint32_t at = lanes + kColS + chalf * 64 + cg * 16;
        uint32_t s0[8], s1[8];
        tmem_ld_frag(at, s0);
        tmem_ld_frag(at + (16u << 16), s1);
        tmem_ld_frag_wait(s0, s1);
        uint32_t bits[4];
        float f[4];
        if constexpr (!FAST) {
          // this thread's columns of the 16, per row
          const int jc = j0 + chalf * 64 + cg * 16;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const CacheRow c = cache_row(imin(q0 + g + 8 * i, q1 - 1), sq.h, sq.Lh, a.K1, a.K2e);
            bits[i] = (range_bits(0, c.pre, jc) | range_bits(c.lo, c.hi, jc)) >> (2 * t);
            f[i] = common ? 1.f : rd[quad * 32 + g + 8 * i];
          }
        }
        uint32_t p0[4], p1[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // 8 columns each
          const ulonglong2 kp = par[(cg * 8 + 4 * i + t) * 2];      // s s, m m
          const ulonglong2 vp = par[(cg * 8 + 4 * i + t) * 2 + 1];  // of V
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint32_t* s = (r < 2 ? s0 : s1) + 4 * i + 2 * (r & 1);
            uint64_t y = f2(s[0], s[1]);
            if constexpr (!FAST) y = f2_mul(y, f2s(f[r]));
            y = f2_fma(y, kp.x, f2_mul(kp.y, qs[r]));
            const uint64_t p = f2_fma(y, f2_tanh(y), y);
            uint32_t pv = f2_bf16(f2_mul(p, vp.x));
            if constexpr (FAST) {
              rest[r] = f2_fma(p, vp.y, rest[r]);
            } else {
              const bool a0 = bits[r] >> (8 * i) & 1u, a1 = bits[r] >> (8 * i + 1) & 1u;
              pv &= (a0 ? 0xffffu : 0u) | (a1 ? 0xffff0000u : 0u);
              const uint64_t pm = f2_mul(p, vp.y);
              rest[r] = f2_add(rest[r],
                               f2(a0 ? (uint32_t)pm : 0u, a1 ? (uint32_t)(pm >> 32) : 0u));
            }
            (r < 2 ? p0 : p1)[2 * i + (r & 1)] = pv;
          }
        }
        // P of columns [32 c, 32 c + 32) in columns [32 c, 32 c + 16)
        const uint32_t to = lanes + kColS + chalf * 64 + (cg >> 1) * 32 + (cg & 1) * 8;
        tmem_st_frag(to, p0);
        tmem_st_frag(to + (16u << 16), p1);
      };
      const int jw = j0 + chalf * 64;  // the warp's columns
      if (common && q0 < q1 && whole(jw, 64)) {
#pragma unroll 2
        for (int cg = 0; cg < 4; ++cg) piece(std::true_type{}, cg);
      } else {
        // an edge of the masks (or rows of differing scales): pieces that no row of
        // the warp sees are zeros
        const CacheRow lo = cache_row(q0, sq.h, sq.Lh, a.K1, a.K2e);
        const CacheRow hi = cache_row(q1 - 1, sq.h, sq.Lh, a.K1, a.K2e);
#pragma unroll 1
        for (int cg = 0; cg < 4; ++cg) {
          const int jc = jw + cg * 16;
          if (q0 >= q1 || (jc >= hi.pre && (jc + 16 <= lo.lo || jc >= hi.hi))) {
            const uint32_t zero[4] = {0, 0, 0, 0};
            const uint32_t to = lanes + kColS + chalf * 64 + (cg >> 1) * 32 + (cg & 1) * 8;
            tmem_st_frag(to, zero);
            tmem_st_frag(to + (16u << 16), zero);
          } else if (common && whole(jc, 16)) {
            piece(std::true_type{}, cg);
          } else {
            piece(std::false_type{}, cg);
          }
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncthreads();
      if (warp == 0) issue_o(n == 0);
      if (n + 1 < nt) {
        store_k(n + 1);
        fence_proxy_async_smem();
        __syncthreads();
        if (warp == 0) issue_s();
      }
    }
  }
  // The candidates' v (see below): all loads before the first use.
  constexpr int NA = D >= 64 ? 2 : 1, NC = D == 128 ? 2 : 1;
  uint4 vv[NA * NC][2];
#pragma unroll
  for (int i = 0; i < NA * NC * 2; ++i) {
    const int la = D >= 64 ? (i >> 1) / NC : chalf;
    const int c0 = D >= 64 ? (chalf * NC + (i >> 1) % NC) * 32 : 0;
    const int r = quad * 32 + 16 * la + 8 * (i & 1) + g;
    vv[i >> 1][i & 1] = make_uint4(0, 0, 0, 0);
    if (S == 1 && r >= cand && r < nr)
      vv[i >> 1][i & 1] = *reinterpret_cast<const uint4*>(
          a.v + (int64_t)(sq.s0 + r0 + r) * a.v_rs + h * D + c0 + 8 * t);
  }
  // rests: a row's four lanes, then the two column halves
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    float x = f2_lo(rest[r]) + f2_hi(rest[r]);
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    if (t == 0) rests[chalf * 128 + quad * 32 + g + 8 * r] = x;
  }
  // the last product; if a wait gave up, whatever was issued
  if (nt > 0) {
    if (ok) {
      ok = phase_wait(bar_o, (nt - 1) & 1, a.t);
    } else {
      drain_wait(bar_s, n & 1);
      if (n > 0) drain_wait(bar_o, (n - 1) & 1);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  // Out: O as 16 x 256-bit fragments, turned among the four lanes of a row so that
  // each has 8 dims in a row (16 bytes of bf16; 64 bytes a row and 8 rows an
  // instruction).  A warp has its quarter's rows and half of the dims, at d = 32
  // half of the rows.
  {
    const int64_t row0 = sq.s0 + r0;
#pragma unroll
    for (int ac = 0; ac < NA * NC; ++ac) {
      const int la = D >= 64 ? ac / NC : chalf;                 // 16 lanes of the quarter
      const int c0 = D >= 64 ? (chalf * NC + ac % NC) * 32 : 0;  // 32 dims
      uint32_t oa[8], ob[8];
      if (nt > 0) {
        const uint32_t at = lanes + ((uint32_t)(16 * la) << 16) + kColO + c0;
        tmem_ld_frag(at, oa);
        tmem_ld_frag(at + 16, ob);
        tmem_ld_frag_wait(oa, ob);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) oa[i] = ob[i] = 0;
      }
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        // y[2 i], y[2 i + 1]: dims 8 i + 2 t, + 1 -> after the turn 8 t + 2 i, + 1
        uint32_t y[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          y[2 * i] = oa[4 * i + 2 * hr];
          y[2 * i + 1] = oa[4 * i + 2 * hr + 1];
          y[4 + 2 * i] = ob[4 * i + 2 * hr];
          y[5 + 2 * i] = ob[4 * i + 2 * hr + 1];
        }
#pragma unroll
        for (int st = 1; st < 4; st <<= 1)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i & st) continue;
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              uint32_t& lo = y[2 * i + z];
              uint32_t& hi = y[2 * (i + st) + z];
              const uint32_t got = __shfl_xor_sync(0xffffffffu, t & st ? lo : hi, st);
              if (t & st) lo = got; else hi = got;
            }
          }
        const int r = quad * 32 + 16 * la + 8 * hr + g;  // row of the block
        if (r >= nr) continue;
        const float rs = nt > 0 ? rests[r] + rests[128 + r] : 0.f;
        if (S > 1) {
          float4* dst = reinterpret_cast<float4*>(
              parts + ((int64_t)blockIdx.x * kBM + r) * D + c0 + 8 * t);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            dst[i] = make_float4(__uint_as_float(y[4 * i]) + rs, __uint_as_float(y[4 * i + 1]) + rs,
                                 __uint_as_float(y[4 * i + 2]) + rs,
                                 __uint_as_float(y[4 * i + 3]) + rs);
          continue;
        }
        const uint32_t v[4] = {vv[ac][hr].x, vv[ac][hr].y, vv[ac][hr].z, vv[ac][hr].w};
        const bool is_cand = r >= cand;
        const float own = rd[256 + r];
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float y0 = __uint_as_float(y[2 * i]) + rs, y1 = __uint_as_float(y[2 * i + 1]) + rs;
          if (is_cand) {
            y0 = fmaf(own, bf_lo(v[i]), y0);
            y1 = fmaf(own, bf_hi(v[i]), y1);
          }
          w[i] = pack_bf16x2(y0 * a.inv_n, y1 * a.inv_n);
        }
        *reinterpret_cast<uint4*>(a.out + (row0 + r) * a.o_rs + h * D + c0 + 8 * t) =
            make_uint4(w[0], w[1], w[2], w[3]);
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
  wait_for_the_last_kernel();
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

// Two blocks fit an SM.  A unit is split while all its parts still run at once, down
// to two tiles each, and further, down to 16 tiles each, until there are half as many
// again, which evens out histories of differing lengths (4 x 4 heads x 8 row tiles
// over up to 128 key tiles: 262 us unsplit, 178 in 2, 136 in 3, 126 in 4, 135 in 5).
// Units of few tiles stay whole (64 x 4 x 4 row tiles over 5 key tiles: 105 us, 203
// in 2).
TcPlan tc_plan(const CacheAttnArgs& a) {
  TcPlan p;
  p.row_tiles = (int)((a.max_new + (int64_t)kBM - 1) / kBM);
  p.units = cache_units(a, kBM);
  const int64_t w = (int64_t)a.K1 + a.K2e + kBM, c = (int64_t)a.t.M * a.t.ps;
  const int64_t tiles = (w < c ? w : c) / kBN + 2;
  const int64_t slots = 2 * kSMs, n = p.units > 0 ? p.units : 1;
  int64_t fill = slots / n;
  fill = fill < tiles / 2 ? fill : tiles / 2;
  int64_t even = (slots * 3 / 2 + n - 1) / n;
  even = even < tiles / 16 ? even : tiles / 16;
  const int64_t S = fill > even ? fill : even;
  p.S = S < 1 ? 1 : (int)S;
  return p;
}

template <int D>
cudaError_t launch_tc(const CacheAttnArgs& a, float* parts, cudaStream_t st) {
  using C = TcCfg<D>;
  const TcPlan p = tc_plan(a);
  if (p.units > 0x7fffffff / 4 / p.S) return cudaErrorNotSupported;
  const cudaError_t e = cudaFuncSetAttribute(
      cache_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  cache_tc_kernel<D><<<(unsigned)(p.units * p.S), kThreads, C::SMEM, st>>>(a, p.S, p.row_tiles,
                                                                         parts);
  const cudaError_t launched = cudaGetLastError();
  if (launched != cudaSuccess || p.S == 1) return launched;
  return launch_early(cache_tc_join_kernel<D>, (unsigned)(p.units * 4), 256, st, a, p.S,
                      p.row_tiles, (const float*)parts);
}

}  // namespace

size_t cache_tc_ws_bytes(const CacheAttnArgs& a, int d) {
  const TcPlan p = tc_plan(a);
  return p.S == 1 ? 0 : align256((size_t)p.units * p.S * kBM * d * sizeof(float));
}

cudaError_t launch_cache_tc(const CacheAttnArgs& a, int d, void* ws, cudaStream_t st) {
  float* parts = static_cast<float*>(ws);
  if (d == 32) return launch_tc<32>(a, parts, st);
  if (d == 64) return launch_tc<64>(a, parts, st);
  return launch_tc<128>(a, parts, st);
}

}  // namespace hstu
