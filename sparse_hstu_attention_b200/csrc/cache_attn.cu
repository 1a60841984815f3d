// SLA HSTU attention of a few new rows per sequence over the 4-bit history
// cache (include/hstu_cache.h): one event per user, or a few rows.
//
//   out_i = (1/N) sum_j M(i,j) SiLU(alpha q_i . k_j) v_j,   k_j, v_j = m + s c
//
// The codes go to the tensor cores as whole numbers and the (s, m) pairs are
// applied to the scores and the probabilities, where they are one per key:
//   q . k_j = s_j (q . c_j) + m_j sum(q)
//   out     = sum_j (P_ij s_j) c_j + sum_j P_ij m_j.
// A nibble becomes the bf16 value 16 + c by one shift and one and-or (bits 3..6
// of 16.0's mantissa), so the 16s are taken off in the same two places:
//   x_j  = s_j (q . (16 + c_j)) + (m_j - 16 s_j) sum(q)
//   out  = sum_j P'_j (16 + c_j) + sum_j (P_j m_j - 16 P'_j),  P' = bf16(P s).
// P' is the only rounding to fewer bits than fp32 (the matrix instruction takes
// bf16), and its 16 is taken off as rounded, so it costs one bf16 rounding of
// P_j s_j against c_j, no more.  Masked pairs are selected to zero before any
// product, so nothing in a masked place reaches a row.
//
// A unit is one (sequence, head, 16 rows); its key tiles of 64 tokens are split
// over a cluster of S blocks and there over the warps.  Each warp streams its
// tiles through its own ring of bulk copies (one per page: a head's codes and
// pairs of a page are contiguous) and keeps everything in registers: S by
// m16n8k16 with the codes as B operand, P, and O += P' V the same way.  SiLU
// attention has no softmax, so partial results only add: warps through shared
// memory, blocks through distributed shared memory, both in a fixed order.
//
// Which key a matrix column stands for is free, so it is chosen for the loads:
// columns 2t, 2t + 1 of score tiles (u, 0) and (u, 1) are tokens 16 t + 4 u
// + {0, 1} and {2, 3}; a thread's K bytes (its quarter of d) and V bytes (16
// tokens of a dim pair) are then single 16-byte loads, without bank conflicts.
//
// Bound: HBM for long histories (d + 8 bytes per token and head).
#include <cooperative_groups.h>

#include "cache_common.cuh"
#include "sm100.cuh"

namespace hstu {

namespace {

using namespace sm100;
namespace cg = cooperative_groups;

constexpr int kW = 4, kThreads = 32 * kW, kRows = 16, kTK = 64, kStages = 2;

template <int D>
struct StepCfg {
  // a stage holds the tile's 1, 2 or 4 page blocks, each page_size * 2 bytes
  // further apart when there are several, so that a warp's V loads from them
  // fall into different banks
  static constexpr int STG = kTK * (D + 8) + 128;
  static constexpr int OFF_SELF = kW * kStages * STG;
  static constexpr int OFF_BAR = OFF_SELF + kRows * 4;
  static constexpr int SMEM = OFF_BAR + kW * kStages * 8;
  static_assert(kStages * STG >= kRows * D * 4, "a warp's result fits its ring");
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

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Nibbles P and P + 4 of w as a bf16 pair 16 + c.
template <int P>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  const uint32_t x = P == 0 ? w << 3 : w >> (4 * P - 3);
  return (x & 0x00780078u) | 0x41804180u;
}

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

template <int D>
__global__ void __launch_bounds__(kThreads, 3)
    cache_step_kernel(const __grid_constant__ CacheAttnArgs a, int S, int row_tiles) {
  using C = StepCfg<D>;
  constexpr int KS = D / 16, WD = D / 32;  // k-steps of q . k, words of a thread's K quarter
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int split = (int)blockIdx.x % S;
  const int unit = (int)blockIdx.x / S;
  const int bh = unit / row_tiles, r0 = (unit % row_tiles) * kRows;
  const int b = bh / a.H, h = bh % a.H;

  // (every block of a cluster takes the same way out)
  CacheSeq sq;
  if (!cache_seq(a, b, &sq) || r0 >= sq.n) return;
  const int nr = imin(kRows, sq.n - r0);
  CacheTiles tl = cache_tiles<kTK>(r0, r0 + nr, sq.h, sq.Lh, a.K1, a.K2e);
  if (cache_status(a.t) != 0) tl.n = 0;
  const int e0 = (int)((int64_t)tl.n * split / S), e1 = (int)((int64_t)tl.n * (split + 1) / S);
  const int mine = e0 + warp < e1 ? (e1 - e0 - warp + kW - 1) / kW : 0;  // this warp's tiles

  const int ps = a.t.ps, lps = a.t.lps, ppt = kTK >> lps;  // pages a tile
  const PageLayout<D> lay(ps);
  const int pitch = lay.bytes + (ps < kTK ? 2 * ps : 0);
  const uint32_t ring = smem_addr(smem) + warp * kStages * C::STG;
  const uint32_t bar = smem_addr(smem) + C::OFF_BAR + warp * kStages * 8;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(bar + 8 * s, 1);
    fence_barrier_init();
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncwarp();

  // Page ids of tiles k0 + lane of this warp, 32 tiles at a time.
  const int32_t* bt = a.t.bt + (int64_t)b * a.t.M;
  const int pages = (sq.Lh + ps - 1) >> lps;
  int id[4];
  auto load_ids = [&](int k0) {
    const int e = e0 + warp + (k0 + lane) * kW;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      id[p] = 0;
      if (p < ppt && e < e1) {
        const int i = tl.at(e) * ppt + p;
        if (i < pages) {
          id[p] = bt[i];
          if (id[p] < 0 || id[p] >= a.t.P) {
            cache_fail(a.t, HSTU_SLA_ERR_BAD_INPUT);
            id[p] = 0;
          }
        }
      }
    }
  };
  auto issue = [&](int k) {
    if ((k & 31) == 0) load_ids(k);
    const int s = k % kStages;
    const int first = tl.at(e0 + warp + k * kW) * ppt;
    const int np = imin(ppt, pages - first);
    if (lane == 0) mbar_expect_tx(bar + 8 * s, (uint32_t)(np * lay.bytes));
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int page = __shfl_sync(0xffffffffu, id[p], k & 31);
      if (lane == 0 && p < np)
        bulk_load(ring + s * C::STG + p * pitch,
                  a.pages + page * a.page_stride + (int64_t)h * lay.bytes, (uint32_t)lay.bytes,
                  bar + 8 * s);
    }
  };
  for (int k = 0; k < kStages && k < mine; ++k) issue(k);

  // Q fragments: k index 2t + {0, 1} (+ 8) of k-step ks is dim t D/4 + 4 ks +
  // {0, 1} ({2, 3}).  sum(q) of rows g and g + 8.
  uint32_t qf[KS][4];
  float sum0 = 0.f, sum1 = 0.f;
  const bool two = nr > 8;
  {
    const bf16* q0 = a.q + (int64_t)(sq.s0 + r0 + g) * a.q_rs + h * D + t * (D / 4);
    const bf16* q1 = q0 + 8 * a.q_rs;
#pragma unroll
    for (int ks = 0; ks < KS; ks += 2) {
      uint4 x = make_uint4(0, 0, 0, 0), y = x;
      if (g < nr) x = *reinterpret_cast<const uint4*>(q0 + 4 * ks);
      if (g + 8 < nr) y = *reinterpret_cast<const uint4*>(q1 + 4 * ks);
      qf[ks][0] = x.x; qf[ks][2] = x.y; qf[ks + 1][0] = x.z; qf[ks + 1][2] = x.w;
      qf[ks][1] = y.x; qf[ks][3] = y.y; qf[ks + 1][1] = y.z; qf[ks + 1][3] = y.w;
      sum0 += (bf_lo(x.x) + bf_hi(x.x)) + (bf_lo(x.y) + bf_hi(x.y)) +
              ((bf_lo(x.z) + bf_hi(x.z)) + (bf_lo(x.w) + bf_hi(x.w)));
      sum1 += (bf_lo(y.x) + bf_hi(y.x)) + (bf_lo(y.y) + bf_hi(y.y)) +
              ((bf_lo(y.z) + bf_hi(y.z)) + (bf_lo(y.w) + bf_hi(y.w)));
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      sum0 += __shfl_xor_sync(0xffffffffu, sum0, o);
      sum1 += __shfl_xor_sync(0xffffffffu, sum1, o);
    }
  }
  // A candidate's own pair: SiLU(alpha q_i . k_i), by a warp per row.
  float* self = reinterpret_cast<float*>(smem + C::OFF_SELF);
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

  const CacheRow c0 = cache_row(r0 + imin(g, nr - 1), sq.h, sq.Lh, a.K1, a.K2e);
  const CacheRow c1 = cache_row(r0 + imin(g + 8, nr - 1), sq.h, sq.Lh, a.K1, a.K2e);
  const CacheFull whole = cache_full(r0, r0 + nr, sq.h, sq.Lh, a.K1, a.K2e);
  const float ha = 0.5f * a.alpha;

  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float rest0 = 0.f, rest1 = 0.f;  // sum P m - 16 P' of rows g, g + 8 (this thread's keys)

  const int pt = (16 * t) >> lps, in = (16 * t) & (ps - 1);    // page and place of tokens 16 t
  const int pg = (16 * (g >> 1)) >> lps, ing = (16 * (g >> 1)) & (ps - 1);
  bool ok = true;
  int k = 0;
  for (; k < mine; ++k) {
    const int s = k % kStages;
    ok = __all_sync(0xffffffffu, bounded_wait(bar + 8 * s, (k / kStages) & 1, a.t));
    if (!ok) break;
    const int j0 = tl.at(e0 + warp + k * kW) * kTK;
    const bool full = whole(j0, kTK);
    const uint32_t stg = ring + s * C::STG;
    const uint32_t kbase = stg + pg * pitch + (ing + (g & 1)) * (D / 2) + t * (D / 8);
    const uint32_t par = stg + pt * pitch + lay.kp + 4 * in;
    uint32_t pf[4][4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
      uint32_t ka[WD], kb[WD];
      lds<WD>(ka, kbase + 4 * u * (D / 2));
      lds<WD>(kb, kbase + (4 * u + 2) * (D / 2));
#pragma unroll
      for (int w = 0; w < WD; ++w) {
        mma16816(sa, qf[2 * w], code_pair<0>(ka[w]), code_pair<1>(ka[w]));
        mma16816(sb, qf[2 * w], code_pair<0>(kb[w]), code_pair<1>(kb[w]));
        mma16816(sa, qf[2 * w + 1], code_pair<2>(ka[w]), code_pair<3>(ka[w]));
        mma16816(sb, qf[2 * w + 1], code_pair<2>(kb[w]), code_pair<3>(kb[w]));
      }
      uint32_t kp[4], vp[4];
      lds<4>(kp, par + 16 * u);
      lds<4>(vp, par + 16 * u + (lay.vp - lay.kp));
      float p0[4], p1[4];
      const int j = j0 + 16 * t + 4 * u;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float ks = bf_lo(kp[e]) * ha, km = fmaf(ks, -16.f, bf_hi(kp[e]) * ha);
        const float x0 = fmaf(e < 2 ? sa[e] : sb[e - 2], ks, km * sum0);
        p0[e] = fmaf(x0, tanh_approx(x0), x0);
        if (two) {
          const float x1 = fmaf(e < 2 ? sa[e + 2] : sb[e], ks, km * sum1);
          p1[e] = fmaf(x1, tanh_approx(x1), x1);
        } else {
          p1[e] = 0.f;
        }
      }
      float q0[4], q1[4], m0[4], m1[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float vs = bf_lo(vp[e]), vm = bf_hi(vp[e]);
        q0[e] = p0[e] * vs;
        m0[e] = p0[e] * vm;
        q1[e] = two ? p1[e] * vs : 0.f;
        m1[e] = two ? p1[e] * vm : 0.f;
        if (!full) {
          const bool see0 = j + e < c0.pre || (j + e >= c0.lo && j + e < c0.hi);
          const bool see1 = j + e < c1.pre || (j + e >= c1.lo && j + e < c1.hi);
          q0[e] = see0 ? q0[e] : 0.f;
          m0[e] = see0 ? m0[e] : 0.f;
          q1[e] = see1 ? q1[e] : 0.f;
          m1[e] = see1 ? m1[e] : 0.f;
        }
      }
      pf[u][0] = pack_bf16x2(q0[0], q0[1]);
      pf[u][1] = pack_bf16x2(q1[0], q1[1]);
      pf[u][2] = pack_bf16x2(q0[2], q0[3]);
      pf[u][3] = pack_bf16x2(q1[2], q1[3]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t w0 = pf[u][e < 2 ? 0 : 2], w1 = pf[u][e < 2 ? 1 : 3];
        rest0 += fmaf(e & 1 ? bf_hi(w0) : bf_lo(w0), -16.f, m0[e]);
        if (two) rest1 += fmaf(e & 1 ? bf_hi(w1) : bf_lo(w1), -16.f, m1[e]);
      }
    }
    const uint32_t vbase = stg + pt * pitch + lay.v + in + g * ps;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint32_t vw[4];
      lds<4>(vw, vbase + 8 * i * ps);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        // low nibbles: dim 2i; high: dim 2i + 1.  Bytes are tokens 0, 2, 1, 3.
        mma16816(o[2 * i], pf[u], code_pair<0>(vw[u]), code_pair<2>(vw[u]));
        mma16816(o[2 * i + 1], pf[u], code_pair<1>(vw[u]), code_pair<3>(vw[u]));
      }
    }
    __syncwarp();
    if (k + kStages < mine) issue(k + kStages);
  }
  if (!ok) {  // copies in flight land before the ring is used again
    for (int i = k; i < mine && i < k + kStages; ++i)
      drain_wait(bar + 8 * (i % kStages), (i / kStages) & 1);
    __syncwarp();
  }

  // The warp's result into its ring, [16][D] fp32.
#pragma unroll
  for (int x = 1; x < 4; x <<= 1) {
    rest0 += __shfl_xor_sync(0xffffffffu, rest0, x);
    rest1 += __shfl_xor_sync(0xffffffffu, rest1, x);
  }
  {
    // columns 2t, 2t + 1 of tile (2i + e) are dims 16 i + 4 t + e and + 2 + e
    float* w = reinterpret_cast<float*>(smem + warp * kStages * C::STG);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      float4 x = make_float4(o[2 * i][0] + rest0, o[2 * i + 1][0] + rest0, o[2 * i][1] + rest0,
                             o[2 * i + 1][1] + rest0);
      *reinterpret_cast<float4*>(w + g * D + 16 * i + 4 * t) = x;
      if (two) {
        x = make_float4(o[2 * i][2] + rest1, o[2 * i + 1][2] + rest1, o[2 * i][3] + rest1,
                        o[2 * i + 1][3] + rest1);
        *reinterpret_cast<float4*>(w + (g + 8) * D + 16 * i + 4 * t) = x;
      }
    }
  }
  __syncthreads();
  // sum of the block's warps, then of the cluster's blocks
  // (in place of warp 0's: an element is read and written by one thread)
  float* part = reinterpret_cast<float*>(smem);
  for (int e = threadIdx.x * 2; e < nr * D; e += 2 * kThreads) {
    float2 x = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      const float2 y = *reinterpret_cast<const float2*>(smem + w * kStages * C::STG + 4 * e);
      x.x += y.x;
      x.y += y.y;
    }
    *reinterpret_cast<float2*>(part + e) = x;
  }
  cg::cluster_group cl = cg::this_cluster();
  if (S > 1) cl.sync(); else __syncthreads();
  for (int e = (split * kThreads + threadIdx.x) * 2; e < nr * D; e += 2 * kThreads * S) {
    float2 x = *reinterpret_cast<const float2*>(S > 1 ? cl.map_shared_rank(part, 0) + e : part + e);
    for (int r = 1; r < S; ++r) {
      const float2 y = *reinterpret_cast<const float2*>(cl.map_shared_rank(part, r) + e);
      x.x += y.x;
      x.y += y.y;
    }
    const int r = e / D, c = e % D;
    const int64_t row = sq.s0 + r0 + r;
    if (r0 + r >= sq.h) {
      const uint32_t v2 = *reinterpret_cast<const uint32_t*>(a.v + row * a.v_rs + h * D + c);
      x.x = fmaf(self[r], bf_lo(v2), x.x);
      x.y = fmaf(self[r], bf_hi(v2), x.y);
    }
    *reinterpret_cast<uint32_t*>(a.out + row * a.o_rs + h * D + c) =
        pack_bf16x2(x.x * a.inv_n, x.y * a.inv_n);
  }
  if (S > 1) cl.sync();  // no block leaves while another reads its sum
}

template <int D>
cudaError_t launch_step(const CacheAttnArgs& a, cudaStream_t st) {
  using C = StepCfg<D>;
  auto kern = cache_step_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const int row_tiles = (a.max_new + kRows - 1) / kRows;
  const int64_t units = (int64_t)a.t.B * a.H * row_tiles;
  // Blocks a unit: enough to fill the GPU about twice, no more than a unit has
  // key tiles for (at least one per warp).
  const int64_t keys =
      imin(a.t.M * a.t.ps, (int)(((int64_t)a.K1 + a.K2e + kRows) < (1 << 30) ? a.K1 + a.K2e + kRows : 1 << 30));
  const int64_t tiles = keys / kTK + 2;
  int S = 1;
  while (S < 8 && units * S < 2 * 148 && tiles >= 2 * S * kW) S *= 2;
  if (units * S > 0x7fffffff) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * S));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, S, row_tiles);
}

}  // namespace

cudaError_t launch_cache_attend(const CacheAttnArgs& a, int d, cudaStream_t st) {
  if (a.T == 0 || a.max_new == 0) return cudaSuccess;
  if (d == 32) return launch_step<32>(a, st);
  if (d == 64) return launch_step<64>(a, st);
  return launch_step<128>(a, st);
}

}  // namespace hstu
