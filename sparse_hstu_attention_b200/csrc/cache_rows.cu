// K/V rows into and out of the 4-bit pages (include/hstu_cache.h).
//
// A block takes TT consecutive rows of one head; D / 8 lanes hold a row, 8
// dims (one word of K codes) each.  Append: the row's minimum and maximum by
// shuffles, then code = round((x - m) * (1 / s)), the rounding to whole numbers
// by adding 1.5 2^23 and the packing of 8 codes by multiply-adds with powers of
// 16 (mod 2^32; what the added constant leaves is taken off at the end).  Even
// lanes divide for K and odd ones for V.  Read: bf16(m + s code) by one bf16
// multiply-add, which rounds once.  (Rounding to fp32 on the way is not the same:
// s code may lie midway between two bf16 numbers, where a small m decides and fp32
// has lost it.)
//
// V codes lie dim pair by dim pair, so one row's bytes are page_size apart.
// Rows of one sequence come in runs of consecutive slots: a run's part in one
// aligned block of 16 tokens (a "group") is gathered in shared memory, column
// by column, and moves as 16-byte pieces.  A tile with too many groups (single
// events of many users) moves single bytes.
//
// Bound: bytes (append reads 4 d and writes d + 8 per token and head), with
// issue slots close behind: 100k rows of 4 x 128 stored in 63 us (4.1 TB/s) and read
// back in 53 (4.9 TB/s); unrolled loops with fewer blocks an SM take 116 to 130 for both.
// (At d = 32 the 32 registers of 7 blocks an SM leave the append of 128-row tiles 60
// bytes a thread in local memory.)
#include "cache_common.cuh"
#include "sm100.cuh"

namespace hstu {

namespace {

constexpr int kThreads = 256;

template <int TT>
struct Groups {
  static constexpr int kMost = TT / 16 + 8;  // groups a tile may hold in shared memory
  static constexpr int kPitch = kMost * 16 + 4;
  int64_t slot[TT];         // -1: no row
  uint8_t* block[TT];       // this head's block of the slot's page
  int16_t group[TT];
  uint32_t mask[kMost];     // places of the group that have a row
  int64_t base[kMost];      // its first slot, a multiple of 16
  int heads[TT / 32 + 1];
};

// Slots of the tile's rows, checked; groups numbered.  Returns their count, or -1
// if the tables' status is set: one answer for the whole block, whose warps may
// read different ones while another block reports a bad slot.
template <int TT>
__device__ __forceinline__ int find_groups(const CacheRowArgs& a, int64_t t0, int head_off,
                                           Groups<TT>* g) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int status = cache_status(a.t);
  const int64_t n_slots = (int64_t)a.t.P << a.t.lps;
  if (tid < TT) {
    int64_t s = t0 + tid < a.T ? a.slots[t0 + tid] : -1;
    if (s >= n_slots) {
      cache_fail(a.t, HSTU_SLA_ERR_BAD_INPUT);
      s = -1;
    }
    s = s < 0 ? -1 : s;
    g->slot[tid] = s;
    g->block[tid] = a.pages + (s < 0 ? 0 : s >> a.t.lps) * a.page_stride + head_off;
  }
  if (tid < Groups<TT>::kMost) g->mask[tid] = 0;
  if (__syncthreads_or(status != 0)) return -1;
  int mine = 0;
  bool head = false;
  if (tid < TT) {
    const int64_t s = g->slot[tid];
    head = s >= 0 && (tid == 0 || (s & 15) == 0 || g->slot[tid - 1] + 1 != s);
  }
  const uint32_t heads = __ballot_sync(0xffffffffu, head);
  if (tid < TT && lane == 0) g->heads[warp] = __popc(heads);
  __syncthreads();
  int total = 0;
  for (int w = 0; w < (TT + 31) / 32; ++w) {
    if (w == warp) mine = total;
    total += g->heads[w];
  }
  if (tid < TT) {
    const int64_t s = g->slot[tid];
    const int k = mine + __popc(heads & (0xffffffffu >> (31 - lane))) - 1;
    g->group[tid] = (int16_t)k;
    if (s >= 0 && total <= Groups<TT>::kMost) {
      if (head) g->base[k] = s & ~int64_t(15);
      atomicOr(&g->mask[k], 1u << (s & 15));
    }
  }
  __syncthreads();
  return total;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bits(__nv_bfloat162 x) {
  return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ __nv_bfloat162 pair(uint32_t x) {
  return *reinterpret_cast<const __nv_bfloat162*>(&x);
}

// (minimum, -maximum) of a row as bf16 (exact); a NaN stays one.
template <int LPR>
__device__ __forceinline__ uint32_t extremes(const uint32_t (&w)[4]) {
  const __nv_bfloat162 lo = __hmin2_nan(__hmin2_nan(pair(w[0]), pair(w[1])),
                                        __hmin2_nan(pair(w[2]), pair(w[3])));
  const __nv_bfloat162 hi = __hmax2_nan(__hmax2_nan(pair(w[0]), pair(w[1])),
                                        __hmax2_nan(pair(w[2]), pair(w[3])));
  const uint32_t x = __byte_perm(bits(lo), bits(hi), 0x5410) ^ 0x80000000u;
  const uint32_t y = __byte_perm(bits(lo), bits(hi), 0x7632) ^ 0x80000000u;
  uint32_t r = bits(__hmin2_nan(pair(x), pair(y)));
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1)
    r = bits(__hmin2_nan(pair(r), pair(__shfl_xor_sync(0xffffffffu, r, o))));
  return r;
}

// Codes of 8 dims, dim i at nibble i (K: at the nibble of a K word).
template <bool K>
__device__ __forceinline__ uint32_t codes(const uint32_t (&w)[4], float m, float inv) {
  constexpr uint32_t kMagic = 0x4b400000u;  // 1.5 2^23
  uint32_t c = 0u - kMagic * 0x11111111u;
  const uint64_t less = sm100::f2s(-m), inv2 = sm100::f2s(inv);
  const float magic = __uint_as_float(kMagic);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    // (the product is rounded before the sum: scalar adds, which no compiler
    // joins with the paired multiply)
    const uint64_t x = sm100::f2_mul(
        sm100::f2_add(sm100::f2(w[e] << 16, w[e] & 0xffff0000u), less), inv2);
    c += __float_as_uint(__fadd_rn(sm100::f2_lo(x), magic)) * (1u << (K ? 4 * e : 8 * e));
    c += __float_as_uint(__fadd_rn(sm100::f2_hi(x), magic)) *
         (1u << (K ? 4 * e + 16 : 8 * e + 4));
  }
  return c;
}

// A token's K and V rows: the lane's codes and the rows' (step, minimum) pairs.
template <int LPR>
__device__ __forceinline__ void quantise(const uint4& xk, const uint4& xv, uint32_t* ck,
                                         uint32_t* cv, uint32_t* pk, uint32_t* pv) {
  const uint32_t k[4] = {xk.x, xk.y, xk.z, xk.w}, v[4] = {xv.x, xv.y, xv.z, xv.w};
  const uint32_t ek = extremes<LPR>(k), ev = extremes<LPR>(v);
  const bool odd = threadIdx.x & 1;
  const uint32_t e = odd ? ev : ek;
  // (max - min) / 15, correctly rounded by one residual from the rounded 1/15
  // (Markstein's theorem)
  const float span = __fsub_rn(-bf_hi(e), bf_lo(e)), q = __fmul_rn(span, 1.f / 15.f);
  float s = __bfloat162float(
      __float2bfloat16_rn(__fmaf_rn(__fmaf_rn(-15.f, q, span), 1.f / 15.f, q)));
  if (s < 1.17549435e-38f) s = 0.f;
  // not for a NaN or an infinity: such a row is NaN, its codes 0
  const bool fine = s <= 3.4e38f;
  const float inv = !fine ? __int_as_float(0x7fc00000) : s > 0.f ? __frcp_rn(s) : 0.f;
  const uint32_t p = fine ? (__float_as_uint(s) >> 16) | (e << 16) : 0x7fc07fc0u;
  const float inv2 = __shfl_xor_sync(0xffffffffu, inv, 1);
  const uint32_t p2 = __shfl_xor_sync(0xffffffffu, p, 1);
  const float ik = odd ? inv2 : inv, iv = odd ? inv : inv2;
  *pk = odd ? p2 : p;
  *pv = odd ? p : p2;
  *ck = isnan(ik) ? 0u : codes<true>(k, bf_lo(ek), ik);
  *cv = isnan(iv) ? 0u : codes<false>(v, bf_lo(ev), iv);
}

template <int D, int TT>
__global__ void __launch_bounds__(kThreads, 7) cache_append_kernel(CacheRowArgs a) {
  constexpr int LPR = D / 8, RPI = kThreads / LPR;  // lanes a row, rows an iteration
  using G = Groups<TT>;
  __shared__ G g;
  __shared__ __align__(16) uint8_t sv[D / 2 * G::kPitch];  // (words of it are moved)
  const int64_t t0 = (int64_t)blockIdx.x * TT;
  const int h = blockIdx.y, ps = a.t.ps;
  const PageLayout<D> lay(ps);
  const int n_groups = find_groups<TT>(a, t0, h * lay.bytes, &g);
  if (n_groups < 0) return;
  const bool grouped = n_groups <= G::kMost;
  const int w = threadIdx.x % LPR;
  const bf16* kp = a.k + (t0 + threadIdx.x / LPR) * a.k_rs + h * D + w * 8;
  const bf16* vp = a.v + (t0 + threadIdx.x / LPR) * a.v_rs + h * D + w * 8;
  const int64_t k_step = RPI * a.k_rs, v_step = RPI * a.v_rs;
#pragma unroll 1
  for (int r0 = threadIdx.x / LPR; r0 < TT; r0 += RPI, kp += k_step, vp += v_step) {
    const int64_t s = g.slot[r0];
    uint4 xk = make_uint4(0, 0, 0, 0), xv = xk;
    if (s >= 0) {
      xk = *reinterpret_cast<const uint4*>(kp);
      xv = *reinterpret_cast<const uint4*>(vp);
    }
    uint32_t ck, pk, cv, pv;
    quantise<LPR>(xk, xv, &ck, &cv, &pk, &pv);
    if (s < 0) continue;
    uint8_t* blk = g.block[r0];
    const int r = (int)s & (ps - 1);
    *reinterpret_cast<uint32_t*>(blk + r * (D / 2) + w * 4) = ck;
    if (w == 0) {
      *reinterpret_cast<uint32_t*>(blk + lay.kp + 4 * r) = pk;
      *reinterpret_cast<uint32_t*>(blk + lay.vp + 4 * r) = pv;
    }
    if (grouped) {
      uint8_t* col = sv + 4 * w * G::kPitch + g.group[r0] * 16 + v_place(r & 15);
#pragma unroll
      for (int e = 0; e < 4; ++e) col[e * G::kPitch] = (uint8_t)(cv >> (8 * e));
    } else {
      uint8_t* col = blk + lay.v + 4 * w * ps + v_place(r);
#pragma unroll
      for (int e = 0; e < 4; ++e) col[e * ps] = (uint8_t)(cv >> (8 * e));
    }
  }
  if (!grouped) return;
  __syncthreads();
  for (int e = threadIdx.x; e < n_groups * (D / 2); e += kThreads) {
    const int k = e / (D / 2), i = e % (D / 2);
    const int64_t s = g.base[k];
    const uint32_t mask = g.mask[k];
    const uint32_t* src = reinterpret_cast<const uint32_t*>(sv + i * G::kPitch + k * 16);
    uint8_t* dst = a.pages + (s >> a.t.lps) * a.page_stride + (int64_t)h * lay.bytes + lay.v +
                   i * ps + ((int)s & (ps - 1));
    if (mask == 0xffffu) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(src[0], src[1], src[2], src[3]);
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t m4 = (mask >> (4 * u)) & 15u;
        if (m4 == 15u) {
          reinterpret_cast<uint32_t*>(dst)[u] = src[u];
        } else if (m4) {
          for (int j = 0; j < 4; ++j)
            if (m4 >> j & 1u) dst[4 * u + v_place(j)] = (uint8_t)(src[u] >> (8 * v_place(j)));
        }
      }
    }
  }
}

// Two values m + s code, the codes in bits 0..3 of the halves: 128 + c is a bf16
// number with c in its last bits.
__device__ __forceinline__ uint32_t dequantise(uint32_t c, __nv_bfloat162 s, __nv_bfloat162 m) {
  const __nv_bfloat162 x =
      __hadd2_rn(pair((c & 0x000f000fu) | 0x43004300u), pair(0xc300c300u));
  return bits(__hfma2(x, s, m));
}

template <int D, int TT>
__global__ void __launch_bounds__(kThreads, 7) cache_read_kernel(CacheRowArgs a) {
  constexpr int LPR = D / 8, RPI = kThreads / LPR;
  using G = Groups<TT>;
  __shared__ G g;
  __shared__ __align__(16) uint8_t sv[D / 2 * G::kPitch];  // (words of it are moved)
  const int64_t t0 = (int64_t)blockIdx.x * TT;
  const int h = blockIdx.y, ps = a.t.ps;
  const PageLayout<D> lay(ps);
  const int n_groups = find_groups<TT>(a, t0, h * lay.bytes, &g);
  if (n_groups < 0) return;
  const bool grouped = n_groups <= G::kMost;
  if (grouped) {
    for (int e = threadIdx.x; e < n_groups * (D / 2); e += kThreads) {
      const int k = e / (D / 2), i = e % (D / 2);
      const int64_t s = g.base[k];
      const uint4 x = *reinterpret_cast<const uint4*>(
          a.pages + (s >> a.t.lps) * a.page_stride + (int64_t)h * lay.bytes + lay.v + i * ps +
          ((int)s & (ps - 1)));
      uint32_t* dst = reinterpret_cast<uint32_t*>(sv + i * G::kPitch + k * 16);
      dst[0] = x.x;
      dst[1] = x.y;
      dst[2] = x.z;
      dst[3] = x.w;
    }
    __syncthreads();
  }
  const int w = threadIdx.x % LPR;
  bf16* ko = a.k + (t0 + threadIdx.x / LPR) * a.k_rs + h * D + w * 8;
  bf16* vo = a.v + (t0 + threadIdx.x / LPR) * a.v_rs + h * D + w * 8;
  const int64_t k_step = RPI * a.k_rs, v_step = RPI * a.v_rs;
#pragma unroll 1
  for (int r0 = threadIdx.x / LPR; r0 < TT; r0 += RPI, ko += k_step, vo += v_step) {
    const int64_t s = g.slot[r0];
    uint4 xk = make_uint4(0, 0, 0, 0), xv = xk;
    if (s >= 0) {
      const uint8_t* blk = g.block[r0];
      const int r = (int)s & (ps - 1);
      const uint32_t kw = *reinterpret_cast<const uint32_t*>(blk + r * (D / 2) + w * 4);
      const uint32_t kp = *reinterpret_cast<const uint32_t*>(blk + lay.kp + 4 * r);
      const uint32_t vp = *reinterpret_cast<const uint32_t*>(blk + lay.vp + 4 * r);
      const uint8_t* col = grouped ? sv + 4 * w * G::kPitch + g.group[r0] * 16 + v_place(r & 15)
                                   : blk + lay.v + 4 * w * ps + v_place(r);
      const int step = grouped ? G::kPitch : ps;
      uint32_t b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = col[e * step];
      __nv_bfloat162 s2 = pair(__byte_perm(kp, 0, 0x1010)), m2 = pair(__byte_perm(kp, 0, 0x3232));
      xk = make_uint4(dequantise(kw, s2, m2), dequantise(kw >> 4, s2, m2),
                      dequantise(kw >> 8, s2, m2), dequantise(kw >> 12, s2, m2));
      s2 = pair(__byte_perm(vp, 0, 0x1010));
      m2 = pair(__byte_perm(vp, 0, 0x3232));
      xv = make_uint4(dequantise(b[0] | b[0] << 12, s2, m2), dequantise(b[1] | b[1] << 12, s2, m2),
                      dequantise(b[2] | b[2] << 12, s2, m2), dequantise(b[3] | b[3] << 12, s2, m2));
    }
    if (t0 + r0 < a.T) {
      *reinterpret_cast<uint4*>(ko) = xk;
      *reinterpret_cast<uint4*>(vo) = xv;
    }
  }
}

// Tiles of 128 rows gather whole groups; a batch too small to fill the GPU
// with them takes tiles of 16.  Measured, 16 rows / 128, append and read, us: 4 heads of
// 128, 1024 rows 3.4 / 8.0 and 3.1 / 5.4, 4096 rows 6.1 / 8.1 and 5.5 / 5.5, 8192 rows 8.7 /
// 9.4 and 8.8 / 6.5, 32768 rows 25.6 / 22.4 and 27.9 / 16.3; 1 head of 32, 8192 rows 3.6 /
// 3.7 and 3.5 / 3.1, 32768 rows 7.0 / 4.6 and 7.0 / 3.6.
template <int D>
cudaError_t launch_rows(const CacheRowArgs& a, bool append, cudaStream_t st) {
  const bool big = (a.T + 127) / 128 * a.H >= kSMs;
  const dim3 grid((unsigned)((a.T + (big ? 127 : 15)) / (big ? 128 : 16)), (unsigned)a.H);
  if (append) {
    if (big) cache_append_kernel<D, 128><<<grid, kThreads, 0, st>>>(a);
    else cache_append_kernel<D, 16><<<grid, kThreads, 0, st>>>(a);
  } else {
    if (big) cache_read_kernel<D, 128><<<grid, kThreads, 0, st>>>(a);
    else cache_read_kernel<D, 16><<<grid, kThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_rows_d(const CacheRowArgs& a, int d, bool append, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  if (d == 32) return launch_rows<32>(a, append, st);
  if (d == 64) return launch_rows<64>(a, append, st);
  return launch_rows<128>(a, append, st);
}

}  // namespace

cudaError_t launch_cache_append(const CacheRowArgs& a, int d, cudaStream_t st) {
  return launch_rows_d(a, d, true, st);
}
cudaError_t launch_cache_read(const CacheRowArgs& a, int d, cudaStream_t st) {
  return launch_rows_d(a, d, false, st);
}

}  // namespace hstu
