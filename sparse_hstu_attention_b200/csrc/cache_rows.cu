// K/V rows into and out of the 4-bit pages (include/hstu_cache.h).
//
// A block takes TT consecutive rows of one head; D / 8 lanes hold a row, 8
// dims (one word of K codes) each.  Append: the row's minimum and maximum by
// shuffles, then code = round((x - m) * (1 / s)); read: bf16(m + s code), one
// fused multiply-add, exact before the rounding to bf16 up to fp32.
//
// V codes lie dim pair by dim pair, so one row's bytes are page_size apart.
// Rows of one sequence come in runs of consecutive slots: a run's part in one
// aligned block of 16 tokens (a "group") is gathered in shared memory, column
// by column, and moves as 16-byte pieces.  A tile with too many groups (single
// events of many users) moves single bytes.
//
// Bound: bytes (append reads 4 d and writes d + 8 per token and head).
#include "cache_common.cuh"

namespace hstu {

namespace {

constexpr int kThreads = 256;

template <int TT>
struct Groups {
  static constexpr int kMost = TT / 16 + 8;  // groups a tile may hold in shared memory
  static constexpr int kPitch = kMost * 16 + 4;
  int64_t slot[TT];    // -1: no row
  int16_t group[TT];
  uint32_t mask[kMost];     // places of the group that have a row
  int64_t base[kMost];      // its first slot, a multiple of 16
  int heads[TT / 32 + 1];
};

// Slots of the tile's rows, checked; groups numbered.  Returns their count.
template <int TT>
__device__ __forceinline__ int find_groups(const CacheRowArgs& a, int64_t t0, Groups<TT>* g) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t n_slots = (int64_t)a.t.P << a.t.lps;
  if (tid < TT) {
    int64_t s = t0 + tid < a.T ? a.slots[t0 + tid] : -1;
    if (s >= n_slots) {
      cache_fail(a.t, HSTU_SLA_ERR_BAD_INPUT);
      s = -1;
    }
    g->slot[tid] = s < 0 ? -1 : s;
  }
  if (tid < Groups<TT>::kMost) g->mask[tid] = 0;
  __syncthreads();
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

// Codes of the lane's 8 dims and the row's (step, minimum) pair: nibble n of
// *word is dim n.  LPR lanes hold one row.
template <int LPR>
__device__ __forceinline__ void quantise(const uint4& x, uint32_t* word, uint32_t* pair) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float f[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = bf_lo(w[e]);
    f[2 * e + 1] = bf_hi(w[e]);
  }
  // minimum and maximum in bf16 pairs (exact); a NaN stays one
  const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(w);
  __nv_bfloat162 lo2 = __hmin2_nan(__hmin2_nan(b[0], b[1]), __hmin2_nan(b[2], b[3]));
  __nv_bfloat162 hi2 = __hmax2_nan(__hmax2_nan(b[0], b[1]), __hmax2_nan(b[2], b[3]));
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) {
    lo2 = __hmin2_nan(lo2, __shfl_xor_sync(0xffffffffu, lo2, o));
    hi2 = __hmax2_nan(hi2, __shfl_xor_sync(0xffffffffu, hi2, o));
  }
  float m = __bfloat162float(__hmin_nan(lo2.x, lo2.y));
  const float hi = __bfloat162float(__hmax_nan(hi2.x, hi2.y));
  float s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi, m), 15.f)));
  const bool fine = s <= 3.4e38f;  // not for a NaN or an infinity
  if (s < 1.17549435e-38f) s = 0.f;
  const float inv = s > 0.f && fine ? __frcp_rn(s) : 0.f;
  uint32_t c = 0;
  if (fine) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int v = __float2int_rn(__fmul_rn(__fsub_rn(f[e], m), inv));
      c |= (uint32_t)imin(v, 15) << (4 * e);
    }
  } else {
    s = m = __int_as_float(0x7fc00000);
  }
  *word = c;
  const __nv_bfloat162 sm = __floats2bfloat162_rn(s, m);
  *pair = *reinterpret_cast<const uint32_t*>(&sm);
}

// Nibbles (dim n at n) to the order of a K word: dims 0 2 4 6 1 3 5 7.
__device__ __forceinline__ uint32_t k_word(uint32_t c) {
  uint32_t r = 0;
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    r |= ((c >> (8 * n)) & 15u) << (4 * n);
    r |= ((c >> (8 * n + 4)) & 15u) << (16 + 4 * n);
  }
  return r;
}

template <int D, int TT>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(CacheRowArgs a) {
  constexpr int LPR = D / 8, RPI = kThreads / LPR;  // lanes a row, rows an iteration
  using G = Groups<TT>;
  __shared__ G g;
  __shared__ uint8_t sv[D / 2 * G::kPitch];
  if (cache_status(a.t) != 0) return;
  const int64_t t0 = (int64_t)blockIdx.x * TT;
  const int h = blockIdx.y, ps = a.t.ps;
  const PageLayout<D> lay(ps);
  const int n_groups = find_groups<TT>(a, t0, &g);
  const bool grouped = n_groups <= G::kMost;
  const int w = threadIdx.x % LPR;
#pragma unroll 2
  for (int r0 = threadIdx.x / LPR; r0 < TT; r0 += RPI) {
    const int64_t s = g.slot[r0];
    uint4 xk = make_uint4(0, 0, 0, 0), xv = xk;
    if (s >= 0) {
      xk = *reinterpret_cast<const uint4*>(a.k + (t0 + r0) * a.k_rs + h * D + w * 8);
      xv = *reinterpret_cast<const uint4*>(a.v + (t0 + r0) * a.v_rs + h * D + w * 8);
    }
    uint32_t ck, pk, cv, pv;
    quantise<LPR>(xk, &ck, &pk);
    quantise<LPR>(xv, &cv, &pv);
    if (s < 0) continue;
    uint8_t* blk = a.pages + (s >> a.t.lps) * a.page_stride + (int64_t)h * lay.bytes;
    const int r = (int)s & (ps - 1);
    *reinterpret_cast<uint32_t*>(blk + r * (D / 2) + w * 4) = k_word(ck);
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

// 8 values m + s code (nibble n of c is dim n), rounded to bf16.
__device__ __forceinline__ uint4 dequantise(uint32_t c, uint32_t pair) {
  const float s = bf_lo(pair), m = bf_hi(pair);
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 v =
        __floats2bfloat162_rn(fmaf(s, (float)((c >> (8 * e)) & 15u), m),
                              fmaf(s, (float)((c >> (8 * e + 4)) & 15u), m));
    o[e] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int D, int TT>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(CacheRowArgs a) {
  constexpr int LPR = D / 8, RPI = kThreads / LPR;
  using G = Groups<TT>;
  __shared__ G g;
  __shared__ uint8_t sv[D / 2 * G::kPitch];
  if (cache_status(a.t) != 0) return;
  const int64_t t0 = (int64_t)blockIdx.x * TT;
  const int h = blockIdx.y, ps = a.t.ps;
  const PageLayout<D> lay(ps);
  const int n_groups = find_groups<TT>(a, t0, &g);
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
#pragma unroll 4
  for (int r0 = threadIdx.x / LPR; r0 < TT; r0 += RPI) {
    if (t0 + r0 >= a.T) break;
    const int64_t s = g.slot[r0];
    uint4 xk = make_uint4(0, 0, 0, 0), xv = xk;
    if (s >= 0) {
      const uint8_t* blk = a.pages + (s >> a.t.lps) * a.page_stride + (int64_t)h * lay.bytes;
      const int r = (int)s & (ps - 1);
      const uint32_t kw = *reinterpret_cast<const uint32_t*>(blk + r * (D / 2) + w * 4);
      uint32_t ck = 0, cv = 0;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        ck |= ((kw >> (4 * n)) & 15u) << (8 * n);
        ck |= ((kw >> (16 + 4 * n)) & 15u) << (8 * n + 4);
      }
      const uint8_t* col = grouped ? sv + 4 * w * G::kPitch + g.group[r0] * 16 + v_place(r & 15)
                                   : blk + lay.v + 4 * w * ps + v_place(r);
      const int step = grouped ? G::kPitch : ps;
#pragma unroll
      for (int e = 0; e < 4; ++e) cv |= (uint32_t)col[e * step] << (8 * e);
      xk = dequantise(ck, *reinterpret_cast<const uint32_t*>(blk + lay.kp + 4 * r));
      xv = dequantise(cv, *reinterpret_cast<const uint32_t*>(blk + lay.vp + 4 * r));
    }
    *reinterpret_cast<uint4*>(a.k + (t0 + r0) * a.k_rs + h * D + w * 8) = xk;
    *reinterpret_cast<uint4*>(a.v + (t0 + r0) * a.v_rs + h * D + w * 8) = xv;
  }
}

// Tiles of 128 rows gather whole groups; a batch too small to fill the GPU
// with them takes tiles of 16.
template <int D>
cudaError_t launch_rows(const CacheRowArgs& a, bool append, cudaStream_t st) {
  const bool big = (a.T + 127) / 128 * a.H >= 148;
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
