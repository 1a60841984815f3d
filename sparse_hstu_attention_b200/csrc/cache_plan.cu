// The plan of a serving step: pages, block tables, slots and lengths, built on
// the device from the step's row counts (include/hstu_cache.h).
//
// Per sequence: new_b = rows - candidates, old_b = 0 if released else
// lengths[b], need_b = ceil((old_b + new_b) / ps) - ceil(old_b / ps) pages, and
// given_b = ceil(lengths[b] / ps) pages come back from a released one.  Two
// exclusive sums over b order the stack: released pages go to
// free_count + sum given + i, and page j of sequence b comes from
// free_count + total given - 1 - (sum need + j).
//
// Bound: latency.  It moves 12 bytes a sequence, 8 a page and 8 a row.  So one
// block does everything of a small step in one launch; a large one takes the
// sums in one block and the per-page and per-row work in a grid.  64 sequences of
// one row 4.5 us; 2048 sequences, 790k rows, a third released, 15.3 us.
#include "cache_common.cuh"

namespace hstu {

namespace {

constexpr int kThreads = 1024;

// Per-sequence sums of the plan, in shared memory or the caller's workspace.
struct PlanWs {
  int32_t ok;       // 0: the plan failed, nothing below holds
  int32_t top;      // free_count + pages given back, before any is taken
  int32_t old_top;  // free_count before the step
  int32_t given;    // pages given back in all
  int32_t pad[60];
  // then int32 old[B], need_sum[B + 1], given_sum[B + 1]
};
static_assert(sizeof(PlanWs) == 256, "plan header");

struct PlanArgs {
  CacheTab t;
  const int32_t* offs;
  const int32_t* nts;
  const int32_t* release;
  int64_t T;
  int64_t* slots;
  PlanWs* ws;
  int32_t *old, *need_sum, *given_sum;
};

__device__ __forceinline__ int warp_scan(int x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Exclusive sums of two values over the block; their totals in *ta, *tb.
__device__ __forceinline__ void block_scan2(int a, int b, int* xa, int* xb, int* ta, int* tb,
                                            int (*sm)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ia = warp_scan(a, lane), ib = warp_scan(b, lane);
  if (lane == 31) {
    sm[0][warp] = ia;
    sm[1][warp] = ib;
  }
  __syncthreads();
  if (warp < 2) sm[warp][lane] = warp_scan(sm[warp][lane], lane);
  __syncthreads();
  *xa = ia - a + (warp ? sm[0][warp - 1] : 0);
  *xb = ib - b + (warp ? sm[1][warp - 1] : 0);
  *ta = sm[0][31];
  *tb = sm[1][31];
  __syncthreads();
}

// Last index i of the non-decreasing x[0..n] with x[i] <= v (x[0] <= v).
__device__ __forceinline__ int last_at_most(const int32_t* x, int n, int v) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (x[mid] <= v) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The block's part: checks, sums and the new stack height.  All or nothing: the
// tables change only if every sequence's step can be done.  PER sequences a thread
// at a time, so that most batches take one scan.
template <int PER>
__device__ bool plan_sums(const PlanArgs& a) {
  __shared__ int sm[2][32];
  __shared__ int s_code;
  const CacheTab& t = a.t;
  const int fc = *t.free_count;
  if (threadIdx.x == 0) s_code = fc < 0 || fc > t.P ? HSTU_SLA_ERR_BAD_INPUT : 0;
  __syncthreads();
  int64_t base_need = 0, base_given = 0;
  for (int c = 0; c < t.B; c += PER * kThreads) {
    const int b0 = c + PER * (int)threadIdx.x;
    int need[PER], given[PER], old[PER], n_sum = 0, g_sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int b = b0 + i;
      need[i] = given[i] = old[i] = 0;
      if (b >= t.B) continue;
      const int o0 = a.offs[b], o1 = a.offs[b + 1], len = t.lengths[b];
      const int nt = a.nts ? a.nts[b] : 0;
      const bool rel = a.release && a.release[b] != 0;
      const int most = t.M * t.ps;
      const bool bad = (b == 0 && o0 != 0) || o0 < 0 || o1 < o0 || (int64_t)o1 > a.T || nt < 0 ||
                       nt > o1 - o0 || len < 0 || len > most;
      const int fresh = bad ? 0 : o1 - o0 - nt, keep = rel || bad ? 0 : len;
      if (bad || fresh > most - keep) {
        s_code = HSTU_SLA_ERR_BAD_INPUT;
        continue;
      }
      old[i] = keep;
      need[i] = ((keep + fresh + t.ps - 1) >> t.lps) - ((keep + t.ps - 1) >> t.lps);
      given[i] = rel ? (len + t.ps - 1) >> t.lps : 0;
    }
    // (at most 2^19 pages a sequence, max_pages: 4096 of them fit 32 bits; over
    // the rounds the sums are held at 2^31 - 1, above any num_pages, where the
    // step fails anyway)
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      n_sum += need[i];
      g_sum += given[i];
    }
    int xn, xg, tn, tg;
    block_scan2(n_sum, g_sum, &xn, &xg, &tn, &tg, sm);
    const int64_t most = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (b0 + i >= t.B) continue;
      a.old[b0 + i] = old[i];
      a.need_sum[b0 + i] = (int32_t)min(base_need + (uint32_t)xn, most);
      a.given_sum[b0 + i] = (int32_t)min(base_given + (uint32_t)xg, most);
      xn += need[i];
      xg += given[i];
    }
    base_need = min(base_need + (uint32_t)tn, most);
    base_given = min(base_given + (uint32_t)tg, most);
  }
  if (threadIdx.x == 0) {
    a.need_sum[t.B] = (int32_t)base_need;
    a.given_sum[t.B] = (int32_t)base_given;
    int code = s_code;
    if (!code && fc + base_given > t.P) code = HSTU_SLA_ERR_BAD_INPUT;
    if (!code && base_need > fc + base_given) code = HSTU_SLA_ERR_NO_PAGES;
    s_code = code;
  }
  __syncthreads();
  const bool ok = s_code == 0;
  if (threadIdx.x == 0) {
    a.ws->ok = ok;
    a.ws->top = fc + (int)base_given;
    a.ws->old_top = fc;
    a.ws->given = (int)base_given;
    *t.status = s_code;
    if (ok) *t.free_count = fc + (int)base_given - (int)base_need;
  }
  __syncthreads();
  return ok;
}

// Released sequence b's pages onto the stack, by a warp.
__device__ __forceinline__ void plan_push(const PlanArgs& a, int old_top, int b, int lane) {
  const int from = a.given_sum[b], n = a.given_sum[b + 1] - from;
  const int32_t* src = a.t.bt + (int64_t)b * a.t.M;
#pragma unroll 4
  for (int i = lane; i < n; i += 32) a.t.free_pages[old_top + from + i] = src[i];
}

__device__ __forceinline__ void plan_length(const PlanArgs& a, int b) {
  a.t.lengths[b] = a.old[b] + a.offs[b + 1] - a.offs[b] - (a.nts ? a.nts[b] : 0);
}

// N rows, row[i] of sequence b[i] (negative: -1 it is): their slots, and the
// block-table entries of those that are the first token of a page.  Entries below
// `have` are only read and the others only written, so rows need no order among
// them.  All rows' loads of one kind go out together.
template <int N>
__device__ __forceinline__ void plan_rows(const PlanArgs& a, int top, const int64_t (&row)[N],
                                          const int (&b)[N], int64_t (&slot)[N]) {
  const CacheTab& t = a.t;
  int o0[N], fresh[N], old[N], taken[N], page[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int x = imax(b[i], 0);
    o0[i] = a.offs[x];
    fresh[i] = a.offs[x + 1];
    old[i] = a.old[x];
    taken[i] = a.need_sum[x];
  }
  if (a.nts) {
#pragma unroll
    for (int i = 0; i < N; ++i) fresh[i] -= a.nts[imax(b[i], 0)];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int pos = old[i] + (int)row[i] - o0[i];
    const int j = pos >> t.lps, have = (old[i] + t.ps - 1) >> t.lps;
    const bool mine = b[i] >= 0 && row[i] < fresh[i];
    const int32_t* src = j < have ? t.bt + (int64_t)b[i] * t.M + j
                                  : t.free_pages + (top - 1 - (taken[i] + j - have));
    page[i] = mine ? *src : -1;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int pos = old[i] + (int)row[i] - o0[i];
    const int j = pos >> t.lps, have = (old[i] + t.ps - 1) >> t.lps, at = pos & (t.ps - 1);
    const bool mine = b[i] >= 0 && row[i] < fresh[i];
    if (mine && j >= have && at == 0) t.bt[(int64_t)b[i] * t.M + j] = page[i];
    slot[i] = mine ? (int64_t)page[i] * t.ps + at : -1;
  }
}

// Steps of up to kOneBlockRows rows and kOneBlockSeqs sequences: one block, the
// sums in shared memory.  Measured, one block / the grid, us, nothing released: 64
// sequences 3.1 / 5.6 at 64 rows, 6.0 / 7.0 at 4096, 9.1 / 7.3 at 8192; 1024 sequences
// 4.8 / 8.5 at 1024 rows, 7.9 / 8.5 at 4096; 2048 sequences 7.0 / 10.4 at 2048 rows,
// 13.4 / 10.5 at 8192.  The host does not know how many pages are released, and many
// sequences that release at once would be quicker by the grid: each 64 pages, 4.6 / 7.6
// for 64 sequences, 23.6 / 10.7 for 1024, 44.8 / 12.5 for 2048.
constexpr int64_t kOneBlockRows = 8192;
constexpr int kOneBlockSeqs = 2048;
template <int PER>
__global__ void __launch_bounds__(kThreads) plan_one_kernel(PlanArgs a) {
  __shared__ PlanWs head;
  __shared__ int32_t sums[3 * kOneBlockSeqs + 2];
  a.ws = &head;
  a.old = sums;
  a.need_sum = sums + a.t.B;
  a.given_sum = a.need_sum + a.t.B + 1;
  const bool ok = plan_sums<PER>(a);
  if (!ok) {
    for (int64_t r = threadIdx.x; r < a.T; r += kThreads) a.slots[r] = -1;
    return;
  }
  const int old_top = a.ws->old_top, top = a.ws->top;
  if (a.release)
    for (int b = threadIdx.x >> 5; b < a.t.B; b += kThreads / 32)
      plan_push(a, old_top, b, threadIdx.x & 31);
  __syncthreads();
  const int rows = a.offs[a.t.B];
  for (int64_t r = threadIdx.x; r < a.T; r += kThreads) {
    const int64_t row[1] = {r};
    const int b[1] = {r < rows ? last_at_most(a.offs, a.t.B - 1, (int)r) : -1};
    int64_t slot[1];
    plan_rows<1>(a, top, row, b, slot);
    a.slots[r] = slot[0];
  }
  for (int b = threadIdx.x; b < a.t.B; b += kThreads) plan_length(a, b);
}

template <int PER>
__global__ void __launch_bounds__(kThreads) plan_sums_kernel(PlanArgs a) {
  plan_sums<PER>(a);
}

__global__ void __launch_bounds__(256) plan_push_kernel(PlanArgs a) {
  wait_for_the_last_kernel();
  const int b = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (a.ws->ok && b < a.t.B) plan_push(a, a.ws->old_top, b, threadIdx.x & 31);
}

// 1024 rows a block: the first row's sequence by a search of 32 probes a step,
// the others' among the 1024 that follow it, in shared memory.
constexpr int kRowsBlock = 1024;
__global__ void __launch_bounds__(256) plan_rows_kernel(PlanArgs a) {
  __shared__ int first, win[kRowsBlock + 1];
  wait_for_the_last_kernel();
  const int64_t row0 = (int64_t)blockIdx.x * kRowsBlock + threadIdx.x;  // and 256, 512, 768 on
  const bool ok = a.ws->ok;
  const int top = a.ws->top, B = a.t.B, rows = a.offs[B];
  const bool some = ok && row0 - threadIdx.x < rows;
  if (some) {
    if (threadIdx.x < 32) {
      const int v = (int)(row0 - threadIdx.x);
      int lo = 0, n = B;  // the sequence is among [lo, lo + n)
      while (n > 1) {
        const int step = (n + 31) / 32, p = lo + (int)threadIdx.x * step;
        const uint32_t le = __ballot_sync(0xffffffffu, p < lo + n && a.offs[p] <= v);
        const int k = 31 - __clz(le);  // (probe 0 always is)
        n = imin(step, n - k * step);
        lo += k * step;
      }
      if (threadIdx.x == 0) first = lo;
    }
    __syncthreads();
    for (int i = threadIdx.x; i <= kRowsBlock; i += 256) win[i] = a.offs[imin(first + i, B)];
    __syncthreads();
  }
  constexpr int N = kRowsBlock / 256;
  int64_t row[N], slot[N];
  int b[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    row[i] = row0 + 256 * i;
    b[i] = -1;
    slot[i] = -1;
    if (some && row[i] < rows)
      b[i] = (int)row[i] < win[kRowsBlock]
                 ? first + last_at_most(win, kRowsBlock - 1, (int)row[i])
                 : last_at_most(a.offs, B - 1, (int)row[i]);
  }
  if (some) plan_rows<N>(a, top, row, b, slot);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (row[i] < a.T) a.slots[row[i]] = slot[i];
    if (ok && row[i] < B) plan_length(a, (int)row[i]);
  }
}

// A thread a row, and a thread a sequence's check.
__global__ void __launch_bounds__(256)
    slot_map_kernel(CacheTab t, const int32_t* offs, int64_t T, int64_t* slots) {
  const int64_t row = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool on = cache_status(t) == 0;
  if (on && row < t.B) {
    const int b = (int)row, o0 = offs[b], o1 = offs[b + 1], len = t.lengths[b];
    if ((b == 0 && o0 != 0) || o0 < 0 || o1 < o0 || (int64_t)o1 > T || len < 0 ||
        len > t.M * t.ps || o1 - o0 > len)
      cache_fail(t, HSTU_SLA_ERR_BAD_INPUT);
  }
  if (row >= T) return;
  int64_t slot = -1;
  if (on && row < offs[t.B] && offs[0] == 0) {
    const int b = last_at_most(offs, t.B - 1, (int)row);
    const int n = offs[b + 1] - offs[b], r = (int)row - offs[b];
    const int len = t.lengths[b];
    const int pos = len - n + r;
    if (r >= 0 && r < n && n <= len && len <= t.M * t.ps) {
      const int page = t.bt[(int64_t)b * t.M + (pos >> t.lps)];
      if (page >= 0 && page < t.P)
        slot = (int64_t)page * t.ps + (pos & (t.ps - 1));
      else
        cache_fail(t, HSTU_SLA_ERR_BAD_INPUT);
    }
  }
  slots[row] = slot;
}

}  // namespace

size_t cache_plan_ws_bytes(int B, int64_t T) {
  if (T <= kOneBlockRows && B <= kOneBlockSeqs) return 0;
  return align256(sizeof(PlanWs) + sizeof(int32_t) * (3 * (size_t)B + 2));
}

cudaError_t launch_cache_plan(const CacheTab& t, const int32_t* offs, const int32_t* nts,
                              const int32_t* release, int64_t T, int64_t* slots, void* ws,
                              cudaStream_t st) {
  PlanArgs a;
  a.t = t;
  a.offs = offs;
  a.nts = nts;
  a.release = release;
  a.T = T;
  a.slots = slots;
  a.ws = static_cast<PlanWs*>(ws);
  a.old = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + sizeof(PlanWs));
  a.need_sum = a.old + t.B;
  a.given_sum = a.need_sum + t.B + 1;
  if (T <= kOneBlockRows && t.B <= kOneBlockSeqs) {
    if (t.B <= kThreads) plan_one_kernel<1><<<1, kThreads, 0, st>>>(a);
    else plan_one_kernel<4><<<1, kThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  if (t.B <= kThreads) plan_sums_kernel<1><<<1, kThreads, 0, st>>>(a);
  else plan_sums_kernel<4><<<1, kThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && release)
    e = launch_early(plan_push_kernel, (unsigned)((t.B + 7) / 8), 256, st, a);
  if (e == cudaSuccess) {
    const int64_t n = T > t.B ? T : t.B;  // a thread a row, and a thread a length
    e = launch_early(plan_rows_kernel, (unsigned)((n + kRowsBlock - 1) / kRowsBlock), 256, st, a);
  }
  return e;
}

cudaError_t launch_cache_slot_map(const CacheTab& t, const int32_t* offs, int64_t T,
                                  int64_t* slots, cudaStream_t st) {
  const int64_t n = T > t.B ? T : t.B;
  slot_map_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(t, offs, T, slots);
  return cudaGetLastError();
}

}  // namespace hstu
