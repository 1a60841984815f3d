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
// sums in one block and the per-page and per-row work in a grid.
#include "cache_common.cuh"

namespace hstu {

namespace {

constexpr int kThreads = 1024;

// Per-sequence sums of the plan, in the caller's workspace.
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

// The block's part: checks, sums, new lengths and stack height.  All or
// nothing: the tables change only if every sequence's step can be done.
__device__ bool plan_sums(const PlanArgs& a) {
  __shared__ int sm[2][32];
  __shared__ int s_code;
  const CacheTab& t = a.t;
  const int fc = *t.free_count;
  if (threadIdx.x == 0) s_code = fc < 0 || fc > t.P ? HSTU_SLA_ERR_BAD_INPUT : 0;
  __syncthreads();
  int64_t base_need = 0, base_given = 0;
  for (int c = 0; c < t.B; c += kThreads) {
    const int b = c + threadIdx.x;
    int need = 0, given = 0, old = 0;
    if (b < t.B) {
      const int o0 = a.offs[b], o1 = a.offs[b + 1], len = t.lengths[b];
      const int nt = a.nts ? a.nts[b] : 0;
      const bool rel = a.release && a.release[b] != 0;
      const int most = t.M * t.ps;
      const bool bad = (b == 0 && o0 != 0) || o0 < 0 || o1 < o0 || (int64_t)o1 > a.T || nt < 0 ||
                       nt > o1 - o0 || len < 0 || len > most;
      old = rel ? 0 : len;
      const int fresh = bad ? 0 : o1 - o0 - nt;
      if (bad || fresh > most - old) {
        s_code = HSTU_SLA_ERR_BAD_INPUT;
        old = 0;
      } else {
        need = ((old + fresh + t.ps - 1) >> t.lps) - ((old + t.ps - 1) >> t.lps);
        given = rel ? (len + t.ps - 1) >> t.lps : 0;
      }
    }
    int xn, xg, tn, tg;
    block_scan2(need, given, &xn, &xg, &tn, &tg, sm);
    // a chunk's sums stay below 1024 * 2^20 (max_pages); over the chunks they
    // are held at 2^31 - 1, above any num_pages, where the step fails anyway
    const int64_t most = 0x7fffffff;
    if (b < t.B) {
      a.old[b] = old;
      a.need_sum[b] = (int32_t)min(base_need + xn, most);
      a.given_sum[b] = (int32_t)min(base_given + xg, most);
    }
    base_need = min(base_need + tn, most);
    base_given = min(base_given + tg, most);
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
  if (ok) {
    for (int b = threadIdx.x; b < t.B; b += kThreads)
      t.lengths[b] = a.old[b] + a.offs[b + 1] - a.offs[b] - (a.nts ? a.nts[b] : 0);
  }
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

// Released page e (of ws->given) onto the stack.
__device__ __forceinline__ void plan_push(const PlanArgs& a, int old_top, int e) {
  const int b = last_at_most(a.given_sum, a.t.B - 1, e);
  a.t.free_pages[old_top + e] = a.t.bt[(int64_t)b * a.t.M + e - a.given_sum[b]];
}

// Row `row`: its slot, and the block-table entry if it is the first token of
// a page.  Entries below `have` are only read and the others only written, so
// rows need no order among them.
__device__ __forceinline__ void plan_row(const PlanArgs& a, int top, int64_t row) {
  int64_t slot = -1;
  const CacheTab& t = a.t;
  const int b = row < a.offs[t.B] ? last_at_most(a.offs, t.B - 1, (int)row) : -1;
  if (b >= 0) {
    const int r = (int)row - a.offs[b];
    const int fresh = a.offs[b + 1] - a.offs[b] - (a.nts ? a.nts[b] : 0);
    if (r < fresh) {
      const int old = a.old[b], pos = old + r;
      const int j = pos >> t.lps, have = (old + t.ps - 1) >> t.lps;
      int page;
      if (j < have) {
        page = t.bt[(int64_t)b * t.M + j];
      } else {
        page = t.free_pages[top - 1 - (a.need_sum[b] + j - have)];
        if ((pos & (t.ps - 1)) == 0) t.bt[(int64_t)b * t.M + j] = page;
      }
      slot = (int64_t)page * t.ps + (pos & (t.ps - 1));
    }
  }
  a.slots[row] = slot;
}

__global__ void __launch_bounds__(kThreads) plan_one_kernel(PlanArgs a) {
  const bool ok = plan_sums(a);
  if (!ok) {
    for (int64_t r = threadIdx.x; r < a.T; r += kThreads) a.slots[r] = -1;
    return;
  }
  const int given = a.ws->given, old_top = a.ws->old_top, top = a.ws->top;
  for (int e = threadIdx.x; e < given; e += kThreads) plan_push(a, old_top, e);
  __syncthreads();
  for (int64_t r = threadIdx.x; r < a.T; r += kThreads) plan_row(a, top, r);
}

__global__ void __launch_bounds__(kThreads) plan_sums_kernel(PlanArgs a) { plan_sums(a); }

__global__ void __launch_bounds__(256) plan_push_kernel(PlanArgs a) {
  if (!a.ws->ok) return;
  const int given = a.ws->given, old_top = a.ws->old_top;
  for (int e = blockIdx.x * 256 + threadIdx.x; e < given; e += gridDim.x * 256)
    plan_push(a, old_top, e);
}

__global__ void __launch_bounds__(256) plan_rows_kernel(PlanArgs a) {
  const int64_t row = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (row >= a.T) return;
  if (!a.ws->ok) {
    a.slots[row] = -1;
    return;
  }
  plan_row(a, a.ws->top, row);
}

__global__ void __launch_bounds__(256)
    slot_map_kernel(CacheTab t, const int32_t* offs, int64_t T, int64_t* slots) {
  const int64_t row = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (row >= T) return;
  int64_t slot = -1;
  if (cache_status(t) == 0 && row < offs[t.B] && offs[0] == 0) {
    const int b = last_at_most(offs, t.B - 1, (int)row);
    const int n = offs[b + 1] - offs[b], r = (int)row - offs[b];
    const int len = t.lengths[b];
    const int pos = len - n + r;
    bool ok = r >= 0 && r < n && n <= len && len <= t.M * t.ps;
    if (ok) {
      const int page = t.bt[(int64_t)b * t.M + (pos >> t.lps)];
      ok = page >= 0 && page < t.P;
      slot = ok ? (int64_t)page * t.ps + (pos & (t.ps - 1)) : -1;
    }
    if (!ok) cache_fail(t, HSTU_SLA_ERR_BAD_INPUT);
  } else if (row == 0 && offs[0] != 0) {
    cache_fail(t, HSTU_SLA_ERR_BAD_INPUT);
  }
  slots[row] = slot;
}

// Rows up to which one block does the whole step.
constexpr int64_t kOneBlockRows = 8192;

}  // namespace

size_t cache_plan_ws_bytes(int B) {
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
  if (T <= kOneBlockRows) {
    plan_one_kernel<<<1, kThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  plan_sums_kernel<<<1, kThreads, 0, st>>>(a);
  if (release) plan_push_kernel<<<148, 256, 0, st>>>(a);
  plan_rows_kernel<<<(unsigned)((T + 255) / 256), 256, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache_slot_map(const CacheTab& t, const int32_t* offs, int64_t T,
                                  int64_t* slots, cudaStream_t st) {
  if (T == 0) return cudaSuccess;
  slot_map_kernel<<<(unsigned)((T + 255) / 256), 256, 0, st>>>(t, offs, T, slots);
  return cudaGetLastError();
}

}  // namespace hstu
