// C ABI of the paged 4-bit history cache: host-side argument checks and
// launches.  See include/hstu_cache.h.
#include <math.h>
#include <string.h>

#include "cache_common.cuh"

namespace hstu {
size_t cache_plan_ws_bytes(int B, int64_t T);
}

using namespace hstu;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int make_tab(const hstu_cache_tables* t, CacheTab* c) {
  if (t == nullptr) return HSTU_SLA_ERR_INVALID_ARG;
  if (t->page_size != 16 && t->page_size != 32 && t->page_size != 64)
    return HSTU_SLA_ERR_UNSUPPORTED;
  if (t->B < 1 || t->num_pages < 1 || t->max_pages < 1) return HSTU_SLA_ERR_INVALID_ARG;
  if (t->max_pages > (1 << 19) || t->B > (1 << 30)) return HSTU_SLA_ERR_UNSUPPORTED;
  const void* ptrs[] = {t->status, t->free_count, t->lengths, t->free_pages, t->block_table};
  for (const void* p : ptrs)
    if (p == nullptr || !aligned(p, 4)) return HSTU_SLA_ERR_INVALID_ARG;
  c->status = t->status;
  c->free_count = t->free_count;
  c->lengths = t->lengths;
  c->free_pages = t->free_pages;
  c->bt = t->block_table;
  c->B = t->B;
  c->M = t->max_pages;
  c->P = t->num_pages;
  c->ps = t->page_size;
  c->lps = t->page_size == 16 ? 4 : t->page_size == 32 ? 5 : 6;
  return HSTU_SLA_OK;
}

int check_rows(const void* p, int64_t rs, int H, int d) {
  if (p == nullptr || !aligned(p, 16)) return HSTU_SLA_ERR_INVALID_ARG;
  if (rs < (int64_t)H * d || rs % 8 != 0) return HSTU_SLA_ERR_INVALID_ARG;
  return HSTU_SLA_OK;
}

int check_heads(int H, int d, int64_t T) {
  if (H < 1 || T < 0) return HSTU_SLA_ERR_INVALID_ARG;
  if (d != 32 && d != 64 && d != 128) return HSTU_SLA_ERR_UNSUPPORTED;
  if (H > 65535 || T > INT32_MAX) return HSTU_SLA_ERR_UNSUPPORTED;
  return HSTU_SLA_OK;
}

int check_pages(const void* pages, int64_t stride, int H, int d, int ps) {
  if (pages == nullptr || !aligned(pages, 16)) return HSTU_SLA_ERR_INVALID_ARG;
  if (stride < (int64_t)H * ps * (d + 8) || stride % 16 != 0) return HSTU_SLA_ERR_INVALID_ARG;
  return HSTU_SLA_OK;
}

int rows_args(const hstu_cache_tables* t, const hstu_cache_rows* r, CacheRowArgs* a) {
  int e = make_tab(t, &a->t);
  if (e) return e;
  if (r == nullptr) return HSTU_SLA_ERR_INVALID_ARG;
  if ((e = check_heads(r->H, r->d, r->T))) return e;
  if ((e = check_pages(r->pages, r->page_stride, r->H, r->d, t->page_size))) return e;
  if (r->T > 0) {
    if (r->slots == nullptr || !aligned(r->slots, 8)) return HSTU_SLA_ERR_INVALID_ARG;
    if ((e = check_rows(r->k, r->k_row_stride, r->H, r->d))) return e;
    if ((e = check_rows(r->v, r->v_row_stride, r->H, r->d))) return e;
  }
  a->H = r->H;
  a->T = r->T;
  a->slots = r->slots;
  a->pages = static_cast<uint8_t*>(r->pages);
  a->page_stride = r->page_stride;
  a->k = static_cast<bf16*>(r->k);
  a->v = static_cast<bf16*>(r->v);
  a->k_rs = r->k_row_stride;
  a->v_rs = r->v_row_stride;
  return HSTU_SLA_OK;
}

int attend_args(const hstu_cache_tables* t, const hstu_cache_attend_params* p, CacheAttnArgs* out) {
  CacheAttnArgs& a = *out;
  memset(&a, 0, sizeof(a));
  int e = make_tab(t, &a.t);
  if (e) return e;
  if (p == nullptr || p->seq_offsets == nullptr) return HSTU_SLA_ERR_INVALID_ARG;
  if ((e = check_heads(p->H, p->d, p->total_tokens))) return e;
  if (p->max_new < 0 || p->K1 < 0 || p->K2 < 0 || p->contextual_len < 0)
    return HSTU_SLA_ERR_INVALID_ARG;
  if (!(p->N > 0.f) || !isfinite(p->N) || !isfinite(p->alpha)) return HSTU_SLA_ERR_INVALID_ARG;
  if ((e = check_pages(p->pages, p->page_stride, p->H, p->d, t->page_size))) return e;
  if (p->total_tokens > 0) {
    if ((e = check_rows(p->q, p->q_row_stride, p->H, p->d))) return e;
    if ((e = check_rows(p->out, p->out_row_stride, p->H, p->d))) return e;
    if (p->num_targets) {
      if ((e = check_rows(p->k, p->k_row_stride, p->H, p->d))) return e;
      if ((e = check_rows(p->v, p->v_row_stride, p->H, p->d))) return e;
    }
  }
  a.H = p->H;
  a.max_new = (int)(p->max_new < p->total_tokens ? p->max_new : p->total_tokens);
  a.T = p->total_tokens;
  a.offs = p->seq_offsets;
  a.nts = p->num_targets;
  a.K1 = p->K1;
  a.K2e = p->K2 > p->contextual_len ? p->K2 : p->contextual_len;
  a.alpha = p->alpha;
  a.inv_n = 1.0f / p->N;
  a.q = static_cast<const bf16*>(p->q);
  a.k = static_cast<const bf16*>(p->k);
  a.v = static_cast<const bf16*>(p->v);
  a.q_rs = p->q_row_stride;
  a.k_rs = p->k_row_stride;
  a.v_rs = p->v_row_stride;
  a.pages = static_cast<const uint8_t*>(p->pages);
  a.page_stride = p->page_stride;
  a.out = static_cast<bf16*>(p->out);
  a.o_rs = p->out_row_stride;
  return HSTU_SLA_OK;
}

// (cudaErrorNotSupported: the launch's own, more blocks than a grid has)
int status_of(cudaError_t e) {
  return e == cudaSuccess             ? HSTU_SLA_OK
         : e == cudaErrorNotSupported ? HSTU_SLA_ERR_UNSUPPORTED
                                      : HSTU_SLA_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t hstu_cache_plan_workspace_bytes(int32_t B, int64_t total_tokens) {
  return B < 1 || total_tokens < 0 ? 0 : cache_plan_ws_bytes(B, total_tokens);
}

int hstu_cache_plan(const hstu_cache_tables* t, const int32_t* seq_offsets,
                    const int32_t* num_targets, const int32_t* release, int64_t total_tokens,
                    int64_t* slots, void* workspace, size_t workspace_bytes,
                    hstu_stream_t stream) {
  CacheTab c;
  const int e = make_tab(t, &c);
  if (e) return e;
  if (seq_offsets == nullptr || total_tokens < 0) return HSTU_SLA_ERR_INVALID_ARG;
  if (total_tokens > INT32_MAX) return HSTU_SLA_ERR_UNSUPPORTED;
  if (total_tokens > 0 && (slots == nullptr || !aligned(slots, 8))) return HSTU_SLA_ERR_INVALID_ARG;
  const size_t need = cache_plan_ws_bytes(c.B, total_tokens);
  if (need > 0 && (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < need))
    return HSTU_SLA_ERR_WORKSPACE;
  return status_of(launch_cache_plan(c, seq_offsets, num_targets, release, total_tokens, slots,
                                     workspace, reinterpret_cast<cudaStream_t>(stream)));
}

int hstu_cache_slot_map(const hstu_cache_tables* t, const int32_t* seq_offsets,
                        int64_t total_tokens, int64_t* slots, hstu_stream_t stream) {
  CacheTab c;
  const int e = make_tab(t, &c);
  if (e) return e;
  if (seq_offsets == nullptr || total_tokens < 0) return HSTU_SLA_ERR_INVALID_ARG;
  if (total_tokens > INT32_MAX) return HSTU_SLA_ERR_UNSUPPORTED;
  if (total_tokens > 0 && (slots == nullptr || !aligned(slots, 8))) return HSTU_SLA_ERR_INVALID_ARG;
  return status_of(launch_cache_slot_map(c, seq_offsets, total_tokens, slots,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

int hstu_cache_append(const hstu_cache_tables* t, const hstu_cache_rows* r,
                      hstu_stream_t stream) {
  CacheRowArgs a;
  const int e = rows_args(t, r, &a);
  if (e) return e;
  return status_of(launch_cache_append(a, r->d, reinterpret_cast<cudaStream_t>(stream)));
}

int hstu_cache_read(const hstu_cache_tables* t, const hstu_cache_rows* r, hstu_stream_t stream) {
  CacheRowArgs a;
  const int e = rows_args(t, r, &a);
  if (e) return e;
  return status_of(launch_cache_read(a, r->d, reinterpret_cast<cudaStream_t>(stream)));
}

size_t hstu_cache_attend_workspace_bytes(const hstu_cache_tables* t,
                                         const hstu_cache_attend_params* p) {
  CacheAttnArgs a;
  return attend_args(t, p, &a) ? 0 : cache_attend_ws_bytes(a, p->d);
}

int hstu_cache_attend(const hstu_cache_tables* t, const hstu_cache_attend_params* p,
                      void* workspace, size_t workspace_bytes, hstu_stream_t stream) {
  CacheAttnArgs a;
  const int e = attend_args(t, p, &a);
  if (e) return e;
  const size_t need = cache_attend_ws_bytes(a, p->d);
  if (need > 0 && (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < need))
    return HSTU_SLA_ERR_WORKSPACE;
  return status_of(
      launch_cache_attend(a, p->d, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

int hstu_cache_get_error(const hstu_cache_tables* t, hstu_stream_t stream) {
  CacheTab c;
  const int e = make_tab(t, &c);
  if (e) return e;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int32_t status = 0;
  cudaError_t ce = cudaMemcpyAsync(&status, c.status, sizeof(status), cudaMemcpyDeviceToHost, st);
  if (ce == cudaSuccess) ce = cudaStreamSynchronize(st);
  return ce == cudaSuccess ? status : HSTU_SLA_ERR_CUDA;
}

}  // extern "C"
