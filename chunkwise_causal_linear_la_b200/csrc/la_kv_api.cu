// la_kv_api.cu -- C ABI of the paged cache and the attention over it: argument
// checks, kernel selection and launch (la_kv_write, la_kv_read, la_paged_attn).
#include <cuda_runtime.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "la_internal.h"

namespace la {
namespace {

la_status fail(la_status s, const char *fmt, ...) {
  char msg[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  return report_error(s, msg);
}

la_status ok() { return report_error(LA_OK, ""); }

bool head_dim_ok(int64_t d) { return d == 16 || d == 32 || d == 64 || d == 128 || d == 256; }

constexpr int32_t kAttnFlags = LA_FLAG_SIMT | LA_FLAG_TEST_WAIT_TIMEOUT;
constexpr int64_t kMaxElems = (int64_t)1 << 34;  // B T H D: 2^31 threads of eight elements

// Positive sizes whose product stays within `most` (no overflow on the way).
bool within(int64_t most, int64_t a, int64_t b, int64_t c = 1, int64_t d = 1) {
  if (a == 0 || b == 0 || c == 0 || d == 0) return true;
  if (a > most / b) return false;
  if (a * b > most / c) return false;
  return a * b * c <= most / d;
}

la_status check_dense(const la_tensor *t, const char *name) {
  if (!t) return fail(LA_ERR_INVALID_ARG, "%s: NULL tensor descriptor", name);
  if (t->dtype != LA_F32 && t->dtype != LA_BF16)
    return fail(LA_ERR_INVALID_ARG, "%s: dtype %d is not LA_F32 or LA_BF16", name, t->dtype);
  if (t->B < 0 || t->T < 0 || t->H <= 0 || t->D <= 0)
    return fail(LA_ERR_INVALID_ARG, "%s: negative or zero size", name);
  if (t->stride_b < 0 || t->stride_t < 0 || t->stride_h < 0)
    return fail(LA_ERR_INVALID_ARG, "%s: negative stride", name);
  if (!head_dim_ok(t->D))
    return fail(LA_ERR_UNSUPPORTED, "%s: head dim %lld not in {16, 32, 64, 128, 256}", name, (long long)t->D);
  if (!within(kMaxElems, t->B, t->T, t->H, t->D) || !within(((int64_t)1 << 31) - 1, t->B, t->T, t->H))
    return fail(LA_ERR_UNSUPPORTED, "%s: more than 2^34 elements or 2^31 - 1 rows", name);
  if (t->B * t->T > 0 && !t->data) return fail(LA_ERR_INVALID_ARG, "%s: NULL data pointer", name);
  const int es = t->dtype == LA_F32 ? 4 : 2;
  if (((uintptr_t)t->data) % 16 != 0) return fail(LA_ERR_INVALID_ARG, "%s: data pointer not 16-byte aligned", name);
  // an axis of one entry is never stepped along: its stride may be anything
  if ((t->B > 1 && (t->stride_b * es) % 16) || (t->T > 1 && (t->stride_t * es) % 16) ||
      (t->H > 1 && (t->stride_h * es) % 16))
    return fail(LA_ERR_INVALID_ARG, "%s: strides must be multiples of 16 bytes", name);
  return LA_OK;
}

// Written tensors: a zero stride along a longer axis would make rows overlap.
la_status check_written(const la_tensor *t, const char *name) {
  if ((t->B > 1 && t->stride_b == 0) || (t->T > 1 && t->stride_t == 0) || (t->H > 1 && t->stride_h == 0))
    return fail(LA_ERR_INVALID_ARG, "%s: zero stride in a tensor that is written", name);
  return LA_OK;
}

la_status check_cache(const la_kv_cache *c, const int32_t *page_table, int64_t max_pages, int64_t n_seqs) {
  if (!c) return fail(LA_ERR_INVALID_ARG, "cache: NULL descriptor");
  if (c->format != LA_KV_BF16 && c->format != LA_KV_E4M3 && c->format != LA_KV_INT8)
    return fail(LA_ERR_INVALID_ARG, "cache: format %d unknown", c->format);
  if (c->n_pages < 0 || c->page_size <= 0 || c->H <= 0 || c->D <= 0)
    return fail(LA_ERR_INVALID_ARG, "cache: negative or zero size");
  if (!head_dim_ok(c->D))
    return fail(LA_ERR_UNSUPPORTED, "cache: head dim %lld not in {16, 32, 64, 128, 256}", (long long)c->D);
  if (c->page_size > 65536 || c->H > 65536 || c->n_pages > 0x7FFFFFFF)
    return fail(LA_ERR_UNSUPPORTED, "cache: page_size or H over 65536, or n_pages over 2^31 - 1");
  const int es = c->format == LA_KV_BF16 ? 2 : 1;
  const int64_t st[3] = {c->stride_page, c->stride_token, c->stride_head};
  const int64_t sz[3] = {c->n_pages, c->page_size, c->H};
  const char *nm[3] = {"page", "token", "head"};
  for (int i = 0; i < 3; ++i) {
    if (sz[i] <= 1) continue;
    if (st[i] <= 0 || (st[i] * es) % 16)
      return fail(LA_ERR_INVALID_ARG, "cache: stride of the %s axis must be a positive multiple of 16 bytes", nm[i]);
    if (st[i] >= ((int64_t)1 << 39) / es)
      return fail(LA_ERR_UNSUPPORTED, "cache: stride of the %s axis over 2^39 bytes", nm[i]);
  }
  if (c->n_pages > 0 && (!c->k || !c->v)) return fail(LA_ERR_INVALID_ARG, "cache: NULL k or v");
  if (((uintptr_t)c->k) % 16 || ((uintptr_t)c->v) % 16)
    return fail(LA_ERR_INVALID_ARG, "cache: k or v not 16-byte aligned");
  if (c->format != LA_KV_BF16) {
    if (c->n_pages > 0 && (!c->k_scale || !c->v_scale))
      return fail(LA_ERR_INVALID_ARG, "cache: the 8-bit formats need k_scale and v_scale");
    if (((uintptr_t)c->k_scale) % 16 || ((uintptr_t)c->v_scale) % 16)
      return fail(LA_ERR_INVALID_ARG, "cache: k_scale or v_scale not 16-byte aligned");
  }
  if (n_seqs < 0) return fail(LA_ERR_INVALID_ARG, "n_seqs is negative");
  if (max_pages < 0) return fail(LA_ERR_INVALID_ARG, "max_pages is negative");
  if (!within((int64_t)1 << 40, max_pages, c->page_size) || !within((int64_t)1 << 40, max_pages, n_seqs))
    return fail(LA_ERR_UNSUPPORTED, "page_table: over 2^40 positions or entries");
  if (n_seqs * max_pages > 0 && !page_table) return fail(LA_ERR_INVALID_ARG, "page_table is NULL");
  if (((uintptr_t)page_table) % 4) return fail(LA_ERR_INVALID_ARG, "page_table not 4-byte aligned");
  return LA_OK;
}

la_status check_seqs(const la_tensor *t, const int32_t *cu_seqlens, int64_t n_seqs) {
  if (cu_seqlens) {
    if (t->B != 1) return fail(LA_ERR_INVALID_ARG, "packed batches (cu_seqlens) need B == 1");
    if (((uintptr_t)cu_seqlens) % 4) return fail(LA_ERR_INVALID_ARG, "cu_seqlens not 4-byte aligned");
    if (t->T > 0x7FFFFFFF) return fail(LA_ERR_UNSUPPORTED, "packed batches hold at most 2^31 - 1 tokens");
  } else if (n_seqs != t->B) {
    return fail(LA_ERR_INVALID_ARG, "n_seqs must equal B when cu_seqlens is NULL");
  }
  if (n_seqs > 0x7FFFFFFE) return fail(LA_ERR_UNSUPPORTED, "more than 2^31 - 2 sequences");
  return LA_OK;
}

TensorView view(const la_tensor *t) { return TensorView{t->data, t->stride_b, t->stride_t, t->stride_h}; }

KvView kv_view(const la_kv_cache *c, const int32_t *table, int64_t max_pages) {
  KvView v;
  v.k = (uint8_t *)c->k;
  v.v = (uint8_t *)c->v;
  v.ks = c->k_scale;
  v.vs = c->v_scale;
  v.format = c->format;
  v.n_pages = c->n_pages;
  v.page_size = (int)c->page_size;
  v.H = (int)c->H;
  v.D = (int)c->D;
  v.s_page = c->stride_page;
  v.s_tok = c->stride_token;
  v.s_head = c->stride_head;
  v.table = table;
  v.max_pages = max_pages;
  return v;
}

la_status kv_move(const la_tensor *k, const la_tensor *v, const int32_t *cu_seqlens, int64_t n_seqs,
                  const la_kv_cache *cache, const int32_t *page_table, int64_t max_pages, const int32_t *pos,
                  bool write, void *stream) {
  la_status s;
  if ((s = check_dense(k, write ? "k" : "k_out")) != LA_OK) return s;
  if ((s = check_dense(v, write ? "v" : "v_out")) != LA_OK) return s;
  if (!write && ((s = check_written(k, "k_out")) != LA_OK || (s = check_written(v, "v_out")) != LA_OK)) return s;
  if (k->dtype != v->dtype) return fail(LA_ERR_INVALID_ARG, "keys and values must share one dtype");
  if (k->B != v->B || k->T != v->T || k->H != v->H || k->D != v->D)
    return fail(LA_ERR_INVALID_ARG, "keys and values disagree on B, T, H or D");
  if ((s = check_cache(cache, page_table, max_pages, n_seqs)) != LA_OK) return s;
  if (cache->H != k->H || cache->D != k->D) return fail(LA_ERR_INVALID_ARG, "the cache has other heads or head dim");
  if ((s = check_seqs(k, cu_seqlens, n_seqs)) != LA_OK) return s;
  if (((uintptr_t)pos) % 4) return fail(LA_ERR_INVALID_ARG, "%s not 4-byte aligned", write ? "kv_len" : "start");
  if (k->B * k->T == 0 || n_seqs == 0) return ok();
  if (write && !pos) return fail(LA_ERR_INVALID_ARG, "kv_len is NULL");
  KvMoveArgs a;
  a.c = kv_view(cache, page_table, max_pages);
  a.k = view(k);
  a.v = view(v);
  a.cu_seqlens = cu_seqlens;
  a.pos = pos;
  a.B = k->B;
  a.T = k->T;
  a.n_seqs = n_seqs;
  a.dtype = k->dtype;
  const cudaError_t e = write ? launch_kv_write(a, (cudaStream_t)stream) : launch_kv_read(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return fail(LA_ERR_CUDA, "cache %s kernel: %s", write ? "write" : "read", cudaGetErrorString(e));
  return ok();
}

}  // namespace
}  // namespace la

using namespace la;

extern "C" {

la_status la_kv_write(const la_tensor *k, const la_tensor *v, const int32_t *cu_seqlens, int64_t n_seqs,
                      const la_kv_cache *cache, const int32_t *page_table, int64_t max_pages, const int32_t *kv_len,
                      void *stream) {
  return kv_move(k, v, cu_seqlens, n_seqs, cache, page_table, max_pages, kv_len, true, stream);
}

la_status la_kv_read(const la_kv_cache *cache, const int32_t *page_table, int64_t max_pages, const int32_t *start,
                     const int32_t *cu_seqlens, int64_t n_seqs, const la_tensor *k_out, const la_tensor *v_out,
                     void *stream) {
  return kv_move(k_out, v_out, cu_seqlens, n_seqs, cache, page_table, max_pages, start, false, stream);
}

int32_t la_paged_attn_path(int64_t H, int64_t D, int64_t H_kv, int64_t page_size, int32_t format, int32_t dtype,
                           int32_t flags) {
  if (H <= 0 || H_kv <= 0 || H % H_kv || !head_dim_ok(D) || page_size <= 0 || page_size > 65536) return -1;
  if (format != LA_KV_BF16 && format != LA_KV_E4M3 && format != LA_KV_INT8) return -1;
  if ((dtype != LA_F32 && dtype != LA_BF16) || (flags & ~kAttnFlags)) return -1;
  return dtype == LA_BF16 && !(flags & LA_FLAG_SIMT) && pa_tc_shape(H, D, H_kv, page_size) ? 1 : 2;
}

size_t la_paged_attn_workspace_size(int64_t B, int64_t T, int64_t H, int64_t D, int64_t n_seqs,
                                    int32_t has_cu_seqlens, int64_t H_kv, int64_t page_size, int32_t format,
                                    int32_t dtype, int32_t flags) {
  const int32_t path = la_paged_attn_path(H, D, H_kv, page_size, format, dtype, flags);
  if (B < 0 || T < 0 || n_seqs < 0 || path < 0 || !within(kMaxElems, B, T, H, D) || n_seqs > 0x7FFFFFFE)
    return (size_t)-1;
  if (path == 2 || B * T == 0 || n_seqs == 0) return 0;
  return pa_workspace_bytes(B, T, H, D, n_seqs, has_cu_seqlens != 0, H_kv, kPagedCtas);
}

la_status la_paged_attn(const la_tensor *q, const la_kv_cache *cache, const int32_t *page_table, int64_t max_pages,
                        const int32_t *kv_len, const int32_t *cu_seqlens, int64_t n_seqs, float scale, int64_t window,
                        const la_tensor *out, float *lse, int32_t flags, void *workspace, size_t workspace_bytes,
                        void *stream) {
  la_status s;
  if ((s = check_dense(q, "q")) != LA_OK) return s;
  if ((s = check_dense(out, "out")) != LA_OK) return s;
  if ((s = check_written(out, "out")) != LA_OK) return s;
  if (q->dtype != out->dtype) return fail(LA_ERR_INVALID_ARG, "q and out must share one dtype");
  if (q->B != out->B || q->T != out->T || q->H != out->H || q->D != out->D)
    return fail(LA_ERR_INVALID_ARG, "q and out disagree on B, T, H or D");
  if ((s = check_cache(cache, page_table, max_pages, n_seqs)) != LA_OK) return s;
  if (cache->D != q->D) return fail(LA_ERR_INVALID_ARG, "the cache has another head dim");
  if (q->H % cache->H) return fail(LA_ERR_INVALID_ARG, "the query heads are not a multiple of the cache's heads");
  if ((s = check_seqs(q, cu_seqlens, n_seqs)) != LA_OK) return s;
  // the kernels weigh by powers of two: the scale times log2(e) has to be a number too
  if (!(scale > 0.f) || !isfinite(scale * 1.4426950408889634f))
    return fail(LA_ERR_INVALID_ARG, "scale must be positive and at most 2.35e38");
  if (window < 0) return fail(LA_ERR_INVALID_ARG, "window is negative");
  if (flags & ~kAttnFlags) return fail(LA_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
  if (((uintptr_t)lse) % 4) return fail(LA_ERR_INVALID_ARG, "lse not 4-byte aligned");
  if (((uintptr_t)kv_len) % 4) return fail(LA_ERR_INVALID_ARG, "kv_len not 4-byte aligned");
  if (workspace && ((uintptr_t)workspace) % 256 != 0)
    return fail(LA_ERR_INVALID_ARG, "workspace not 256-byte aligned");
  if (q->B * q->T == 0 || n_seqs == 0) return ok();
  if (!kv_len) return fail(LA_ERR_INVALID_ARG, "kv_len is NULL");
  PagedArgs a;
  a.c = kv_view(cache, page_table, max_pages);
  a.q = view(q);
  a.out = out->data;
  a.o_sb = out->stride_b;
  a.o_st = out->stride_t;
  a.o_sh = out->stride_h;
  a.lse = lse;
  a.cu_seqlens = cu_seqlens;
  a.kv_len = kv_len;
  a.B = q->B;
  a.T = q->T;
  a.n_seqs = n_seqs;
  a.H = (int)q->H;
  a.dtype = q->dtype;
  a.test_wait_timeout = (flags & LA_FLAG_TEST_WAIT_TIMEOUT) != 0;
  a.scale = scale;
  a.window = window > 0x7FFFFFFF ? 0 : (int)window;  // positions are int32: a wider window hides nothing
  const size_t need = la_paged_attn_workspace_size(q->B, q->T, q->H, q->D, n_seqs, cu_seqlens != nullptr, cache->H,
                                                   cache->page_size, cache->format, q->dtype, flags);
  if (need == (size_t)-1) return fail(LA_ERR_UNSUPPORTED, "the batch is too large");
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(LA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? workspace_bytes : 0);
  cudaError_t e;
  if (need > 0 && pa_tc_supported(a)) {
    int device = 0;
    if ((e = bind_device(&device)) != cudaSuccess)
      return fail(LA_ERR_CUDA, "cudaGetDevice / cudaSetDevice: %s", cudaGetErrorString(e));
    const char *why = "";
    e = launch_paged_tc(a, kPagedCtas, workspace, (cudaStream_t)stream, &why);
    if (e != cudaSuccess)
      return fail(LA_ERR_CUDA, "paged attention, tensor cores: %s%s%s", cudaGetErrorString(e), *why ? ": " : "", why);
    return ok();
  }
  e = launch_paged_simt(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return fail(LA_ERR_CUDA, "paged attention kernel: %s", cudaGetErrorString(e));
  return ok();
}

}  // extern "C"
