// C entry points of the paged-cache operators: argument checks, workspace layout, launches.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "kernels.h"
#include "paged.h"

namespace thin {
int record_error(int s, const char* msg);
}

namespace {

using namespace thin;

thin_attn_status err(thin_attn_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return (thin_attn_status)record_error((int)s, buf);
}

constexpr int64_t kIntMax = 0x7FFFFFFF;
constexpr int kMaxTop = 4096;

size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

int esize(int dtype) { return dtype == THIN_ATTN_FP32 ? 4 : dtype == THIN_ATTN_E4M3 ? 1 : 2; }
bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }
bool strides16(int es, int64_t a, int64_t b, int64_t c = 0) { return a * es % 16 == 0 && b * es % 16 == 0 && c * es % 16 == 0; }

thin_attn_status check_types(int dtype, int cache) {
  if (dtype != THIN_ATTN_FP32 && dtype != THIN_ATTN_BF16 && dtype != THIN_ATTN_FP16)
    return err(THIN_ATTN_EINVAL, "dtype %d", dtype);
  if (cache != dtype && !(cache == THIN_ATTN_E4M3 && dtype != THIN_ATTN_FP32))
    return err(THIN_ATTN_EUNSUPPORTED, "cache type %d with type %d: the same type, or e4m3 under bf16 or fp16", cache,
               dtype);
  return THIN_ATTN_OK;
}

thin_attn_status check_pool(int cache, int H, int E, int D, int page, int n_pages) {
  const int m = cache == THIN_ATTN_E4M3 ? 16 : 8;
  if (E < 8 || E > 256 || E % m || D < 8 || D > 256 || D % m)
    return err(THIN_ATTN_EINVAL, "E=%d D=%d: widths must be multiples of %d in [8, 256]", E, D, m);
  if (H < 1 || page < 1 || n_pages < 1) return err(THIN_ATTN_EINVAL, "H=%d page=%d n_pages=%d must be >= 1", H, page, n_pages);
  if ((int64_t)page * n_pages > kIntMax * 64) return err(THIN_ATTN_EINVAL, "pool of %d pages of %d slots too large", n_pages, page);
  if (page > 65536) return err(THIN_ATTN_EINVAL, "page=%d above 65536", page);
  return THIN_ATTN_OK;
}

thin_attn_status check_attention(const thin_attn_paged_attention_args* a) {
  if (!a) return err(THIN_ATTN_EINVAL, "args is null");
  if (a->struct_size != sizeof *a) return err(THIN_ATTN_EINVAL, "struct_size %u, not %zu", a->struct_size, sizeof *a);
  thin_attn_status s = check_types(a->dtype, a->cache_dtype);
  if (s == THIN_ATTN_OK) s = check_pool(a->cache_dtype, a->H, a->E, a->D, a->page, a->n_pages);
  if (s != THIN_ATTN_OK) return s;
  if (a->N < 0 || a->R < 0 || a->W < 0) return err(THIN_ATTN_EINVAL, "N=%d R=%d W=%d must be >= 0", a->N, a->R, a->W);
  if (a->Hq < a->H || a->Hq % a->H) return err(THIN_ATTN_EINVAL, "%d query heads over %d key heads", a->Hq, a->H);
  if ((int64_t)a->N * a->Hq > kIntMax / 64) return err(THIN_ATTN_EINVAL, "N * Hq = %lld too large", (long long)a->N * a->Hq);
  if ((int64_t)a->W * a->page > kIntMax - 4096) return err(THIN_ATTN_EINVAL, "W * page = %lld too large", (long long)a->W * a->page);
  if (!a->rows && a->N > a->R) return err(THIN_ATTN_EINVAL, "%d tokens without rows over %d requests", a->N, a->R);
  if (!(a->scale >= 0.f && a->scale <= 2.3e38f))   // scale log2 e is a finite number too
    return err(THIN_ATTN_EINVAL, "scale=%g: expected 0 to 2.3e38", a->scale);
  if (a->window < 0) return err(THIN_ATTN_EINVAL, "window=%d", a->window);
  if (a->top < 0 || a->top > kMaxTop) return err(THIN_ATTN_EINVAL, "top=%d outside 0..%d", a->top, kMaxTop);
  if (a->top) {
    if (a->window) return err(THIN_ATTN_EUNSUPPORTED, "page selection takes no window");
    if (a->first < 0 || a->last < 1 || (int64_t)a->first + a->last > a->top)
      return err(THIN_ATTN_EINVAL, "first=%d last=%d top=%d: need first >= 0, last >= 1, first + last <= top", a->first,
                 a->last, a->top);
    if (a->N > 65535 || a->H > 65535) return err(THIN_ATTN_EUNSUPPORTED, "page selection of %d tokens, %d heads: at most 65535", a->N, a->H);
    if ((int64_t)a->N * a->H * a->W > kIntMax) return err(THIN_ATTN_EUNSUPPORTED, "page selection over N * H * W = %lld pages", (long long)a->N * a->H * a->W);
    if (a->Hq / a->H > kMaxGroup)
      return err(THIN_ATTN_EUNSUPPORTED, "page selection with %d queries per key head: at most %d", a->Hq / a->H, kMaxGroup);
  }
  return THIN_ATTN_OK;
}

struct Layout {
  size_t ids, keys, words, attn, bytes;
};
Layout layout_of(const thin_attn_paged_attention_args& a) {
  Layout l{};
  size_t at = 0;
  if (a.top) {
    l.ids = at;
    at += al256((size_t)a.N * a.H * a.top * 4);
    l.keys = at;
    at += al256((size_t)a.N * 4);
    l.words = at;
    at += al256(paged_select_workspace(a));
  }
  l.attn = at;
  l.bytes = at + al256(paged_attention_workspace(a));
  return l;
}

thin_attn_status launched(cudaError_t e, const char* what) {
  if (e != cudaSuccess) return err(THIN_ATTN_ECUDA, "%s: %s", what, cudaGetErrorString(e));
  return THIN_ATTN_OK;
}

}  // namespace

extern "C" {

thin_attn_status thin_attn_paged_plan(const thin_attn_paged_plan_args* a, void* stream) {
  if (!a) return err(THIN_ATTN_EINVAL, "args is null");
  if (a->struct_size != sizeof *a) return err(THIN_ATTN_EINVAL, "struct_size %u, not %zu", a->struct_size, sizeof *a);
  if (a->R < 0 || a->W < 0 || a->page < 1 || a->n_pages < 0 || a->max_tokens < 0)
    return err(THIN_ATTN_EINVAL, "R=%d W=%d page=%d n_pages=%d max_tokens=%d", a->R, a->W, a->page, a->n_pages, a->max_tokens);
  if (a->R > kMaxRequests) return err(THIN_ATTN_EUNSUPPORTED, "%d requests, at most %d", a->R, kMaxRequests);
  if (a->max_tokens > kIntMax / 2) return err(THIN_ATTN_EUNSUPPORTED, "max_tokens=%d, at most %lld", a->max_tokens, (long long)kIntMax / 2);
  if (a->R > 1 && a->table_row < a->W) return err(THIN_ATTN_EINVAL, "table rows of %d ids, %lld apart, overlap", a->W, (long long)a->table_row);
  if (a->R && (!a->lengths || !a->n_new || !a->lengths_out || !a->status)) return err(THIN_ATTN_EINVAL, "null request array");
  if (a->R && a->W && !a->table) return err(THIN_ATTN_EINVAL, "null table");
  if (a->n_pages && !a->free_pages) return err(THIN_ATTN_EINVAL, "null free_pages");
  if (!a->n_free || !a->n_free_out || !a->cu) return err(THIN_ATTN_EINVAL, "null n_free or cu");
  if (a->max_tokens && (!a->slots || !a->rows || !a->context)) return err(THIN_ATTN_EINVAL, "null token array");
  DeviceGuard dg(a->device);
  if (!dg.ok) return err(THIN_ATTN_ECUDA, "cannot select device %d", a->device);
  return launched(launch_paged_plan(*a, (cudaStream_t)stream), "paged plan");
}

thin_attn_status thin_attn_paged_release(const thin_attn_paged_release_args* a, void* stream) {
  if (!a) return err(THIN_ATTN_EINVAL, "args is null");
  if (a->struct_size != sizeof *a) return err(THIN_ATTN_EINVAL, "struct_size %u, not %zu", a->struct_size, sizeof *a);
  if (a->R < 0 || a->W < 0 || a->page < 1 || a->n_pages < 0)
    return err(THIN_ATTN_EINVAL, "R=%d W=%d page=%d n_pages=%d", a->R, a->W, a->page, a->n_pages);
  if (a->R > kMaxRequests) return err(THIN_ATTN_EUNSUPPORTED, "%d requests, at most %d", a->R, kMaxRequests);
  if (a->R > 1 && a->table_row < a->W) return err(THIN_ATTN_EINVAL, "table rows of %d ids, %lld apart, overlap", a->W, (long long)a->table_row);
  if (a->R == 0) return THIN_ATTN_OK;
  if (!a->keep || !a->lengths || !a->n_free || (a->W && !a->table) || (a->n_pages && !a->free_pages))
    return err(THIN_ATTN_EINVAL, "null array");
  DeviceGuard dg(a->device);
  if (!dg.ok) return err(THIN_ATTN_ECUDA, "cannot select device %d", a->device);
  return launched(launch_paged_release(*a, (cudaStream_t)stream), "paged release");
}

thin_attn_status thin_attn_paged_append(const thin_attn_paged_append_args* a, void* stream) {
  if (!a) return err(THIN_ATTN_EINVAL, "args is null");
  if (a->struct_size != sizeof *a) return err(THIN_ATTN_EINVAL, "struct_size %u, not %zu", a->struct_size, sizeof *a);
  thin_attn_status s = check_types(a->dtype, a->cache_dtype);
  if (s == THIN_ATTN_OK) s = check_pool(a->cache_dtype, a->H, a->E, a->D, a->page, a->n_pages);
  if (s != THIN_ATTN_OK) return s;
  if (a->N < 0) return err(THIN_ATTN_EINVAL, "N=%d", a->N);
  if ((int64_t)a->N * a->H > kIntMax / 64) return err(THIN_ATTN_EINVAL, "N * H = %lld too large", (long long)a->N * a->H);
  if (a->N == 0) return THIN_ATTN_OK;
  if (!a->k || !a->v || !a->slots || !a->k_pages || !a->v_pages) return err(THIN_ATTN_EINVAL, "null tensor pointer");
  if (a->cache_dtype == THIN_ATTN_E4M3 && (!a->k_scale || !a->v_scale)) return err(THIN_ATTN_EINVAL, "e4m3 needs k_scale and v_scale");
  if (!a->bounds != !a->exps) return err(THIN_ATTN_EINVAL, "bounds and exps go together");
  const int es = esize(a->dtype), cs = esize(a->cache_dtype);
  if (!aligned16(a->k) || !aligned16(a->v) || !aligned16(a->k_pages) || !aligned16(a->v_pages) ||
      !strides16(es, a->k_token, a->k_head) || !strides16(es, a->v_token, a->v_head) ||
      !strides16(cs, a->kp_page, a->kp_head, a->kp_row) || !strides16(cs, a->vp_page, a->vp_head, a->vp_row))
    return err(THIN_ATTN_EINVAL, "tensor pointers and strides must be multiples of 16 bytes");
  if (a->bounds && (uintptr_t)a->bounds % 8) return err(THIN_ATTN_EINVAL, "bounds must be 8-byte aligned");
  DeviceGuard dg(a->device);
  if (!dg.ok) return err(THIN_ATTN_ECUDA, "cannot select device %d", a->device);
  return launched(launch_paged_append(*a, (cudaStream_t)stream), "paged append");
}

thin_attn_status thin_attn_paged_attention_workspace(const thin_attn_paged_attention_args* a, size_t* bytes) {
  if (!bytes) return err(THIN_ATTN_EINVAL, "bytes is null");
  *bytes = 0;
  thin_attn_status s = check_attention(a);
  if (s != THIN_ATTN_OK) return s;
  *bytes = layout_of(*a).bytes;
  return THIN_ATTN_OK;
}

thin_attn_status thin_attn_paged_attention(const thin_attn_paged_attention_args* a, void* stream) {
  thin_attn_status s = check_attention(a);
  if (s != THIN_ATTN_OK) return s;
  if (a->N == 0) return THIN_ATTN_OK;
  if (!a->q || !a->k_pages || !a->v_pages || !a->lengths || !a->out || (a->W && a->R && !a->table))
    return err(THIN_ATTN_EINVAL, "null tensor pointer");
  if (a->cache_dtype == THIN_ATTN_E4M3 && (!a->k_scale || !a->v_scale)) return err(THIN_ATTN_EINVAL, "e4m3 needs k_scale and v_scale");
  if (a->top && (!a->bounds || !a->exps)) return err(THIN_ATTN_EINVAL, "page selection needs bounds and exps");
  const int es = esize(a->dtype), cs = esize(a->cache_dtype);
  if (!aligned16(a->q) || !aligned16(a->out) || !aligned16(a->k_pages) || !aligned16(a->v_pages) ||
      !strides16(es, a->q_token, a->q_head) || !strides16(es, a->out_token, a->out_head) ||
      !strides16(cs, a->kp_page, a->kp_head, a->kp_row) || !strides16(cs, a->vp_page, a->vp_head, a->vp_row))
    return err(THIN_ATTN_EINVAL, "tensor pointers and strides must be multiples of 16 bytes");
  if (a->top && !aligned16(a->bounds)) return err(THIN_ATTN_EINVAL, "bounds must be 16-byte aligned");
  const Layout l = layout_of(*a);
  if (l.bytes && (!a->workspace || a->workspace_bytes < l.bytes || (uintptr_t)a->workspace % 256))
    return err(THIN_ATTN_EINVAL, "workspace of %zu bytes, %zu needed, 256-byte aligned", a->workspace_bytes, l.bytes);
  DeviceGuard dg(a->device);
  if (!dg.ok) return err(THIN_ATTN_ECUDA, "cannot select device %d", a->device);
  cudaStream_t st = (cudaStream_t)stream;
  char* ws = (char*)a->workspace;
  PagedAttn p{};
  p.a = *a;
  const float sc = a->scale > 0.f ? a->scale : (float)(1.0 / std::sqrt((double)a->E));
  p.scale_log2e = (float)((double)sc * 1.4426950408889634);
  if (a->page > 1) {
    // s = ceil(log2 page), mul = ceil(2^(31 + s) / page): off by less than page <= 2^s, so exact below 2^31
    int s2 = 0;
    while ((1 << s2) < a->page) ++s2;
    p.page_mul = (uint32_t)((((uint64_t)1 << (31 + s2)) + a->page - 1) / a->page);
    p.page_shift = s2 - 1;
  }
  if (a->top) {
    int32_t* ids = (int32_t*)(ws + l.ids);
    int32_t* keys = (int32_t*)(ws + l.keys);
    s = launched(launch_paged_select(*a, ids, keys, ws + l.words, st), "page selection");
    if (s != THIN_ATTN_OK) return s;
    p.ids = ids;
    p.ids_token = (int64_t)a->H * a->top;
    p.ids_head = a->top;
    p.list_rows = 0;
    p.list_width = a->top;
    p.follows = true;
    p.keys = keys;
  } else {
    p.ids = a->table;
    p.ids_token = a->table_row;
    p.ids_head = 0;
    p.list_rows = a->rows != nullptr;
    p.list_width = a->W;
    p.keys = a->lengths;
  }
  return launched(launch_paged_attention(p, ws + l.attn, st), "paged attention");
}

}  // extern "C"
