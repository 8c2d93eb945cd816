// gqaw_paged_check.cuh -- what the host sides of the paged operators share: the checks of sizes, strides,
// pointers and overlaps, and the parameters that every kernel takes from the arguments.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "gqaw_paged.cuh"

namespace gqaw {

void set_error(const char *msg);
void count_launch();
bool workspace_tickets_need_clear(const void *ws, size_t t0, size_t t1);

namespace pcheck {

constexpr int kSms = 152;

inline gqaw_status fail(gqaw_status s, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_error(buf);
  return s;
}
inline gqaw_status cuda_fail(cudaError_t e, const char *what) { return fail(GQAW_ECUDA, "%s: %s", what, cudaGetErrorString(e)); }

inline bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
inline long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
inline bool head_size_ok(int D) { return D == 8 || D == 16 || D == 32 || D == 64 || D == 128 || D == 256; }

// A tensor that a call reads or writes, as the bytes from its first to its last element.
struct Range {
  const char *lo, *hi;
  const char *name;
};
inline Range range_of(const void *p, unsigned long long bytes, const char *name) {
  return Range{static_cast<const char *>(p), static_cast<const char *>(p) + bytes, name};
}
inline bool overlap(const Range &x, const Range &y) { return x.lo < y.hi && y.lo < x.hi; }

// Bytes of n rows of `row` elements that lie `stride` elements apart.
inline unsigned long long rows_bytes(long long n, long long stride, long long row, int es) {
  return n <= 0 ? 0ull : ((unsigned long long)(n - 1) * (unsigned long long)stride + (unsigned long long)row) * (unsigned)es;
}

// What a tensor's strides reach over, and its bytes, stay far inside 64 bits (and inside what an
// address can hold).
constexpr long long kMaxStride = 1ll << 40, kMaxElements = 1ll << 48;

// n blocks of `block` elements that lie `stride` elements apart; kMaxElements if that or more.
inline long long reach(long long n, long long stride, long long block) {
  const __int128 x = n <= 0 ? 0 : (__int128)(n - 1) * stride + block;
  return x < kMaxElements ? (long long)x : kMaxElements;
}

inline gqaw_status row_stride(const char *name, int64_t given, long long row, int es, long long n, long long *out) {
  *out = given ? given : row;
  if (given < 0 || (given && given < row)) return fail(GQAW_EINVAL, "%s %lld: 0 or at least %lld", name, (long long)given, row);
  if (given > kMaxStride) return fail(GQAW_EUNSUPPORTED, "%s %lld is too large", name, (long long)given);
  if (*out * es % 16 != 0) return fail(GQAW_EINVAL, "%s %lld is not a multiple of 16 bytes", name, *out);
  if (reach(n, *out, row) == kMaxElements) return fail(GQAW_EUNSUPPORTED, "%s %lld is too large for %lld tokens", name, *out, n);
  return GQAW_OK;
}

inline gqaw_status check_tensor(const char *name, const void *p, size_t al = 16) {
  if (!p) return fail(GQAW_EINVAL, "%s is NULL", name);
  if (!aligned(p, al)) return fail(GQAW_EINVAL, "%s is not %zu-byte aligned", name, al);
  return GQAW_OK;
}

inline gqaw_status check_rotary(const void *cos, const void *sin, int dim, int len, int head_size, int *rot_dim) {
  *rot_dim = 0;
  if (!cos && !sin) return GQAW_OK;
  if (!cos || !sin) return fail(GQAW_EINVAL, "cos_cache and sin_cache go together");
  const int rd = dim ? dim : head_size;
  if (rd < 2 || rd % 2 != 0 || rd > head_size)
    return fail(GQAW_EINVAL, "rotary_dim %d must be even and in [2, head_size=%d]", dim, head_size);
  if (len < 1) return fail(GQAW_EINVAL, "rotary_cache_len %d < 1", len);
  *rot_dim = rd;
  return GQAW_OK;
}

inline gqaw_status check_tables(const void *cos, const void *sin, const void *ids, int es) {
  if (!aligned(cos, es) || !aligned(sin, es)) return fail(GQAW_EINVAL, "cos_cache / sin_cache are not %d-byte aligned", es);
  if (ids && !aligned(ids, 8)) return fail(GQAW_EINVAL, "position_ids is not 8-byte aligned");
  return GQAW_OK;
}

inline gqaw_status check_workspace(const void *ws, size_t have, size_t need) {
  if (!ws) return fail(GQAW_EWORKSPACE, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(GQAW_EWORKSPACE, "workspace is not 256-byte aligned");
  if (have < need) return fail(GQAW_EWORKSPACE, "workspace_bytes %zu < required %zu", have, need);
  return GQAW_OK;
}

// The call is about to launch on the current device, where a tensor of the host or of another GPU
// may fault.  One pointer a call is looked at, the workspace or the norms' rows, and refused if it is
// such: it tells a caller's current device from its tensors'.  The binding holds all tensors of a
// call to one device; another caller's are its own, since a look at each takes 73 ns, a
// microsecond for all beside the 3 of the call.
inline gqaw_status check_device(const void *p, const char *name) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  cudaPointerAttributes at;
  e = cudaPointerGetAttributes(&at, p);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return cuda_fail(e, name);
  }
  if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged)
    return fail(GQAW_EINVAL, "%s is not device memory", name);
  if (at.type == cudaMemoryTypeDevice && at.device != dev)
    return fail(GQAW_EINVAL, "%s is on device %d, the current device is %d", name, at.device, dev);
  return GQAW_OK;
}

// Sizes and strides of a call that no kernel's choice changes.
struct PagedSizes {
  int es, rot_dim, group;
  long long qs, ks, vs, os;
};

inline gqaw_status check_paged_sizes(const gqaw_paged_args *a, PagedSizes *L) {
  if (!a) return fail(GQAW_EINVAL, "args is NULL");
  if (a->batch_size < 0) return fail(GQAW_EINVAL, "batch_size %d < 0", a->batch_size);
  if (a->total_new_tokens < 0) return fail(GQAW_EINVAL, "total_new_tokens %d < 0", a->total_new_tokens);
  if (a->max_new_tokens < 0 || a->max_new_tokens > a->total_new_tokens)
    return fail(GQAW_EINVAL, "max_new_tokens %d must be in [0, total_new_tokens=%d]", a->max_new_tokens, a->total_new_tokens);
  if (a->num_heads < 1 || a->kv_num_heads < 1)
    return fail(GQAW_EINVAL, "num_heads %d and kv_num_heads %d must be >= 1", a->num_heads, a->kv_num_heads);
  if (a->num_heads % a->kv_num_heads != 0)
    return fail(GQAW_EINVAL, "num_heads %d is not a multiple of kv_num_heads %d", a->num_heads, a->kv_num_heads);
  if (a->dtype != GQAW_F32 && a->dtype != GQAW_BF16) return fail(GQAW_EINVAL, "unknown dtype %d", a->dtype);
  if (a->head_size < 1) return fail(GQAW_EINVAL, "head_size %d < 1", a->head_size);
  if (!head_size_ok(a->head_size))
    return fail(GQAW_EUNSUPPORTED, "head_size %d: supported are 8, 16, 32, 64, 128, 256", a->head_size);
  if (a->num_heads > 32767) return fail(GQAW_EUNSUPPORTED, "num_heads %d > 32767", a->num_heads);
  if (a->page_size < 1) return fail(GQAW_EINVAL, "page_size %d < 1", a->page_size);
  if (a->num_pages < 0) return fail(GQAW_EINVAL, "num_pages %d < 0", a->num_pages);
  if (a->page_table_width < 0) return fail(GQAW_EINVAL, "page_table_width %d < 0", a->page_table_width);
  if (a->max_sequence_length < a->max_new_tokens)
    return fail(GQAW_EINVAL, "max_sequence_length %d < max_new_tokens %d", a->max_sequence_length, a->max_new_tokens);
  if (a->max_sequence_length > (long long)a->page_table_width * a->page_size)
    return fail(GQAW_EINVAL, "max_sequence_length %d > page_table_width %d x page_size %d", a->max_sequence_length,
                a->page_table_width, a->page_size);
  if (a->local_window_size < 0) return fail(GQAW_EINVAL, "local_window_size %d < 0", a->local_window_size);
  if (!(a->scale >= 0.f) || !std::isfinite(a->scale)) return fail(GQAW_EINVAL, "scale must be finite and >= 0");
  if (!(a->softcap >= 0.f) || !std::isfinite(a->softcap)) return fail(GQAW_EINVAL, "softcap must be finite and >= 0");
  if (!(a->norm_eps >= 0.f) || !std::isfinite(a->norm_eps)) return fail(GQAW_EINVAL, "norm_eps must be finite and >= 0");
  if (a->reserved != 0) return fail(GQAW_EINVAL, "reserved must be 0");
  if ((long long)a->total_new_tokens * (a->num_heads + 2LL * a->kv_num_heads) > 0x7fffffffLL)
    return fail(GQAW_EUNSUPPORTED, "more than 2^31 - 1 rows");
  L->es = a->dtype == GQAW_F32 ? 4 : 2;
  gqaw_status s = check_rotary(a->cos_cache, a->sin_cache, a->rotary_dim, a->rotary_cache_len, a->head_size, &L->rot_dim);
  if (s != GQAW_OK) return s;
  const long long D = a->head_size, qrow = a->num_heads * D, krow = a->kv_num_heads * D;
  if ((s = row_stride("query_stride", a->query_stride, qrow, L->es, a->total_new_tokens, &L->qs)) != GQAW_OK ||
      (s = row_stride("key_stride", a->key_stride, krow, L->es, a->total_new_tokens, &L->ks)) != GQAW_OK ||
      (s = row_stride("value_stride", a->value_stride, krow, L->es, a->total_new_tokens, &L->vs)) != GQAW_OK ||
      (s = row_stride("output_stride", a->output_stride, qrow, L->es, a->total_new_tokens, &L->os)) != GQAW_OK)
    return s;
  L->group = a->num_heads / a->kv_num_heads;
  return GQAW_OK;
}

inline gqaw_status check_paged_index(const gqaw_paged_args *a) {
  const struct {
    const void *p;
    const char *name;
    size_t al;
    bool need;
  } idx[] = {{a->query_start, "query_start", 4, true},
             {a->seqlens_k, "seqlens_k", 4, true},
             {a->page_table, "page_table", 4, a->page_table_width > 0},
             {a->head_sink, "head_sink", 4, false}};
  for (auto &x : idx) {
    if (!x.p && x.need) return fail(GQAW_EINVAL, "%s is NULL", x.name);
    if (x.p && !aligned(x.p, x.al)) return fail(GQAW_EINVAL, "%s is not %zu-byte aligned", x.name, x.al);
  }
  for (const void *w : {a->query_weight, a->key_weight})
    if (w && !aligned(w, 16)) return fail(GQAW_EINVAL, "query_weight / key_weight are not 16-byte aligned");
  return GQAW_OK;
}

// All but the cache, the kernel's tiling and what a launch changes.
inline void fill_paged(const gqaw_paged_args *a, const PagedSizes &L, PagedParams *p) {
  std::memset(p, 0, sizeof(*p));
  char *ws = static_cast<char *>(a->workspace);
  p->q = a->query;
  p->k = a->key;
  p->v = a->value;
  p->out = a->output;
  p->qs = L.qs, p->ks = L.ks, p->vs = L.vs, p->os = L.os;
  p->table = a->page_table;
  p->qstart = a->query_start;
  p->seqlens = a->seqlens_k;
  p->sink = a->head_sink;
  p->sink_mode = a->head_sink ? 1 : (a->smooth_softmax ? 2 : 0);
  p->B = a->batch_size;
  p->N = a->total_new_tokens;
  p->max_new = a->max_new_tokens;
  p->max_len = a->max_sequence_length;
  p->Nq = a->num_heads;
  p->Nkv = a->kv_num_heads;
  p->D = a->head_size;
  p->page = a->page_size;
  p->npages = a->num_pages;
  p->width = a->page_table_width;
  p->W = a->local_window_size >= a->max_sequence_length ? 0 : a->local_window_size;  // a window of everything is none
  p->group = L.group;
  const float scale = a->scale > 0.f ? a->scale : 1.0f / std::sqrt((float)a->head_size);
  p->qscale = a->softcap > 0.f ? scale / a->softcap : scale * kLog2e;
  p->capmul = a->softcap > 0.f ? a->softcap * kLog2e : 0.f;
  p->status = reinterpret_cast<uint32_t *>(ws);
  p->tickets = reinterpret_cast<uint32_t *>(ws + kPagedTicketOffset);
  p->partials = reinterpret_cast<float *>(ws + kPagedPartialOffset);
  p->qw = a->query_weight;
  p->kw = a->key_weight;
  p->rcos = a->cos_cache;
  p->rsin = a->sin_cache;
  p->pos_ids = reinterpret_cast<const long long *>(a->position_ids);
  p->rot_dim = L.rot_dim;
  p->rot_inter = a->rotary_interleaved ? 1 : 0;
  p->rot_len = a->rotary_cache_len;
  p->eps = a->norm_eps;
}

}  // namespace pcheck
}  // namespace gqaw
