// gqaw_paged_host.cu -- the C ABI of the paged operators and the per-head norms
// (include/gqaw.h): argument checks, the choice of kernel, launches.  No allocation and no
// synchronisation.
#include "gqaw_paged_check.cuh"
#include "gqaw_paged_tc.cuh"

namespace gqaw {
cudaError_t launch_paged_rows(const PagedParams &p, int nq, int nk, int nv, bool paged, bool bf16, cudaStream_t stream);
bool encode_tensor_map(CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
                       const cuuint32_t *box, bool bf16);
cudaError_t launch_paged_f32_decode(const PagedParams &p, const PagedMaps &maps, int rows, int sms, cudaStream_t stream);
cudaError_t launch_paged_decode(const PagedParams &p, const PagedMaps &maps, int rows, int grid, cudaStream_t stream);
cudaError_t launch_paged_prefill(const PagedParams &p, const PagedMaps &maps, int halves, int grid, cudaStream_t stream);
cudaError_t launch_paged_rows_attend_f32(const PagedParams &p, int bm, int grid, cudaStream_t stream);
cudaError_t launch_paged_rows_attend_bf16(const PagedParams &p, int bm, int grid, cudaStream_t stream);
cudaError_t launch_paged_warp_attend_f32(const PagedParams &p, int rows, int sms, cudaStream_t stream);
cudaError_t launch_paged_warp_attend_bf16(const PagedParams &p, int rows, int sms, cudaStream_t stream);
}  // namespace gqaw

namespace {

using gqaw::PagedParams;

using namespace gqaw::pcheck;

// ------------------------------------------------------------------------------ norms

struct QkPlan {
  int es, rot_dim;
  long long qs, ks, qos, kos;
};

gqaw_status plan_qk(const gqaw_qk_args *a, QkPlan *L) {
  if (!a) return fail(GQAW_EINVAL, "args is NULL");
  if (a->num_tokens < 0) return fail(GQAW_EINVAL, "num_tokens %d < 0", a->num_tokens);
  if (a->num_heads < 0 || a->kv_num_heads < 0)
    return fail(GQAW_EINVAL, "num_heads %d and kv_num_heads %d must be >= 0", a->num_heads, a->kv_num_heads);
  if (a->dtype != GQAW_F32 && a->dtype != GQAW_BF16) return fail(GQAW_EINVAL, "unknown dtype %d", a->dtype);
  if (a->head_size < 1) return fail(GQAW_EINVAL, "head_size %d < 1", a->head_size);
  if (!head_size_ok(a->head_size))
    return fail(GQAW_EUNSUPPORTED, "head_size %d: supported are 8, 16, 32, 64, 128, 256", a->head_size);
  if (!(a->norm_eps >= 0.f) || !std::isfinite(a->norm_eps)) return fail(GQAW_EINVAL, "norm_eps must be finite and >= 0");
  if (a->reserved != 0) return fail(GQAW_EINVAL, "reserved must be 0");
  if ((long long)a->num_heads + a->kv_num_heads > 65535) return fail(GQAW_EUNSUPPORTED, "more than 65535 heads");
  if ((long long)a->num_tokens * (a->num_heads + a->kv_num_heads) > 0x7fffffffLL)
    return fail(GQAW_EUNSUPPORTED, "more than 2^31 - 1 rows");
  L->es = a->dtype == GQAW_F32 ? 4 : 2;
  gqaw_status s = check_rotary(a->cos_cache, a->sin_cache, a->rotary_dim, a->rotary_cache_len, a->head_size, &L->rot_dim);
  if (s != GQAW_OK) return s;
  const long long qrow = (long long)a->num_heads * a->head_size, krow = (long long)a->kv_num_heads * a->head_size;
  if (a->num_heads && ((s = row_stride("query_stride", a->query_stride, qrow, L->es, a->num_tokens, &L->qs)) != GQAW_OK ||
                       (s = row_stride("query_out_stride", a->query_out_stride, qrow, L->es, a->num_tokens, &L->qos)) != GQAW_OK))
    return s;
  if (a->kv_num_heads && ((s = row_stride("key_stride", a->key_stride, krow, L->es, a->num_tokens, &L->ks)) != GQAW_OK ||
                          (s = row_stride("key_out_stride", a->key_out_stride, krow, L->es, a->num_tokens, &L->kos)) != GQAW_OK))
    return s;
  return GQAW_OK;
}

// An output is its own input at the same stride, or shares no byte with anything.
gqaw_status check_qk_pointers(const gqaw_qk_args *a, const QkPlan &L) {
  gqaw_status s;
  const long long N = a->num_tokens;
  Range in[2], out[2];
  int n = 0;
  bool place[2];
  if (a->num_heads) {
    if ((s = check_tensor("query", a->query)) != GQAW_OK || (s = check_tensor("query_out", a->query_out)) != GQAW_OK) return s;
    in[n] = range_of(a->query, rows_bytes(N, L.qs, (long long)a->num_heads * a->head_size, L.es), "query");
    out[n] = range_of(a->query_out, rows_bytes(N, L.qos, (long long)a->num_heads * a->head_size, L.es), "query_out");
    place[n++] = a->query == a->query_out && L.qs == L.qos;
  }
  if (a->kv_num_heads) {
    if ((s = check_tensor("key", a->key)) != GQAW_OK || (s = check_tensor("key_out", a->key_out)) != GQAW_OK) return s;
    in[n] = range_of(a->key, rows_bytes(N, L.ks, (long long)a->kv_num_heads * a->head_size, L.es), "key");
    out[n] = range_of(a->key_out, rows_bytes(N, L.kos, (long long)a->kv_num_heads * a->head_size, L.es), "key_out");
    place[n++] = a->key == a->key_out && L.ks == L.kos;
  }
  // Query and key as slices of one fused tensor interleave without sharing a byte: their
  // ranges overlap, but each token's rows lie apart within one common stride.
  auto woven = [](const Range &x, long long sx, unsigned long long rx, const Range &y, long long sy, unsigned long long ry,
                  int es) {
    if (sx != sy || x.lo == y.lo) return false;
    const Range &f = x.lo < y.lo ? x : y, &g = x.lo < y.lo ? y : x;
    const unsigned long long rf = x.lo < y.lo ? rx : ry, rg = x.lo < y.lo ? ry : rx;
    const unsigned long long gap = (unsigned long long)(g.lo - f.lo);
    return gap >= rf && gap + rg <= (unsigned long long)sx * es;
  };
  const long long si[2] = {a->num_heads ? L.qs : L.ks, L.ks}, so[2] = {a->num_heads ? L.qos : L.kos, L.kos};
  const unsigned long long row[2] = {
      (unsigned long long)(a->num_heads ? a->num_heads : a->kv_num_heads) * a->head_size * L.es,
      (unsigned long long)a->kv_num_heads * a->head_size * L.es};
  for (int i = 0; i < n; ++i)
    for (int k = 0; k < n; ++k) {
      if (overlap(out[i], in[k]) && !(i == k && place[i]) && !woven(out[i], so[i], row[i], in[k], si[k], row[k], L.es))
        return fail(GQAW_EINVAL, "%s overlaps %s", out[i].name, in[k].name);
      if (i < k && overlap(out[i], out[k]) && !woven(out[i], so[i], row[i], out[k], so[k], row[k], L.es))
        return fail(GQAW_EINVAL, "%s overlaps %s", out[i].name, out[k].name);
    }
  for (const void *w : {a->query_weight, a->key_weight})
    if (w && !aligned(w, 16)) return fail(GQAW_EINVAL, "query_weight / key_weight are not 16-byte aligned");
  if (L.rot_dim) {
    if ((s = check_tables(a->cos_cache, a->sin_cache, a->position_ids, L.es)) != GQAW_OK) return s;
    if (!a->position_ids) return fail(GQAW_EINVAL, "position_ids is NULL");
    if ((s = check_workspace(a->workspace, a->workspace_bytes, 256)) != GQAW_OK) return s;
  }
  return GQAW_OK;
}

// ------------------------------------------------------------------------------ paged

enum Path { kRows = 0, kDecode = 1, kPrefill = 2, kWarp = 3, kF32 = 4 };

struct Plan : PagedSizes {
  int path, bm, rows, halves, hblocks, gb, tpt, grid;
  long long sp, sh, sr;
  size_t off_q, off_qlo, ws_bytes;
  bool split_q;         // turned queries in two parts
  int few;              // kPrefill: sequences of at most this many tokens go to the decode kernel (0: none)
};

gqaw_status plan_paged(const gqaw_paged_args *a, Plan *L) {
  gqaw_status s = check_paged_sizes(a, L);
  if (s != GQAW_OK) return s;
  const long long D = a->head_size, qrow = a->num_heads * D;
  if (!a->page_stride && !a->head_stride && !a->row_stride) {
    L->sr = D;
    L->sh = D * a->page_size;
    L->sp = L->sh * a->kv_num_heads;
  } else {
    L->sp = a->page_stride;
    L->sh = a->head_stride;
    L->sr = a->row_stride;
    for (long long x : {L->sp, L->sh, L->sr}) {
      if (x < D) return fail(GQAW_EINVAL, "page_stride, head_stride and row_stride: all 0, or each at least head_size");
      if (x > kMaxStride) return fail(GQAW_EUNSUPPORTED, "a page stride of %lld is too large", x);
      if (x * L->es % 16 != 0) return fail(GQAW_EINVAL, "a page stride of %lld is not a multiple of 16 bytes", x);
    }
    // no two rows share an element: heads within rows, or rows within heads, inside a page
    const long long h = a->kv_num_heads, r = a->page_size, of_head = reach(r, L->sr, D), of_row = reach(h, L->sh, D);
    const bool rows_inside = L->sh >= of_head && L->sp >= reach(h, L->sh, of_head);
    const bool heads_inside = L->sr >= of_row && L->sp >= reach(r, L->sr, of_row);
    if (!rows_inside && !heads_inside) return fail(GQAW_EINVAL, "the page strides make rows of the cache overlap");
  }
  if (reach(a->num_pages, L->sp, reach(a->kv_num_heads, L->sh, reach(a->page_size, L->sr, D))) == kMaxElements)
    return fail(GQAW_EUNSUPPORTED, "the pages reach over 2^48 elements or more");

  // The kernel.  A query tile is tokens times the query heads of a kv head (a block of them
  // when they are more than the tile has rows).
  const long long rows = (long long)std::max(1, a->max_new_tokens) * L->group;
  // The tensor cores take bf16 with head sizes from 64 on, and pages that tile 128 keys in
  // whole 8-row groups of the swizzled layout.
  auto tiled = [&](int keys) {  // may a tile of `keys` keys come by tensor TMA?
    return a->page_size % 8 == 0 && (keys % a->page_size == 0 || a->page_size % keys == 0) && a->num_pages > 0 &&
           std::max(L->sp, std::max(L->sh, L->sr)) * L->es < (1ll << 40) && std::max(L->qs, qrow) * L->es < (1ll << 40);
  };
  const bool tc = a->dtype == GQAW_BF16 && D >= 64 && tiled(128);
  size_t part_rows;  // rows of partial results per CTA
  if (tc && rows <= 8) {
    L->path = kDecode;
    L->gb = L->group;
    L->hblocks = 1;
    L->tpt = std::max(1, a->max_new_tokens);
    part_rows = 16;
    // no more CTAs than key tiles there can be
    const long long span = a->local_window_size > 0 ? std::min<long long>(a->max_sequence_length, (long long)a->local_window_size + a->max_new_tokens)
                                                     : a->max_sequence_length;
    L->grid = (int)std::max(1ll, std::min<long long>(kSms, (long long)std::min(a->batch_size, gqaw::kPagedItems) *
                                                               a->kv_num_heads * (ceil_div(span, 128) + 1)));
  } else if (tc && L->group <= 128) {
    L->path = kPrefill;
    L->gb = L->group;
    L->hblocks = 1;
    // two query tiles of 128 rows at once when a sequence may fill more than one
    L->halves = rows > 128 && D <= 128 ? 2 : 1;
    L->tpt = L->halves * (128 / L->group);
    part_rows = 128 * L->halves;
    L->grid = kSms;
    // A sequence of a token or two fills at most 8 of the 256 rows, yet its key tiles cost half of
    // a full one's and more.  Where the batch may hold many (the others hold at most
    // max_new_tokens, which bounds their number), they go to the decode kernel, in a launch of
    // its own: 32 contexts of 4096 to 32768 beside a chunk of 512, 491 -> 379 us.  The launch
    // costs 4 to 8 us when there are none, what kShort sequence heads of 2000 keys win; at 20
    // sequences of 128 to 8192 keys and two chunks both ways take 119 us.  Head size 256, one
    // tile of 128 rows, loses (160 -> 195 us).
    constexpr int kShort = 64;
    const long long tok = L->halves == 2 && L->group <= 8 ? 8 / L->group : 0;
    const long long spare = (long long)a->total_new_tokens - a->batch_size * tok;
    if (tok && (a->batch_size - (spare > 0 ? ceil_div(spare, a->max_new_tokens) : 0)) * a->kv_num_heads >= kShort) L->few = (int)tok;
  } else if (rows <= 8 && D * L->es <= 512) {
    L->path = a->dtype == GQAW_F32 && D >= 32 && tiled(16) ? kF32 : kWarp;
    L->gb = L->group;
    L->hblocks = 1;
    L->tpt = std::max(1, a->max_new_tokens);
    part_rows = 16;
    L->grid = kSms * 2;  // at most two CTAs a SM
  } else {
    L->path = kRows;
    L->bm = rows <= 16 ? 16 : D == 256 ? 64 : 128;
    L->grid = L->bm == 16 ? kSms * 4 : kSms;
    L->gb = std::min(L->group, L->bm);
    L->hblocks = (int)ceil_div(L->group, L->gb);
    L->tpt = std::max(1, L->bm / L->gb);
    part_rows = L->bm;
  }
  L->rows = (int)std::min<long long>(rows, 1 << 20);
  L->ws_bytes = gqaw::kPagedPartialOffset + align256((size_t)L->grid * 2 * part_rows * (D + 4) * 4);
  L->off_q = L->ws_bytes;
  L->ws_bytes += align256((size_t)a->total_new_tokens * qrow * L->es);
  // What bf16 leaves of a turned query is kept beside it, and both parts multiply the keys: the
  // rounding of the queries alone otherwise adds 0.0014 to the outputs' error of 0.0016.
  L->split_q = a->dtype == GQAW_BF16;
  L->off_qlo = L->ws_bytes;
  if (L->split_q) L->ws_bytes += align256((size_t)a->total_new_tokens * qrow * L->es);
  return GQAW_OK;
}

// The last byte of the cache that any page id in range can reach, plus one.
unsigned long long pages_bytes(const gqaw_paged_args *a, const Plan &L) {
  if (a->num_pages == 0) return 0;
  return ((unsigned long long)(a->num_pages - 1) * L.sp + (unsigned long long)(a->kv_num_heads - 1) * L.sh +
          (unsigned long long)(a->page_size - 1) * L.sr + a->head_size) * L.es;
}

// Do the rows of two caches of the same strides lie apart, though the bytes between their first and
// last overlap?  With the strides ascending, a block of a level is what its inner dimensions reach
// over, and the blocks lie a stride apart: two caches woven at that level have each other's blocks
// between their own (a page's, a head's or a row's keys beside its values), and the levels outside it
// step over what both reach over together.
bool woven_pages(const gqaw_paged_args *a, const Plan &L) {
  struct {
    long long stride, count;
  } dim[3] = {{L.sr, a->page_size}, {L.sh, a->kv_num_heads}, {L.sp, a->num_pages}};
  std::sort(dim, dim + 3, [](const auto &x, const auto &y) { return x.stride < y.stride; });
  const long long gap = std::llabs(static_cast<const char *>(a->key_pages) - static_cast<const char *>(a->value_pages)) / L.es;
  long long block = a->head_size;
  for (int k = 0; k < 3; ++k) {
    if (dim[k].count < 2) continue;  // such a dimension may have any stride
    if (gap >= block) {
      long long both = gap + block;
      bool apart = true;
      for (int i = k; i < 3; ++i)
        if (dim[i].count > 1) {
          apart = apart && both <= dim[i].stride;
          both += (dim[i].count - 1) * dim[i].stride;
        }
      if (apart) return true;
    }
    block += (dim[k].count - 1) * dim[k].stride;
  }
  return false;
}

gqaw_status check_paged_pointers(const gqaw_paged_args *a, const Plan &L, bool append, bool attend) {
  gqaw_status s;
  const long long N = a->total_new_tokens, D = a->head_size;
  const unsigned long long pb = pages_bytes(a, L);
  Range all[8];
  int n = 0, nw = 0;  // written ranges first
  if ((s = check_workspace(a->workspace, a->workspace_bytes, L.ws_bytes)) != GQAW_OK) return s;
  all[n++] = range_of(a->workspace, L.ws_bytes, "workspace");
  if (attend) {
    if ((s = check_tensor("query", a->query)) != GQAW_OK || (s = check_tensor("output", a->output)) != GQAW_OK) return s;
    all[n++] = range_of(a->output, rows_bytes(N, L.os, a->num_heads * D, L.es), "output");
  }
  if (pb) {
    if ((s = check_tensor("key_pages", a->key_pages)) != GQAW_OK || (s = check_tensor("value_pages", a->value_pages)) != GQAW_OK)
      return s;
  }
  if (append) {
    if ((s = check_tensor("key", a->key)) != GQAW_OK || (s = check_tensor("value", a->value)) != GQAW_OK) return s;
    all[n++] = range_of(a->key_pages, pb, "key_pages");
    all[n++] = range_of(a->value_pages, pb, "value_pages");
  }
  nw = n;
  if (!append) {
    all[n++] = range_of(a->key_pages, pb, "key_pages");
    all[n++] = range_of(a->value_pages, pb, "value_pages");
  } else {
    all[n++] = range_of(a->key, rows_bytes(N, L.ks, a->kv_num_heads * D, L.es), "key");
    all[n++] = range_of(a->value, rows_bytes(N, L.vs, a->kv_num_heads * D, L.es), "value");
  }
  if (attend) all[n++] = range_of(a->query, rows_bytes(N, L.qs, a->num_heads * D, L.es), "query");
  for (int i = 0; i < nw; ++i)
    for (int k = i + 1; k < n; ++k) {
      if (!overlap(all[i], all[k])) continue;
      const bool kv = std::strcmp(all[i].name, "key_pages") == 0 && std::strcmp(all[k].name, "value_pages") == 0;
      if (kv && woven_pages(a, L)) continue;
      return fail(GQAW_EINVAL, "%s overlaps %s", all[i].name, all[k].name);
    }
  if ((s = check_paged_index(a)) != GQAW_OK) return s;
  if (L.rot_dim && append && (s = check_tables(a->cos_cache, a->sin_cache, a->position_ids, L.es)) != GQAW_OK) return s;
  return GQAW_OK;
}

void fill(const gqaw_paged_args *a, const Plan &L, PagedParams *p) {
  fill_paged(a, L, p);
  // without pages no row is read, but copies of no bytes still name a source: a valid address
  p->kp = a->num_pages ? a->key_pages : a->workspace;
  p->vp = a->num_pages ? a->value_pages : a->workspace;
  p->sp = L.sp, p->sh = L.sh, p->sr = L.sr;
  p->hblocks = L.hblocks;
  p->gb = L.gb;
  p->tpt = L.tpt;
}

gqaw_status run_rows(const PagedParams &p, int nq, int nk, int nv, bool paged, bool bf16, cudaStream_t st) {
  const cudaError_t e = gqaw::launch_paged_rows(p, nq, nk, nv, paged, bf16, st);
  if (e != cudaSuccess) return cuda_fail(e, "row kernel launch");
  gqaw::count_launch();
  return GQAW_OK;
}

// Tensor maps: 128-byte rows of the swizzle (64 bf16 or 32 fp32 dimensions), boxes of whole
// pages or of a tile's rows.
// tokens: those of a query box.
gqaw_status make_maps(const gqaw_paged_args *a, const Plan &L, const PagedParams &p, int tokens, gqaw::PagedMaps *m) {
  const bool bf16 = a->dtype == GQAW_BF16;
  const cuuint64_t D = (cuuint64_t)a->head_size, es = (cuuint64_t)L.es;
  const cuuint32_t inner = (cuuint32_t)(128 / L.es);
  const int keys = L.path == kF32 ? 16 : 128;
  const cuuint64_t cd[4] = {D, (cuuint64_t)a->page_size, (cuuint64_t)a->kv_num_heads, (cuuint64_t)a->num_pages};
  const cuuint64_t cst[3] = {(cuuint64_t)L.sr * es, (cuuint64_t)L.sh * es, (cuuint64_t)L.sp * es};
  const cuuint32_t cb[4] = {inner, (cuuint32_t)std::min(a->page_size, keys), 1, 1};
  bool ok = gqaw::encode_tensor_map(&m->k, a->key_pages, 4, cd, cst, cb, bf16) &&
            gqaw::encode_tensor_map(&m->v, a->value_pages, 4, cd, cst, cb, bf16);
  if (L.path == kF32) {
    m->q = m->ql = m->k;  // not used: queries come by ordinary loads
  } else {
    const cuuint64_t qd[3] = {D, (cuuint64_t)a->num_heads, (cuuint64_t)a->total_new_tokens};
    const cuuint64_t qst[2] = {D * es, (cuuint64_t)p.qs * es};
    const cuuint32_t qb[3] = {inner, (cuuint32_t)L.group, (cuuint32_t)tokens};
    ok = ok && gqaw::encode_tensor_map(&m->q, p.q, 3, qd, qst, qb, bf16);
    m->ql = m->q;
    if (p.qlo) ok = ok && gqaw::encode_tensor_map(&m->ql, p.qlo, 3, qd, qst, qb, bf16);
  }
  return ok ? GQAW_OK : fail(GQAW_ECUDA, "cuTensorMapEncodeTiled failed for the paged attention");
}

// The attention, a launch for every kPagedItems sequences.
gqaw_status run_paged_attend(const gqaw_paged_args *a, const Plan &L, PagedParams p, cudaStream_t st) {
  if (gqaw::workspace_tickets_need_clear(a->workspace, gqaw::kPagedTicketOffset, gqaw::kPagedPartialOffset)) {
    const cudaError_t e = cudaMemsetAsync(p.tickets, 0, gqaw::kPagedTickets * 4, st);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync (tickets)");
  }
  gqaw::PagedMaps maps, few_maps;
  gqaw_status s = GQAW_OK;
  if (L.path == kDecode || L.path == kPrefill || L.path == kF32)
    s = make_maps(a, L, p, L.path == kPrefill ? L.tpt / L.halves : L.tpt, &maps);
  if (s == GQAW_OK && L.few) s = make_maps(a, L, p, L.few, &few_maps);
  if (s != GQAW_OK) return s;
  p.s_lo = L.few + 1;
  p.s_hi = a->max_new_tokens;
  for (int b0 = 0; b0 < a->batch_size; b0 += gqaw::kPagedItems) {
    p.B = std::min(gqaw::kPagedItems, a->batch_size - b0);
    p.table = a->page_table + (long long)b0 * a->page_table_width;
    p.qstart = a->query_start + b0;
    p.seqlens = a->seqlens_k + b0;
    const bool f32 = a->dtype == GQAW_F32;
    cudaError_t e;
    switch (L.path) {
      case kDecode: e = gqaw::launch_paged_decode(p, maps, L.rows, L.grid, st); break;
      case kPrefill:
        e = gqaw::launch_paged_prefill(p, maps, L.halves, L.grid, st);
        if (e == cudaSuccess && L.few) {
          gqaw::count_launch();
          PagedParams few = p;
          few.s_lo = 1;
          few.s_hi = few.tpt = L.few;
          e = gqaw::launch_paged_decode(few, few_maps, L.few * L.group, kSms, st);
        }
        break;
      case kF32: e = gqaw::launch_paged_f32_decode(p, maps, L.rows, kSms, st); break;
      case kWarp:
        e = f32 ? gqaw::launch_paged_warp_attend_f32(p, L.rows, kSms, st)
                : gqaw::launch_paged_warp_attend_bf16(p, L.rows, kSms, st);
        break;
      default:
        e = f32 ? gqaw::launch_paged_rows_attend_f32(p, L.bm, L.grid, st)
                : gqaw::launch_paged_rows_attend_bf16(p, L.bm, L.grid, st);
    }
    if (e != cudaSuccess) return cuda_fail(e, "paged attention kernel launch");
    gqaw::count_launch();
  }
  return GQAW_OK;
}

gqaw_status run_paged(const gqaw_paged_args *a, void *stream, bool append, bool attend) {
  Plan L{};
  gqaw_status s = plan_paged(a, &L);
  if (s != GQAW_OK) return s;
  if (a->batch_size == 0 || a->total_new_tokens == 0 || a->max_new_tokens == 0) return GQAW_OK;  // no token, nothing to do
  s = check_paged_pointers(a, L, append, attend);
  if (s != GQAW_OK) return s;
  if ((s = check_device(a->workspace, "workspace")) != GQAW_OK) return s;
  PagedParams p;
  fill(a, L, &p);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (append) {
    const bool turn_q = attend && (L.rot_dim > 0 || a->query_weight);
    p.qout = static_cast<char *>(a->workspace) + L.off_q;
    p.qos = (long long)a->num_heads * a->head_size;
    if (turn_q && L.split_q) p.qlo = static_cast<char *>(a->workspace) + L.off_qlo;
    s = run_rows(p, turn_q ? a->num_heads : 0, a->kv_num_heads, a->kv_num_heads, true, a->dtype == GQAW_BF16, st);
    if (s != GQAW_OK) return s;
    if (turn_q) {
      p.q = p.qout;
      p.qs = p.qos;
    }
  }
  return attend ? run_paged_attend(a, L, p, st) : GQAW_OK;
}

}  // namespace

extern "C" {

gqaw_status gqaw_qk_norm_rotary(const gqaw_qk_args *a, void *stream) {
  QkPlan L{};
  gqaw_status s = plan_qk(a, &L);
  if (s != GQAW_OK) return s;
  if (a->num_tokens == 0 || a->num_heads + a->kv_num_heads == 0) return GQAW_OK;
  s = check_qk_pointers(a, L);
  if (s != GQAW_OK) return s;
  if ((s = check_device(a->num_heads ? a->query : a->key, a->num_heads ? "query" : "key")) != GQAW_OK) return s;
  PagedParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = a->query;
  p.k = a->key;
  p.qout = a->query_out;
  p.kout = a->key_out;
  p.qs = L.qs, p.ks = L.ks, p.qos = L.qos, p.kos = L.kos;
  p.N = a->num_tokens;
  p.D = a->head_size;
  p.qw = a->query_weight;
  p.kw = a->key_weight;
  p.eps = a->norm_eps;
  p.rcos = a->cos_cache;
  p.rsin = a->sin_cache;
  p.pos_ids = reinterpret_cast<const long long *>(a->position_ids);
  p.rot_dim = L.rot_dim;
  p.rot_inter = a->rotary_interleaved ? 1 : 0;
  p.rot_len = a->rotary_cache_len;
  p.status = static_cast<uint32_t *>(a->workspace);
  return run_rows(p, a->num_heads, a->kv_num_heads, 0, false, a->dtype == GQAW_BF16, static_cast<cudaStream_t>(stream));
}

size_t gqaw_paged_workspace_bytes(const gqaw_paged_args *args) {
  Plan L{};
  return plan_paged(args, &L) == GQAW_OK ? L.ws_bytes : 0;
}

gqaw_status gqaw_paged_append(const gqaw_paged_args *args, void *stream) { return run_paged(args, stream, true, false); }

gqaw_status gqaw_paged_attend(const gqaw_paged_args *args, void *stream) { return run_paged(args, stream, false, true); }

gqaw_status gqaw_paged_step(const gqaw_paged_args *args, void *stream) { return run_paged(args, stream, true, true); }

size_t gqaw_qk_args_size(void) { return sizeof(gqaw_qk_args); }

size_t gqaw_paged_args_size(void) { return sizeof(gqaw_paged_args); }

}  // extern "C"
