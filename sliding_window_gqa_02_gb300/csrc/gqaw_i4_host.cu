// gqaw_i4_host.cu -- the C ABI of the operators on paged caches held in 4 bits (include/gqaw.h):
// argument checks, the choice of kernel, launches.  No allocation and no synchronisation.
#include "gqaw_i4.cuh"
#include "gqaw_paged_check.cuh"
#include "gqaw_paged_tc.cuh"

namespace gqaw {
cudaError_t launch_i4_rows(const I4Params &p, int nq, int nk, int nv, bool read, bool bf16, cudaStream_t stream);
cudaError_t launch_i4_prefill(const I4Params &p, const PagedMaps &maps, int grid, cudaStream_t stream);
cudaError_t launch_i4_expand(const I4Params &p, void *k, void *v, int32_t *table, int width, int pages, int sms, cudaStream_t stream);
cudaError_t launch_paged_prefill(const PagedParams &p, const PagedMaps &maps, int halves, int grid, cudaStream_t stream);
bool encode_tensor_map(CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
                       const cuuint32_t *box, bool bf16);
cudaError_t launch_i4_attend_bf16(const I4Params &p, int nt, int sms, cudaStream_t stream);
cudaError_t launch_i4_attend_split(const I4Params &p, int nt, int sms, cudaStream_t stream);
cudaError_t launch_i4_attend_f32(const I4Params &p, int nt, int sms, cudaStream_t stream);
}  // namespace gqaw

namespace {

using gqaw::I4Params;
using namespace gqaw::pcheck;

// The attention's kernels: up to 8 nt query rows of a kv head at once; the bf16 prompt kernel with tiles written
// from codes; the same over bf16 pages that a pass before it expands.
enum I4Path { kRows = 0, kTiles = 1, kExpand = 2 };

struct I4Plan : PagedSizes {
  long long sp, sh, sr;          // codes, bytes
  long long tp, th, tr;          // scales, elements
  long long kos, vos;
  int path;
  int halves;                    // kExpand, kTiles: query tiles of 128 rows at once
  int pages, width;              // kExpand: pages of 128 rows in the workspace, and entries of a row of their table
  int nt;                        // operands of 8 query rows
  int few;                       // sequences of at most this many tokens go to the kernel of 8 rows (0: none)
  int gb, hblocks, tpt;
  size_t off_q, off_qlo, off_k, off_v, off_table, ws_bytes;
};

// Strides of one part of the cache: rows of `row` units.  `unit`: what a stride is a multiple of.
gqaw_status page_strides(const char *what, int64_t page, int64_t head, int64_t rows, long long row, long long unit,
                         const gqaw_paged_args *a, long long *sp, long long *sh, long long *sr) {
  if (!page && !head && !rows) {
    *sr = row;
    *sh = row * a->page_size;
    *sp = *sh * a->kv_num_heads;
  } else {
    *sp = page;
    *sh = head;
    *sr = rows;
    for (long long x : {*sp, *sh, *sr}) {
      if (x < row) return fail(GQAW_EINVAL, "the page, head and row strides of the %s: all 0, or each at least %lld", what, row);
      if (x / unit >= 1ll << 32) return fail(GQAW_EUNSUPPORTED, "a stride of the %s of %lld is too large", what, x);
      if (x % unit != 0) return fail(GQAW_EINVAL, "a stride of the %s of %lld is not a multiple of %lld", what, x, unit);
    }
    // no two rows share a byte: heads within rows, or rows within heads, inside a page
    const long long h = a->kv_num_heads, r = a->page_size, of_head = reach(r, *sr, row), of_row = reach(h, *sh, row);
    const bool rows_inside = *sh >= of_head && *sp >= reach(h, *sh, of_head);
    const bool heads_inside = *sr >= of_row && *sp >= reach(r, *sr, of_row);
    if (!rows_inside && !heads_inside) return fail(GQAW_EINVAL, "the strides make rows of the %s overlap", what);
  }
  if (*sp / unit >= 1ll << 32) return fail(GQAW_EUNSUPPORTED, "a page of the %s of %lld is too large", what, *sp);
  if (reach(a->num_pages, *sp, reach(a->kv_num_heads, *sh, reach(a->page_size, *sr, row))) == kMaxElements)
    return fail(GQAW_EUNSUPPORTED, "the %s reach over 2^48 elements or more", what);
  return GQAW_OK;
}

gqaw_status plan_i4(const gqaw_paged_i4_args *x, I4Plan *L) {
  if (!x) return fail(GQAW_EINVAL, "args is NULL");
  const gqaw_paged_args *a = &x->paged;
  gqaw_status s = check_paged_sizes(a, L);
  if (s != GQAW_OK) return s;
  const long long D = a->head_size, krow = a->kv_num_heads * D;
  if (D < gqaw::kI4Group) return fail(GQAW_EUNSUPPORTED, "head_size %d: a 4-bit cache takes 32, 64, 128, 256", a->head_size);
  if ((s = page_strides("codes", a->page_stride, a->head_stride, a->row_stride, D / 2, 16, a, &L->sp, &L->sh, &L->sr)) != GQAW_OK ||
      (s = page_strides("scales", x->scale_page_stride, x->scale_head_stride, x->scale_row_stride, D / gqaw::kI4Group,
                        D / gqaw::kI4Group, a, &L->tp, &L->th, &L->tr)) != GQAW_OK ||
      (s = row_stride("key_out_stride", x->key_out_stride, krow, L->es, a->total_new_tokens, &L->kos)) != GQAW_OK ||
      (s = row_stride("value_out_stride", x->value_out_stride, krow, L->es, a->total_new_tokens, &L->vos)) != GQAW_OK)
    return s;
  // The kernel: 8 query rows of a kv head a product, more by query tiles that read the keys again (from L2): 16
  // rows at once, whose registers leave 8 warps a SM, take as long (16 x 8 tokens at 6000 keys, window 4096,
  // 109 us both ways) or longer (head size 64 56 -> 67, 256 91 -> 136), and 32 longer still (156).  In fp32, where
  // every product is two, 16 are faster (a prompt of 1024 259 -> 214 us, 8 x 8 tokens 72 -> 60).
  const long long rows = (long long)std::max(1, a->max_new_tokens) * L->group;
  L->nt = rows > 8 && a->dtype == GQAW_F32 && D <= 128 ? 2 : 1;
  L->path = kRows;
  // Many rows in bf16: the 5th-generation tensor cores, whose tiles of keys cost as much for 1 row as for 128.  16
  // chunks at 6000 keys (window 4096, 8 heads) cross at 36 rows with head size 64, 50 with 128, 62 with 256.
  // With little work in all (rows times keys) their fixed part decides, a CTA that joins a unit's many cuts: one
  // chunk at 6000 keys and head size 128, 128 rows 67 us and 44 by rows, 256 72 and 76; at 1000 keys 256 rows
  // 40 and 38 (head size 256 43 and 62, 128 rows 43 and 27); 4 chunks of 48 rows at 6000 70 and 64, of 128 66
  // and 134; one of 128 at 32000 105 and 154.
  const long long span = a->local_window_size > 0 ? std::min<long long>(a->max_sequence_length, (long long)a->local_window_size + a->max_new_tokens)
                                                   : a->max_sequence_length;
  constexpr double kLittle = 1e7;
  const bool little = rows <= (D == 256 ? 128 : 256) && (double)a->total_new_tokens * a->num_heads * span <= kLittle;
  const bool many = a->dtype == GQAW_BF16 && D >= 64 && L->group <= 128 && rows > (D == 256 ? 64 : 40) && !little &&
                    std::max<long long>(L->qs, a->num_heads * D) * L->es < (1ll << 40);
  // Single tokens among chunks would fill 8 of the rows: they have a launch of their own where there
  // may be many (the others hold at most max_new_tokens, which bounds their number)
  constexpr int kShort = 64;
  const int seqs = std::min(gqaw::kPagedItems, a->batch_size);
  const long long tok = (L->nt > 1 || many) && L->group <= 8 ? 8 / L->group : 0;
  const long long spare = (long long)a->total_new_tokens - a->batch_size * tok;
  if (tok && (a->batch_size - (spare > 0 ? ceil_div(spare, a->max_new_tokens) : 0)) * a->kv_num_heads >= kShort) L->few = (int)tok;
  if (many) {
    // Expanded where a sequence may have more than one query tile and the workspace does not grow beyond kMost:
    // for every sequence what its tokens attend (row ranges that repeat rows may make chunks of all)
    constexpr unsigned long long kMost = 2ull << 30;
    L->halves = D <= 128 ? 2 : 1;
    L->tpt = L->halves * (128 / L->group);
    const long long pages = seqs * (ceil_div(span, 128) + 1);
    const unsigned long long bytes = (unsigned long long)pages * 128 * a->kv_num_heads * D * 4;
    if (D == 256 ? bytes <= kMost : a->max_new_tokens > L->tpt && bytes <= kMost)
      L->path = kExpand;
    else if (D <= 128)
      L->path = kTiles;
    L->pages = (int)pages;
    L->width = (int)ceil_div(a->max_sequence_length, 128);
  }
  const int tile = L->path != kRows ? 128 * L->halves : 8 * L->nt;
  L->gb = L->path != kRows ? L->group : std::min(L->group, tile);
  L->hblocks = (int)ceil_div(L->group, L->gb);
  if (L->path == kRows) L->tpt = std::max(1, tile / L->gb);
  L->ws_bytes = gqaw::kPagedPartialOffset + align256((size_t)kSms * 2 * tile * (D + 4) * 4);
  L->off_q = L->ws_bytes;
  L->ws_bytes += align256((size_t)a->total_new_tokens * a->num_heads * D * L->es);
  L->off_qlo = L->ws_bytes;  // what bf16 leaves of turned queries
  if (a->dtype == GQAW_BF16) L->ws_bytes += align256((size_t)a->total_new_tokens * a->num_heads * D * L->es);
  if (L->path == kExpand) {
    const size_t half = align256((size_t)L->pages * 128 * a->kv_num_heads * D * 2);
    L->off_k = L->ws_bytes;
    L->off_v = L->off_k + half;
    L->off_table = L->off_v + half;
    L->ws_bytes = L->off_table + align256((size_t)seqs * L->width * 4);
  }
  return GQAW_OK;
}

// A part of the cache as bytes: three strides, each with a count, and the row inside.
struct Part {
  Range all;
  struct {
    long long stride, count;
  } dim[3];  // the largest stride first
  long long row;
  int n;     // dimensions of more than one element
};

Part part_of(const void *p, const char *name, const gqaw_paged_args *a, long long sp, long long sh, long long sr, long long row, int unit) {
  Part x;
  x.row = row * unit;
  x.n = 0;
  const struct {
    long long stride, count;
  } dims[3] = {{sp, a->num_pages}, {sh, a->kv_num_heads}, {sr, a->page_size}};
  unsigned long long bytes = (unsigned long long)x.row;
  for (const auto &d : dims) {
    bytes += (unsigned long long)(d.count > 0 ? d.count - 1 : 0) * d.stride * unit;
    if (d.count > 1) x.dim[x.n++] = {d.stride * unit, d.count};
  }
  std::sort(x.dim, x.dim + x.n, [](const auto &u, const auto &v) { return u.stride > v.stride; });
  x.all = range_of(p, a->num_pages ? bytes : 0, name);
  return x;
}

// Do two parts of the cache lie apart, though the bytes between their first and last overlap?  At a level down to
// which their strides agree, what the inner dimensions of one reach over lies between two of the other's; and of the levels
// outside it, each steps over what both reach over together.
bool woven_parts(const Part &x, const Part &y) {
  const Part &f = x.all.lo < y.all.lo ? x : y, &g = x.all.lo < y.all.lo ? y : x;
  const long long gap = g.all.lo - f.all.lo;
  auto inner = [](const Part &p, int from) {
    long long b = p.row;
    for (int i = from; i < p.n; ++i) b += (p.dim[i].count - 1) * p.dim[i].stride;
    return b;
  };
  for (int k = 0; k < f.n && k < g.n && f.dim[k].stride == g.dim[k].stride && f.dim[k].count == g.dim[k].count; ++k) {
    long long both = gap + inner(g, k + 1);
    bool apart = gap >= inner(f, k + 1) && both <= f.dim[k].stride;
    for (int i = k; i > 0; --i) apart = apart && (both += (f.dim[i].count - 1) * f.dim[i].stride) <= f.dim[i - 1].stride;
    if (apart) return true;
  }
  return false;
}

enum What { kAppend = 1, kAttend = 2, kRead = 4 };

gqaw_status check_i4_pointers(const gqaw_paged_i4_args *x, const I4Plan &L, int what) {
  const gqaw_paged_args *a = &x->paged;
  gqaw_status s;
  const long long N = a->total_new_tokens, D = a->head_size;
  const bool append = what & kAppend, attend = what & kAttend, read = what & kRead;
  const size_t need = attend ? L.ws_bytes : 256;  // an append and a read only flag
  if ((s = check_workspace(a->workspace, a->workspace_bytes, need)) != GQAW_OK) return s;
  const size_t scale_row = (size_t)D / gqaw::kI4Group * 2;
  if (a->num_pages) {
    if ((s = check_tensor("key_pages", a->key_pages)) != GQAW_OK || (s = check_tensor("value_pages", a->value_pages)) != GQAW_OK ||
        (s = check_tensor("key_scales", x->key_scales, scale_row)) != GQAW_OK ||
        (s = check_tensor("value_scales", x->value_scales, scale_row)) != GQAW_OK)
      return s;
  }
  const Part part[4] = {part_of(a->key_pages, "key_pages", a, L.sp, L.sh, L.sr, D / 2, 1),
                        part_of(a->value_pages, "value_pages", a, L.sp, L.sh, L.sr, D / 2, 1),
                        part_of(x->key_scales, "key_scales", a, L.tp, L.th, L.tr, D / gqaw::kI4Group, 2),
                        part_of(x->value_scales, "value_scales", a, L.tp, L.th, L.tr, D / gqaw::kI4Group, 2)};
  if (append)
    for (int i = 0; i < 4; ++i)
      for (int k = i + 1; k < 4; ++k)
        if (overlap(part[i].all, part[k].all) && !woven_parts(part[i], part[k]))
          return fail(GQAW_EINVAL, "%s overlaps %s", part[i].all.name, part[k].all.name);
  struct {
    Range r;
    bool written, cache;
  } t[10];
  int n = 0;
  auto add = [&](const Range &r, bool written, bool cache = false) { t[n++] = {r, written, cache}; };
  add(range_of(a->workspace, need, "workspace"), true);
  for (const Part &p : part) add(p.all, append, true);
  if (attend) {
    if ((s = check_tensor("query", a->query)) != GQAW_OK || (s = check_tensor("output", a->output)) != GQAW_OK) return s;
    add(range_of(a->output, rows_bytes(N, L.os, a->num_heads * D, L.es), "output"), true);
    add(range_of(a->query, rows_bytes(N, L.qs, a->num_heads * D, L.es), "query"), false);
  }
  if (append) {
    if ((s = check_tensor("key", a->key)) != GQAW_OK || (s = check_tensor("value", a->value)) != GQAW_OK) return s;
    add(range_of(a->key, rows_bytes(N, L.ks, a->kv_num_heads * D, L.es), "key"), false);
    add(range_of(a->value, rows_bytes(N, L.vs, a->kv_num_heads * D, L.es), "value"), false);
  }
  const int outs = n;
  if (read) {
    if (!x->key_out && !x->value_out) return fail(GQAW_EINVAL, "key_out and value_out are NULL");
    for (const void *p : {x->key_out, x->value_out})
      if (p && !aligned(p, 16)) return fail(GQAW_EINVAL, "key_out / value_out are not 16-byte aligned");
    if (x->key_out) add(range_of(x->key_out, rows_bytes(N, L.kos, a->kv_num_heads * D, L.es), "key_out"), true);
    if (x->value_out) add(range_of(x->value_out, rows_bytes(N, L.vos, a->kv_num_heads * D, L.es), "value_out"), true);
  }
  for (int i = 0; i < n; ++i)
    for (int k = i + 1; k < n; ++k) {
      if (!(t[i].written || t[k].written) || (t[i].cache && t[k].cache) || !overlap(t[i].r, t[k].r)) continue;
      if (i >= outs && L.kos == L.vos) {  // both read into one tensor, a token's keys beside its values
        const long long gap = std::llabs(t[i].r.lo - t[k].r.lo), row = a->kv_num_heads * D * L.es;
        if (gap >= row && gap + row <= L.kos * L.es) continue;
      }
      return fail(GQAW_EINVAL, "%s overlaps %s", t[i].r.name, t[k].r.name);
    }
  if ((s = check_paged_index(a)) != GQAW_OK) return s;
  if (L.rot_dim && append && (s = check_tables(a->cos_cache, a->sin_cache, a->position_ids, L.es)) != GQAW_OK) return s;
  return GQAW_OK;
}

// The attention, a launch (or two) for every kPagedItems sequences.
gqaw_status run_attend(const gqaw_paged_args *a, const I4Plan &L, I4Params p, cudaStream_t st) {
  if (gqaw::workspace_tickets_need_clear(a->workspace, gqaw::kPagedTicketOffset, gqaw::kPagedPartialOffset)) {
    const cudaError_t e = cudaMemsetAsync(p.tickets, 0, gqaw::kPagedTickets * 4, st);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync (tickets)");
  }
  const long long D = a->head_size;
  p.sp16 = (uint32_t)(L.sp / 16);
  p.sr16 = (uint32_t)(L.sr / 16);
  p.tpg = (uint32_t)(L.tp / (D / gqaw::kI4Group));
  p.trg = (uint32_t)(L.tr / (D / gqaw::kI4Group));
  p.blocks = gqaw::i4_blocks(a->page_size, D, L.sr, L.tr);
  p.to_values = static_cast<const char *>(p.vp) - static_cast<const char *>(p.kp);
  p.to_value_scales = reinterpret_cast<const char *>(p.vscale) - reinterpret_cast<const char *>(p.kscale);
  gqaw::PagedMaps maps;
  gqaw::PagedParams wide;  // kExpand: the attention over the expanded pages
  if (L.path != kRows) {
    std::memset(&maps, 0, sizeof(maps));
    const cuuint64_t qd[3] = {(cuuint64_t)D, (cuuint64_t)a->num_heads, (cuuint64_t)a->total_new_tokens};
    const cuuint64_t qst[2] = {(cuuint64_t)D * 2, (cuuint64_t)p.qs * 2};
    const cuuint32_t qb[3] = {64, (cuuint32_t)L.group, (cuuint32_t)(L.tpt / L.halves)};
    bool ok = gqaw::encode_tensor_map(&maps.q, p.q, 3, qd, qst, qb, true);
    maps.ql = maps.q;
    if (p.qlo) ok = ok && gqaw::encode_tensor_map(&maps.ql, p.qlo, 3, qd, qst, qb, true);
    if (L.path == kExpand) {
      char *ws = static_cast<char *>(a->workspace);
      wide = p;
      wide.kp = ws + L.off_k;
      wide.vp = ws + L.off_v;
      wide.sr = D;
      wide.sh = 128 * D;
      wide.sp = wide.sh * a->kv_num_heads;
      wide.table = reinterpret_cast<const int32_t *>(ws + L.off_table);
      wide.page = 128;
      wide.npages = L.pages;
      wide.width = L.width;
      const cuuint64_t cd[4] = {(cuuint64_t)D, 128, (cuuint64_t)a->kv_num_heads, (cuuint64_t)L.pages};
      const cuuint64_t cst[3] = {(cuuint64_t)wide.sr * 2, (cuuint64_t)wide.sh * 2, (cuuint64_t)wide.sp * 2};
      const cuuint32_t cb[4] = {64, 128, 1, 1};
      ok = ok && gqaw::encode_tensor_map(&maps.k, wide.kp, 4, cd, cst, cb, true) &&
           gqaw::encode_tensor_map(&maps.v, wide.vp, 4, cd, cst, cb, true);
    }
    if (!ok) return fail(GQAW_ECUDA, "cuTensorMapEncodeTiled failed for the attention over a 4-bit cache");
  }
  auto launch = [&](const I4Params &x, int nt) {
    const cudaError_t e = a->dtype == GQAW_F32 ? gqaw::launch_i4_attend_f32(x, nt, kSms, st)
                          : x.qlo              ? gqaw::launch_i4_attend_split(x, nt, kSms, st)
                                               : gqaw::launch_i4_attend_bf16(x, nt, kSms, st);
    if (e == cudaSuccess) gqaw::count_launch();
    return e;
  };
  for (int b0 = 0; b0 < a->batch_size; b0 += gqaw::kPagedItems) {
    p.B = std::min(gqaw::kPagedItems, a->batch_size - b0);
    p.table = a->page_table + (long long)b0 * a->page_table_width;
    p.qstart = a->query_start + b0;
    p.seqlens = a->seqlens_k + b0;
    p.s_lo = L.few + 1;
    p.s_hi = a->max_new_tokens;
    p.gb = L.gb;
    p.hblocks = L.hblocks;
    p.tpt = L.tpt;
    cudaError_t e;
    switch (L.path) {
      case kExpand:
        e = gqaw::launch_i4_expand(p, wide.kp, wide.vp, const_cast<int32_t *>(wide.table), L.width, L.pages, kSms, st);
        if (e != cudaSuccess) break;
        gqaw::count_launch();
        wide.B = p.B;
        wide.qstart = p.qstart;
        wide.seqlens = p.seqlens;
        wide.s_lo = p.s_lo;
        wide.s_hi = p.s_hi;
        wide.gb = p.gb;
        wide.hblocks = p.hblocks;
        wide.tpt = p.tpt;
        e = gqaw::launch_paged_prefill(wide, maps, L.halves, kSms, st);
        if (e == cudaSuccess) gqaw::count_launch();
        break;
      case kTiles:
        e = gqaw::launch_i4_prefill(p, maps, kSms, st);
        if (e == cudaSuccess) gqaw::count_launch();
        break;
      default: e = launch(p, L.nt);
    }
    if (e == cudaSuccess && L.few) {
      I4Params few = p;
      few.s_lo = 1;
      few.s_hi = few.tpt = L.few;
      few.gb = L.group;
      few.hblocks = 1;
      e = launch(few, 1);
    }
    if (e != cudaSuccess) return cuda_fail(e, "attention kernel launch");
  }
  return GQAW_OK;
}

gqaw_status run_i4(const gqaw_paged_i4_args *x, void *stream, int what) {
  I4Plan L{};
  gqaw_status s = plan_i4(x, &L);
  if (s != GQAW_OK) return s;
  const gqaw_paged_args *a = &x->paged;
  if (a->batch_size == 0 || a->total_new_tokens == 0 || a->max_new_tokens == 0) return GQAW_OK;  // no token, nothing to do
  if ((s = check_i4_pointers(x, L, what)) != GQAW_OK) return s;
  if ((s = check_device(a->workspace, "workspace")) != GQAW_OK) return s;
  I4Params p;
  std::memset(&p, 0, sizeof(p));
  fill_paged(a, L, &p);
  // without pages no row is read, but copies of no bytes still name a source: a valid address, of every head
  if (!a->num_pages) L.sp = L.sh = L.sr = L.tp = L.th = L.tr = 0;
  p.kp = a->num_pages ? a->key_pages : a->workspace;
  p.vp = a->num_pages ? a->value_pages : a->workspace;
  p.kscale = static_cast<uint16_t *>(a->num_pages ? x->key_scales : a->workspace);
  p.vscale = static_cast<uint16_t *>(a->num_pages ? x->value_scales : a->workspace);
  p.sp = L.sp, p.sh = L.sh, p.sr = L.sr;
  p.tp = L.tp, p.th = L.th, p.tr = L.tr;
  // ceil(2^(31 + l) / page) with 2^l >= page: its excess over the quotient, below 1, times j stays below 2^31 (Granlund, Montgomery)
  int l = 0;
  while ((1ll << l) < a->page_size) ++l;
  p.div_shift = 31 + l;
  p.div_mul = (uint32_t)(((unsigned __int128)1 << (31 + l)) / a->page_size + (((unsigned __int128)1 << (31 + l)) % a->page_size != 0));
  p.ko = x->key_out, p.vo = x->value_out;
  p.kos = L.kos, p.vos = L.vos;
  const bool bf16 = a->dtype == GQAW_BF16;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (what & kRead) {
    e = gqaw::launch_i4_rows(p, 0, x->key_out ? a->kv_num_heads : 0, x->value_out ? a->kv_num_heads : 0, true, bf16, st);
    if (e != cudaSuccess) return cuda_fail(e, "read kernel launch");
    gqaw::count_launch();
    return GQAW_OK;
  }
  if (what & kAppend) {
    const bool turn_q = (what & kAttend) && (L.rot_dim > 0 || a->query_weight);
    p.qout = static_cast<char *>(a->workspace) + L.off_q;
    p.qos = (long long)a->num_heads * a->head_size;
    if (turn_q && bf16) p.qlo = static_cast<char *>(a->workspace) + L.off_qlo;
    e = gqaw::launch_i4_rows(p, turn_q ? a->num_heads : 0, a->kv_num_heads, a->kv_num_heads, false, bf16, st);
    if (e != cudaSuccess) return cuda_fail(e, "append kernel launch");
    gqaw::count_launch();
    if (turn_q) {
      p.q = p.qout;
      p.qs = p.qos;
    }
  }
  return what & kAttend ? run_attend(a, L, p, st) : GQAW_OK;
}

}  // namespace

extern "C" {

size_t gqaw_paged_i4_workspace_bytes(const gqaw_paged_i4_args *args) {
  I4Plan L{};
  return plan_i4(args, &L) == GQAW_OK ? L.ws_bytes : 0;
}

gqaw_status gqaw_paged_i4_append(const gqaw_paged_i4_args *args, void *stream) { return run_i4(args, stream, kAppend); }

gqaw_status gqaw_paged_i4_attend(const gqaw_paged_i4_args *args, void *stream) { return run_i4(args, stream, kAttend); }

gqaw_status gqaw_paged_i4_step(const gqaw_paged_i4_args *args, void *stream) { return run_i4(args, stream, kAppend | kAttend); }

gqaw_status gqaw_paged_i4_read(const gqaw_paged_i4_args *args, void *stream) { return run_i4(args, stream, kRead); }

size_t gqaw_paged_i4_args_size(void) { return sizeof(gqaw_paged_i4_args); }

}  // extern "C"
