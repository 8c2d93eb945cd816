// gqaw_paged.cuh -- parameters of the paged operators and the schedule that their attention
// kernels share.
//
// Schedule.  A unit is (sequence, head block, query tile): `tpt` consecutive new tokens of
// one sequence times the query heads of one kv head, against the key tiles (KEYS positions,
// aligned to KEYS) that any of them attends.  Sequences differ wildly in length, so the unit
// list is made on the device: every CTA scans the batch's lengths (a few KB from L2, about
// a microsecond) into a list of the sequences with work and the running count of their key
// tiles, which closed forms give without visiting the query tiles.  Then either
//   - split: CTA c takes tiles [c V / G, (c + 1) V / G) of the flattened sequence of all
//     units' tiles: equal work whatever the lengths.  A unit cut by a boundary is finished by
//     the last of its contributors, through partial results and a ticket; or
//   - whole: CTA c takes unit c alone, when the units fit in the grid and the longest costs
//     no more than an equal share plus the second unit epilogue that a cut brings
//     (kEpilogueTiles tiles each: a merge is a chain of dependent memory round trips).
// The ticket of a cut unit is indexed by the CTA it starts in (at most one unit leaves a CTA
// at its end), so the tickets have a fixed place whatever the shapes.
#pragma once

#include "gqaw_internal.cuh"

namespace gqaw {

constexpr int kPagedItems = 256;            // sequences of one launch; larger batches take several
constexpr int kPagedTickets = 1024;         // one per CTA
constexpr size_t kPagedTicketOffset = 256;  // after the status word
constexpr size_t kPagedPartialOffset = kPagedTicketOffset + kPagedTickets * 4;

struct PagedParams {
  const void *q, *k, *v;
  void *out;
  void *kp, *vp;
  long long qs, ks, vs, os;         // elements between tokens
  long long sp, sh, sr;             // elements between pages, heads, rows of the cache
  const int32_t *table, *qstart, *seqlens;
  const float *sink;
  int sink_mode;
  int B, N, max_new, max_len, Nq, Nkv, D, page, npages, width, W;  // W: 0 without a window
  int group, hblocks, gb;           // query heads per kv head; head blocks of gb heads per kv head
  int tpt;                          // tokens per query tile
  float qscale, capmul;             // as in Params
  uint32_t *status, *tickets;
  float *partials;
  // norm and rotation (gqaw_paged_rows.cu)
  const void *qw, *kw, *rcos, *rsin;
  const long long *pos_ids;
  int rot_dim, rot_inter, rot_len;
  float eps;
  void *qout, *kout;                // gqaw_qk_norm_rotary: where the rows go
  long long qos, kos;
};

__device__ __forceinline__ void pflag(const PagedParams &p, uint32_t bits) { atomicOr(p.status, bits); }

// A sequence with new tokens, as the schedule keeps it in shared memory.
struct PItem {
  long long tiles;  // key tiles of all sequences before this one
  long long units;  // units before it (64 bits: malformed row ranges may repeat rows)
  int b, T, qs, S;
};

// Where a CTA starts: found once, by one thread, and copied by every role's walker.
struct PStart {
  long long tb, te;  // this CTA's flattened tiles (split), or units (whole)
  long long pos;     // split: flattened index of the first tile of the unit it starts in
  int it, hu, r;     // that unit
  int G;             // CTAs that share the tiles
  bool whole;
};

struct PSched {
  PItem items[kPagedItems];
  long long V, U;   // key tiles and units in all
  int n;            // sequences with work
  int longest;      // key tiles of the longest unit
  long long wsum[32], wunits[32];
  int wcnt[32], wmax[32];
  PStart start;
};

// sum over i in [0, n) of floor((a i + b) / m); a, b >= 0, m > 0.
__device__ inline long long floor_sum(long long n, long long m, long long a, long long b) {
  long long s = 0;
  while (n > 0) {
    s += n * (n - 1) / 2 * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const long long y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const long long t = m;
    m = a;
    a = t;
  }
  return s;
}

template <int KEYS>
struct PTiles {
  long long P;
  int S, tpt, W, rt;
  __device__ __forceinline__ PTiles(const PagedParams &p, int T, int S_)
      : P((long long)T - S_), S(S_), tpt(p.tpt), W(p.W), rt((S_ + p.tpt - 1) / p.tpt) {}
  // first and one past the last key tile of query tile r
  __device__ __forceinline__ int lo(int r) const {
    const long long j = W > 0 ? P + (long long)r * tpt - W + 1 : 0;
    return (int)((j > 0 ? j : 0) / KEYS);
  }
  __device__ __forceinline__ int hi(int r) const {
    const long long s1 = (long long)(r + 1) * tpt < S ? (long long)(r + 1) * tpt : S;
    return (int)((P + s1 - 1) / KEYS) + 1;
  }
  // key tiles of query tiles [0, r)
  __device__ __forceinline__ long long before(int r) const {
    if (r <= 0) return 0;
    if (r == 1) return hi(0) - lo(0);
    const int full = r == rt ? r - 1 : r;  // the last query tile may be short
    long long s = full + floor_sum(full, KEYS, tpt, P + tpt - 1) + (r == rt ? hi(r - 1) : 0);
    if (W > 0) {
      const long long need = (long long)W - 1 - P;
      const long long i0 = need > 0 ? (need + tpt - 1) / tpt : 0;
      if (i0 < r) s -= floor_sum(r - i0, KEYS, tpt, P + i0 * tpt - W + 1);
    }
    return s;
  }
  // most key tiles of any query tile (an upper bound, exact for one)
  __device__ __forceinline__ int most() const {
    if (rt == 1) return hi(0) - lo(0);
    const int all = hi(rt - 1), span = W > 0 ? (int)(((long long)W - 2 + tpt) / KEYS) + 2 : all;
    return all < span ? all : span;
  }
};

constexpr int kEpilogueTiles = 6;

template <int KEYS>
__device__ inline void sched_start(const PagedParams &p, PSched *s, int cta, int grid) {
  PStart w;
  const long long V = s->V;
  const int heads = p.Nkv * p.hblocks;
  // at least a few tiles a CTA: a cut costs more than it saves below that
  w.G = (int)min((long long)grid, max(1LL, max(s->U, (V + 3) / 4)));
  w.whole = s->U <= grid && s->longest + kEpilogueTiles <= (V + w.G - 1) / w.G + 2 * kEpilogueTiles;
  w.it = w.hu = w.r = 0;
  w.pos = 0;
  if (w.whole) {
    w.tb = cta;
    w.te = cta < s->U ? cta + 1 : cta;
  } else {
    w.tb = cta < w.G ? cta * V / w.G : 0;
    w.te = cta < w.G ? (cta + 1) * V / w.G : 0;
  }
  if (w.tb < w.te) {
    int a = 0, b = s->n - 1;  // the last item that starts at or before tb
    while (a < b) {
      const int m = (a + b + 1) / 2;
      if ((w.whole ? s->items[m].units : s->items[m].tiles) <= w.tb)
        a = m;
      else
        b = m - 1;
    }
    w.it = a;
    const PItem &x = s->items[a];
    const PTiles<KEYS> t(p, x.T, x.S);
    if (w.whole) {
      const int off = (int)(w.tb - x.units);
      w.hu = off / t.rt;
      w.r = off - w.hu * t.rt;
    } else {
      const long long per = t.before(t.rt), off = w.tb - x.tiles;
      w.hu = (int)(off / per);
      const long long rem = off - w.hu * per;
      int c = 0, d = t.rt - 1;
      while (c < d) {
        const int m = (c + d + 1) / 2;
        if (t.before(m) <= rem)
          c = m;
        else
          d = m - 1;
      }
      w.r = c;
      w.pos = x.tiles + w.hu * per + t.before(c);
    }
    if (w.hu >= heads) w.te = w.tb;  // cannot happen: the counts above are of these units
  }
  s->start = w;
}

// Builds the list and this CTA's start; all `nt` threads of the CTA (a multiple of 32) call
// it, and it ends with a barrier.  CTA 0 flags the malformed sequences.
template <int KEYS>
__device__ inline void sched_build(const PagedParams &p, PSched *s, int nt) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
  const int heads = p.Nkv * p.hblocks;
  long long base = 0, units = 0;
  int count = 0, longest = 0;
  for (int b0 = 0; b0 < p.B; b0 += nt) {
    const int b = b0 + tid;
    long long n = 0, u = 0;
    int mx = 0, has = 0, T = 0, q0 = 0, S = 0;
    if (b < p.B) {
      q0 = p.qstart[b];
      const int q1 = p.qstart[b + 1];
      const long long TT = (long long)p.seqlens[b] + 1;
      S = q1 - q0;
      if (q0 < 0 || q1 < q0 || q1 > p.N || S > p.max_new || TT < S || TT > p.max_len) {
        if (blockIdx.x == 0) pflag(p, GQAW_DEV_BAD_SEQLEN);
      } else if (S > 0) {
        T = (int)TT;
        const PTiles<KEYS> t(p, T, S);
        has = 1;
        n = t.before(t.rt) * heads;
        u = (long long)t.rt * heads;
        mx = t.most();
      }
    }
    long long in = n, iu = u;  // inclusive scans over the warp, then over the warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, in, o);
      const long long y = __shfl_up_sync(0xffffffffu, iu, o);
      if (lane >= o) in += x, iu += y;
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    const uint32_t vote = __ballot_sync(0xffffffffu, has);
    if (lane == 31) {
      s->wsum[warp] = in;
      s->wunits[warp] = iu;
      s->wcnt[warp] = __popc(vote);
      s->wmax[warp] = mx;
    }
    __syncthreads();
    long long at = base + in - n, au = units + iu - u;
    int ac = count + __popc(vote & ((1u << lane) - 1u));
    for (int w = 0; w < nw; ++w) {
      if (w < warp) at += s->wsum[w], au += s->wunits[w], ac += s->wcnt[w];
      base += s->wsum[w];
      units += s->wunits[w];
      count += s->wcnt[w];
      longest = max(longest, s->wmax[w]);
    }
    if (has) s->items[ac] = PItem{at, au, b, T, q0, S};
    __syncthreads();
  }
  if (tid == 0) {
    s->V = base;
    s->n = count;
    s->U = units;
    s->longest = longest;
    sched_start<KEYS>(p, s, blockIdx.x, gridDim.x);
  }
  __syncthreads();
}

// The unit a walker stands on, and the part of its key tiles that this CTA does.
struct PUnit {
  int b, hu;           // sequence, head unit (kv head * hblocks + block)
  int row0, ntok;      // first row of query / output, tokens
  long long qpos;      // position of the first token
  int kt, nt;          // first key tile, key tiles of the unit
  int k0, k1;          // this CTA's tiles [k0, k1) of the nt
  long long g0;        // flattened index of its first tile (split)
};

// Walks the units of this CTA.
template <int KEYS>
struct PWalk {
  const PSched *s;
  PStart w;
  int heads;
  bool started;

  __device__ __forceinline__ PWalk(const PagedParams &p, const PSched *s_)
      : s(s_), w(s_->start), heads(p.Nkv * p.hblocks), started(false) {}
  // the CTA whose range holds flattened tile x
  __device__ __forceinline__ int owner(long long x) const { return (int)(((x + 1) * w.G - 1) / s->V); }

  __device__ inline bool next(const PagedParams &p, PUnit &u) {
    if (w.tb >= w.te) return false;
    if (started) {
      if (w.whole || w.pos >= w.te) return false;
      const int rt = (s->items[w.it].S + p.tpt - 1) / p.tpt;
      if (++w.r == rt) {
        w.r = 0;
        if (++w.hu == heads) {
          w.hu = 0;
          if (++w.it >= s->n) return false;
        }
      }
    }
    started = true;
    const PItem &x = s->items[w.it];
    const PTiles<KEYS> t(p, x.T, x.S);
    u.b = x.b;
    u.hu = w.hu;
    u.row0 = x.qs + w.r * p.tpt;
    u.ntok = min(p.tpt, x.S - w.r * p.tpt);
    u.qpos = t.P + (long long)w.r * p.tpt;
    u.kt = t.lo(w.r);
    u.nt = t.hi(w.r) - u.kt;
    u.g0 = w.pos;
    if (w.whole) {
      u.k0 = 0;
      u.k1 = u.nt;
    } else {
      u.k0 = (int)max(0LL, w.tb - w.pos);
      u.k1 = (int)min((long long)u.nt, w.te - w.pos);
      w.pos += u.nt;
    }
    return true;
  }
};

// Row offset (elements) of position j of sequence b, kv head h; -1 when its table entry is bad.
__device__ __forceinline__ long long cache_row(const PagedParams &p, int b, int h, int j) {
  const int pg = j / p.page;
  const int id = p.table[(long long)b * p.width + pg];
  if ((unsigned)id >= (unsigned)p.npages) return -1;
  return id * p.sp + h * p.sh + (long long)(j - pg * p.page) * p.sr;
}

__device__ __forceinline__ float paged_sink_log2(const PagedParams &p, int h) {
  if (p.sink_mode == 1) return p.sink[h] * kLog2e;
  return p.sink_mode == 2 ? 0.f : -INFINITY;
}

// softcap: tanh with its own saturation; an absolute error of about 1e-7
__device__ __forceinline__ float cap_logit(const PagedParams &p, float x) { return p.capmul * tanhf(x); }

}  // namespace gqaw
