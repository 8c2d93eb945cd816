// gqaw_paged_sched.cuh -- the schedule of the paged attention kernels: which key tiles of
// which units each CTA takes.  No CUDA in here, so that the host can compile it too and check it
// for any batch.
//
// Schedule.  A unit is (sequence, head block, query tile): `tpt` consecutive new tokens of
// one sequence times the query heads of one kv head, against the key tiles (KEYS positions,
// aligned to KEYS) that any of them attends.  Sequences differ wildly in length, so the unit
// list is made on the device: every CTA scans the batch's lengths (a few KB from L2, about
// a microsecond) into a list of the sequences with work and the running count of their key
// tiles, which closed forms give without visiting the query tiles.  A unit costs its key tiles
// and, whatever their number, `unit_cost` tiles more (the pipeline drains and fills, rows go
// out: 4 us of a 128-row unit against 1.1 us a tile; a batch of short prompts counted without it
// left some CTAs twice the time of others).  Then either
//   - split: CTA c takes [c V / G, (c + 1) V / G) of the flattened sequence of all units' cost,
//     each unit's fixed part first: equal work whatever the lengths.  A unit whose tiles a
//     boundary cuts is finished by the last of its contributors, through partial results and a
//     ticket; or
//   - whole: CTA c takes unit c alone, when the units fit in the grid and the longest costs no
//     more than an equal share plus `merge_tiles`, what a cut costs (a merge is a chain of
//     dependent memory round trips).
// The ticket of a cut unit is indexed by the CTA it starts in (at most one unit leaves a CTA
// at its end), so the tickets have a fixed place whatever the shapes.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define GQAW_HD __host__ __device__ inline
#else
#define GQAW_HD inline
#endif

namespace gqaw {

constexpr int kPagedItems = 256;  // sequences of one launch; larger batches take several

// A vote of a whole warp: bit i is pred(i).  The host goes over the 32 lanes.
template <typename F>
GQAW_HD uint32_t warp_vote(F pred) {
#ifdef __CUDA_ARCH__
  return __ballot_sync(0xffffffffu, pred((int)(threadIdx.x & 31)));
#else
  uint32_t m = 0;
  for (int i = 0; i < 32; ++i) m |= pred(i) ? 1u << i : 0u;
  return m;
#endif
}
GQAW_HD int bits_set(uint32_t m) {
#ifdef __CUDA_ARCH__
  return __popc(m);
#else
  return __builtin_popcount(m);
#endif
}

// The batch as the device sees it: sequence b has rows [qstart[b], qstart[b + 1]) and length
// seqlens[b] + 1.
struct PBatch {
  const int32_t *qstart, *seqlens;
  int B, N, max_new, max_len;
};

// Is a sequence with rows [q0, q1) and length len + 1 one that no call touches?
GQAW_HD bool malformed(const PBatch &p, int q0, int q1, int len) {
  const long long S = (long long)q1 - q0, T = (long long)len + 1;
  return q0 < 0 || S < 0 || q1 > p.N || S > p.max_new || T < S || T > p.max_len;
}

// The sequence that row n belongs to: qstart[b] <= n < qstart[b + 1], and not malformed; -1 when
// there is none.  On the device a whole warp calls it.  The last b with qstart[b] <= n is
// searched 32 ways at a time, which finds it where the starts ascend.  Where they do not it may be
// any sequence: so what was found is checked, and if the row is not its own every sequence is asked,
// but for a row behind all of them (the padding of a batch).
GQAW_HD int find_sequence(const PBatch &p, int n) {
  auto owns = [&](int b) {
    const int q0 = p.qstart[b], q1 = p.qstart[b + 1];
    return q0 <= n && n < q1 && !malformed(p, q0, q1, p.seqlens[b]);
  };
  int lo = 0, size = p.B;
  for (bool first = true; size > 1 || first; first = false) {
    const int step = (size + 31) / 32;
    const int c = bits_set(warp_vote([&](int lane) { return lane * step < size && p.qstart[lo + lane * step] <= n; }));
    if (c == 0) break;
    const int rest = size - (c - 1) * step;
    lo += (c - 1) * step;
    size = step < rest ? step : rest;
  }
  if (owns(lo)) return lo;
  const bool behind = !warp_vote([&](int lane) {
    int top = 0;
#pragma unroll 8
    for (int b = lane; b <= p.B; b += 32) top = top > p.qstart[b] ? top : p.qstart[b];
    return top > n;
  });
  for (int b0 = 0; b0 < p.B && !behind; b0 += 32) {
    const uint32_t m = warp_vote([&](int lane) { return b0 + lane < p.B && owns(b0 + lane); });
    if (m) return b0 + bits_set((m & (0u - m)) - 1u);
  }
  return -1;
}

// What the schedule needs to know of a call.
struct PShape {
  int tpt, W, heads;    // tokens per query tile; window (0: none); kv heads x head blocks
  int unit_cost;        // key tiles that a unit costs beside its own
  int merge_tiles = 7;  // ... and what a cut costs
  // At least so many tiles a CTA: a cut costs more than it saves below that (one sequence of 1000
  // keys and 8 kv heads: 11.9 us; at least four a CTA 15.9, one 11.8, but 2000 keys 12.2, 14.3, 13.4)
  int min_tiles = 2;
};

// A sequence with new tokens, as the schedule keeps it in shared memory.
struct PItem {
  long long tiles;  // cost of all sequences before this one, in key tiles
  long long units;  // units before it (64 bits: malformed row ranges may repeat rows)
  int b, T, qs, S;
};

// Where a CTA starts: found once, by one thread, and copied by every role's walker.
struct PStart {
  long long tb, te;  // this CTA's part of the flattened cost (split), or units (whole)
  long long pos;     // split: where the unit it starts in begins
  int it, hu, r;     // that unit
  int G;             // CTAs that share the tiles
  bool whole;
};

struct PSched {
  PItem items[kPagedItems];
  long long V, U;   // cost and units in all
  int n;            // sequences with work
  int longest;      // cost of the longest unit
  PStart start;
};

// sum over i in [0, n) of floor((a i + b) / m); a, b >= 0, m > 0.
GQAW_HD long long floor_sum(long long n, long long m, long long a, long long b) {
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
  int S, tpt, W, rt, c0;
  GQAW_HD PTiles(const PShape &p, int T, int S_)
      : P((long long)T - S_), S(S_), tpt(p.tpt), W(p.W), rt((S_ + p.tpt - 1) / p.tpt), c0(p.unit_cost) {}
  // first and one past the last key tile of query tile r
  GQAW_HD int lo(int r) const {
    const long long j = W > 0 ? P + (long long)r * tpt - W + 1 : 0;
    return (int)((j > 0 ? j : 0) / KEYS);
  }
  GQAW_HD int hi(int r) const {
    const long long s1 = (long long)(r + 1) * tpt < S ? (long long)(r + 1) * tpt : S;
    return (int)((P + s1 - 1) / KEYS) + 1;
  }
  // cost of query tiles [0, r) for one head
  GQAW_HD long long before(int r) const {
    if (r <= 0) return 0;
    if (r == 1) return hi(0) - lo(0) + c0;
    const int full = r == rt ? r - 1 : r;  // the last query tile may be short
    long long s = (long long)r * c0 + full + floor_sum(full, KEYS, tpt, P + tpt - 1) + (r == rt ? hi(r - 1) : 0);
    if (W > 0) {
      const long long need = (long long)W - 1 - P;
      const long long i0 = need > 0 ? (need + tpt - 1) / tpt : 0;
      if (i0 < r) s -= floor_sum(r - i0, KEYS, tpt, P + i0 * tpt - W + 1);
    }
    return s;
  }
  // most that any query tile costs (an upper bound, exact for one)
  GQAW_HD int most() const {
    if (rt == 1) return hi(0) - lo(0) + c0;
    const int all = hi(rt - 1), span = W > 0 ? (int)(((long long)W - 2 + tpt) / KEYS) + 2 : all;
    return (all < span ? all : span) + c0;
  }
};

// The last i in [0, n) with le(i), for le that holds at 0 and, once false, stays false: 32 places
// at a time, for le may be a chain of divisions.  On the device a whole warp calls it.
template <typename F>
GQAW_HD int last_where(int n, F le) {
  int lo = 0;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int c = bits_set(warp_vote([&](int lane) { return lane * step < n && le(lo + lane * step); }));
    lo += (c - 1) * step;
    n = step < n - (c - 1) * step ? step : n - (c - 1) * step;
  }
  return lo;
}

// Where CTA `cta` starts; on the device a whole warp computes it.
template <int KEYS>
GQAW_HD PStart sched_start(const PShape &p, const PSched *s, int cta, int grid) {
  PStart w;
  const long long V = s->V;
  const int heads = p.heads;
  const long long most = (V + p.min_tiles - 1) / p.min_tiles, want = s->U > most ? s->U : most;
  w.G = (int)(want < 1 ? 1 : want < grid ? want : grid);
  w.whole = s->U <= grid && s->longest <= (V + w.G - 1) / w.G + p.merge_tiles;
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
    const int a = last_where(s->n, [&](int m) { return (w.whole ? s->items[m].units : s->items[m].tiles) <= w.tb; });
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
      const int c = last_where(t.rt, [&](int m) { return t.before(m) <= rem; });
      w.r = c;
      w.pos = x.tiles + w.hu * per + t.before(c);
    }
    if (w.hu >= heads) w.te = w.tb;  // cannot happen: the counts above are of these units
  }
  return w;
}

// The unit a walker stands on, and the part of its key tiles that this CTA does.
struct PUnit {
  int b, hu;           // sequence, head unit (kv head * hblocks + block)
  int row0, ntok;      // first row of query / output, tokens
  long long qpos;      // position of the first token
  int kt, nt;          // first key tile, key tiles of the unit
  int k0, k1;          // this CTA's tiles [k0, k1) of the nt
  long long g0;        // its first tile in the flattened cost (split)
};

// Walks the units of this CTA.
template <int KEYS>
struct PWalk {
  const PSched *s;
  PStart w;
  int heads;
  bool started;

  GQAW_HD PWalk(const PShape &p, const PSched *s_)
      : s(s_), w(s_->start), heads(p.heads), started(false) {}
  // the CTA whose part holds x of the flattened cost
  GQAW_HD int owner(long long x) const { return (int)(((x + 1) * w.G - 1) / s->V); }

  // The next unit with tiles for this CTA (a boundary may fall into a unit's fixed part).
  GQAW_HD bool next(const PShape &p, PUnit &u) {
    for (;;) {
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
      u.ntok = x.S - w.r * p.tpt < p.tpt ? x.S - w.r * p.tpt : p.tpt;
      u.qpos = t.P + (long long)w.r * p.tpt;
      u.kt = t.lo(w.r);
      u.nt = t.hi(w.r) - u.kt;
      u.k0 = 0;
      u.k1 = u.nt;
      u.g0 = w.pos + p.unit_cost;
      if (w.whole) return true;
      if (w.tb > u.g0) u.k0 = (int)(w.tb - u.g0);
      if (w.te < u.g0 + u.nt) u.k1 = (int)(w.te - u.g0 > 0 ? w.te - u.g0 : 0);
      w.pos = u.g0 + u.nt;
      if (u.k0 < u.k1) return true;
    }
  }
};

}  // namespace gqaw
