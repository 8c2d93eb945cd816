// The schedule of the paged attention kernels with any of their tile widths and unit costs,
// compiled for the host, and the search that a warp makes in it.
#include <type_traits>
#include <vector>

#include "gqaw_paged_sched.cuh"

namespace {

using namespace gqaw;

template <int KEYS>
bool run(const int *lens, int n, const PShape &p, int grid, long long *out, long long cap, long long *rows, long long *totals) {
  std::vector<char> mem(sizeof(PSched));
  PSched *s = reinterpret_cast<PSched *>(mem.data());
  s->V = s->U = 0;
  s->n = s->longest = 0;
  int row = 0;
  for (int b = 0; b < n; ++b) {
    const int S = lens[2 * b], T = lens[2 * b + 1];
    if (S > 0) {
      const PTiles<KEYS> t(p, T, S);
      s->items[s->n++] = PItem{s->V, s->U, b, T, row, S};
      s->V += t.before(t.rt) * p.heads;
      s->U += (long long)t.rt * p.heads;
      s->longest = s->longest > t.most() ? s->longest : t.most();
    }
    row += S;
  }
  *rows = 0;
  for (int cta = 0; cta < grid; ++cta) {
    s->start = sched_start<KEYS>(p, s, cta, grid);
    PWalk<KEYS> w(p, s);
    PUnit u;
    while (w.next(p, u)) {
      if (*rows >= cap) return false;
      const bool whole = s->start.whole;
      const long long v[12] = {cta, u.b, u.hu, u.row0, u.ntok, u.qpos, u.kt, u.nt, u.k0, u.k1,
                               whole ? cta : w.owner(u.g0), whole ? cta : w.owner(u.g0 + u.nt - 1)};
      long long *o = out + 12 * (*rows)++;
      for (int i = 0; i < 12; ++i) o[i] = v[i];
    }
  }
  totals[0] = s->V;
  totals[1] = s->U;
  totals[2] = s->start.whole;
  return true;
}

}  // namespace

extern "C" {

// lens: (S, T) per sequence.  out: 12 numbers per (CTA, unit), as in paged_sched_host.cpp.  Returns
// the count of rows, -1 where they are more than `cap`, -2 for a tile width that no kernel has.
long long paged_schedule_of(const int *lens, int n, int tpt, int window, int heads, int grid, int keys, int unit_cost,
                            long long *out, long long cap, long long *totals) {
  const PShape p{tpt, window, heads, unit_cost};
  long long rows = 0;
  bool ok = false;
  switch (keys) {
    case 16: ok = run<16>(lens, n, p, grid, out, cap, &rows, totals); break;
    case 32: ok = run<32>(lens, n, p, grid, out, cap, &rows, totals); break;
    case 128: ok = run<128>(lens, n, p, grid, out, cap, &rows, totals); break;
    default: return -2;
  }
  return ok ? rows : -1;
}

// last_where over [0, n) with the places up to `last` true.
int paged_last_where(int n, int last) {
  return gqaw::last_where(n, [&](int i) { return i <= last; });
}

}  // extern "C"
