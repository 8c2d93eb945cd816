// The schedule of the paged attention kernels, compiled for the host: what every CTA of a grid
// takes, as one flat list for the test to check.
#include <type_traits>
#include <vector>

#include "gqaw_paged_sched.cuh"

extern "C" {

// lens: (S, T) per sequence.  out: 12 numbers per (CTA, unit): cta, b, hu, row0, ntok, qpos, kt,
// nt, k0, k1, first owner, last owner.  Returns the count of rows (or -1 if `cap` is too small);
// totals: V, U, whole.
long long paged_schedule(const int *lens, int n, int tpt, int window, int heads, int grid, int keys32, int unit_cost, long long *out,
                         long long cap, long long *totals) {
  using namespace gqaw;
  const PShape p{tpt, window, heads, unit_cost};
  std::vector<char> mem(sizeof(PSched));
  PSched *s = reinterpret_cast<PSched *>(mem.data());
  long long rows = 0;
  auto run = [&](auto keys) -> bool {
    constexpr int KEYS = decltype(keys)::value;
    s->V = s->U = 0;
    s->n = s->longest = 0;
    int row = 0;
    for (int b = 0; b < n; ++b) {
      const int S = lens[2 * b], T = lens[2 * b + 1];
      if (S > 0) {
        const PTiles<KEYS> t(p, T, S);
        s->items[s->n++] = PItem{s->V, s->U, b, T, row, S};
        s->V += t.before(t.rt) * heads;
        s->U += (long long)t.rt * heads;
        s->longest = s->longest > t.most() ? s->longest : t.most();
      }
      row += S;
    }
    for (int cta = 0; cta < grid; ++cta) {
      s->start = sched_start<KEYS>(p, s, cta, grid);
      PWalk<KEYS> w(p, s);
      PUnit u;
      while (w.next(p, u)) {
        if (rows >= cap) return false;
        long long *o = out + 12 * rows++;
        const bool whole = s->start.whole;
        const long long v[12] = {cta, u.b, u.hu, u.row0, u.ntok, u.qpos, u.kt, u.nt, u.k0, u.k1,
                                 whole ? cta : w.owner(u.g0), whole ? cta : w.owner(u.g0 + u.nt - 1)};
        for (int i = 0; i < 12; ++i) o[i] = v[i];
      }
    }
    totals[0] = s->V;
    totals[1] = s->U;
    totals[2] = s->start.whole;
    return true;
  };
  const bool ok = keys32 ? run(std::integral_constant<int, 32>()) : run(std::integral_constant<int, 128>());
  return ok ? rows : -1;
}

}  // extern "C"
