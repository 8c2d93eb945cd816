// The schedule of the attention over 4-bit caches, compiled for the host: the paged one with its own
// costs of a cut and of a short unit.
#include "paged_sched_kernels_host.cpp"

extern "C" long long i4_schedule(const int *lens, int n, int tpt, int window, int heads, int grid, int keys, int unit_cost,
                                 int merge_tiles, int min_tiles, long long *out, long long cap, long long *totals) {
  PShape p{tpt, window, heads, unit_cost};
  p.merge_tiles = merge_tiles;
  p.min_tiles = min_tiles;
  long long rows = 0;
  return keys == 32 && run<32>(lens, n, p, grid, out, cap, &rows, totals) ? rows : -1;
}
