// Which sequence a new row belongs to, compiled for the host.
#include "gqaw_paged_sched.cuh"

extern "C" {

// For each of `rows` rows, the sequence that the append gives it to (-1: none).
void paged_owners(const int *qstart, const int *seqlens, int B, int N, int max_new, int max_len, int rows, int *out) {
  const gqaw::PBatch p{qstart, seqlens, B, N, max_new, max_len};
  for (int n = 0; n < rows; ++n) out[n] = gqaw::find_sequence(p, n);
}

}  // extern "C"
