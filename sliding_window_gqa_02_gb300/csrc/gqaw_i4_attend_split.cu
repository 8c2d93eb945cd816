// gqaw_i4_attend_split.cu -- instances of the attention over 4-bit caches: bf16 rows, turned queries in two parts.
#include "gqaw_i4_attend.cuh"

namespace gqaw {

cudaError_t launch_i4_attend_split(const I4Params &p, int nt, int sms, cudaStream_t stream) {
  return launch_i4_attend_t<__nv_bfloat16, 2>(p, nt, sms, stream);
}

}  // namespace gqaw
