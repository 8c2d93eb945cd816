// gqaw_i4_attend_f32.cu -- instances of the attention over 4-bit caches: fp32 rows.
#include "gqaw_i4_attend.cuh"

namespace gqaw {

cudaError_t launch_i4_attend_f32(const I4Params &p, int nt, int sms, cudaStream_t stream) {
  return launch_i4_attend_t<float, 2>(p, nt, sms, stream);
}

}  // namespace gqaw
