// gqaw_paged_attend_f32.cu -- f32 instances of the CUDA-core paged attention.
#include "gqaw_paged_attend_launch.cuh"

namespace gqaw {
cudaError_t launch_paged_rows_attend_f32(const PagedParams &p, int bm, int grid, cudaStream_t stream) {
  return launch_paged_rows_attend<float>(p, bm, grid, stream);
}
cudaError_t launch_paged_warp_attend_f32(const PagedParams &p, int rows, int sms, cudaStream_t stream) {
  return launch_paged_warp_attend<float>(p, rows, sms, stream);
}
}  // namespace gqaw
