// gqaw_paged_attend_bf16.cu -- bf16 instances of the CUDA-core paged attention.
#include "gqaw_paged_attend_launch.cuh"

namespace gqaw {
cudaError_t launch_paged_rows_attend_bf16(const PagedParams &p, int bm, int grid, cudaStream_t stream) {
  return launch_paged_rows_attend<__nv_bfloat16>(p, bm, grid, stream);
}
cudaError_t launch_paged_warp_attend_bf16(const PagedParams &p, int rows, int sms, cudaStream_t stream) {
  return launch_paged_warp_attend<__nv_bfloat16>(p, rows, sms, stream);
}
}  // namespace gqaw
