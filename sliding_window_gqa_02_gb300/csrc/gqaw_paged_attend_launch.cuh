// gqaw_paged_attend_launch.cuh -- launcher of the CUDA-core paged attention (one instance per
// head size and query-tile height).
#pragma once

#include <atomic>

#include "gqaw_paged_attend.cuh"

namespace gqaw {

template <typename T, int D, int BM>
cudaError_t launch_paged_rows_attend_one(const PagedParams &p, int grid, cudaStream_t stream) {
  constexpr int kMaxDevices = 64, kSmem = prow::Lay<T, D, BM>::kTotal;
  static std::atomic<bool> ready[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(paged_rows_attend_kernel<T, D, BM>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) ready[dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(prow::Lay<T, D, BM>::kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see pdl_wait()
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged_rows_attend_kernel<T, D, BM>, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_paged_rows_attend(const PagedParams &p, int bm, int grid, cudaStream_t stream) {
  if (bm == 16) {
    switch (p.D) {
      case 8: return launch_paged_rows_attend_one<T, 8, 16>(p, grid, stream);
      case 16: return launch_paged_rows_attend_one<T, 16, 16>(p, grid, stream);
      case 32: return launch_paged_rows_attend_one<T, 32, 16>(p, grid, stream);
      case 64: return launch_paged_rows_attend_one<T, 64, 16>(p, grid, stream);
      case 128: return launch_paged_rows_attend_one<T, 128, 16>(p, grid, stream);
      default: return launch_paged_rows_attend_one<T, 256, 16>(p, grid, stream);
    }
  }
  switch (p.D) {
    case 8: return launch_paged_rows_attend_one<T, 8, 128>(p, grid, stream);
    case 16: return launch_paged_rows_attend_one<T, 16, 128>(p, grid, stream);
    case 32: return launch_paged_rows_attend_one<T, 32, 128>(p, grid, stream);
    case 64: return launch_paged_rows_attend_one<T, 64, 128>(p, grid, stream);
    case 128: return launch_paged_rows_attend_one<T, 128, 128>(p, grid, stream);
    default: return launch_paged_rows_attend_one<T, 256, 64>(p, grid, stream);
  }
}

}  // namespace gqaw
