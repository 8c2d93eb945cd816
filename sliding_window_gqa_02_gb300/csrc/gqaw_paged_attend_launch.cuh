// gqaw_paged_attend_launch.cuh -- launcher of the CUDA-core paged attention (one instance per
// head size and query-tile height).
#pragma once

#include <atomic>
#include <type_traits>

#include "gqaw_paged_warp.cuh"

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

template <typename T, int D, int RM>
cudaError_t launch_paged_warp_attend_one(const PagedParams &p, int sms, cudaStream_t stream) {
  using L = pwarp::Lay<T, D>;
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> ready[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(paged_warp_attend_kernel<T, D, RM>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kTotal);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) ready[dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sms * L::kPerSm));
  cfg.blockDim = dim3(L::kThreads);
  cfg.dynamicSmemBytes = L::kTotal;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see pdl_wait()
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged_warp_attend_kernel<T, D, RM>, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// At most 8 rows; head size 256 only for types of 2 bytes (two rings of 1 KB rows do not fit).
template <typename T>
cudaError_t launch_paged_warp_attend(const PagedParams &p, int rows, int sms, cudaStream_t stream) {
  auto pick = [&](auto d) {
    constexpr int D = decltype(d)::value;
    return rows <= 4 ? launch_paged_warp_attend_one<T, D, 4>(p, sms, stream)
                     : launch_paged_warp_attend_one<T, D, 8>(p, sms, stream);
  };
  switch (p.D) {
    case 8: return pick(std::integral_constant<int, 8>());
    case 16: return pick(std::integral_constant<int, 16>());
    case 32: return pick(std::integral_constant<int, 32>());
    case 64: return pick(std::integral_constant<int, 64>());
    case 128: return pick(std::integral_constant<int, 128>());
    default:
      if constexpr (sizeof(T) == 2) return pick(std::integral_constant<int, 256>());
      return cudaErrorInvalidValue;
  }
}

}  // namespace gqaw
