// gqaw_i4_pre.cu -- instances of the prompt kernel for caches in 4 bits: bf16, head sizes 64 and 128, more
// than 40 query rows of a kv head.
#include "gqaw_paged_pre.cuh"

namespace gqaw {

// The queries come in two parts where p.qlo is set.
cudaError_t launch_i4_prefill(const I4Params &p, const PagedMaps &maps, int grid, cudaStream_t stream) {
  static std::atomic<bool> ready[4][kPrefillDevices];
  auto two = [&](auto d, auto split, int i) {
    return launch_prefill(paged_prefill2_kernel<d.value, split.value, I4Params>, ready[i], ppre::threads2<I4Params>,
                          ppre::Lay2<d.value, split.value>::kAlloc, p, maps, grid, stream);
  };
  constexpr std::integral_constant<int, 64> d64{};
  constexpr std::integral_constant<int, 128> d128{};
  constexpr std::true_type split{};
  constexpr std::false_type whole{};
  if (p.D == 64) return p.qlo ? two(d64, split, 0) : two(d64, whole, 1);
  return p.qlo ? two(d128, split, 2) : two(d128, whole, 3);
}

}  // namespace gqaw
