// gqaw_paged_pre.cu -- instances of the prompt kernels for bf16 caches.
#include "gqaw_paged_pre.cuh"

namespace gqaw {

// What the models on the host take from this file: the schedule's cost of a unit, and the buffers of odd bits.
namespace model {
constexpr int kUnitCost = 3;
constexpr int kOddBufs = 3;
static_assert(kUnitCost == ppre::kUnitCost && kOddBufs == ppre::kOddBufs, "the kernels'");
}  // namespace model

// halves: query tiles of 128 rows per unit, 1 or 2 (2: head sizes 64 and 128).  The queries come
// in two parts where p.qlo is set.
cudaError_t launch_paged_prefill(const PagedParams &p, const PagedMaps &maps, int halves, int grid, cudaStream_t stream) {
  static std::atomic<bool> ready[10][kPrefillDevices];
  auto one = [&](auto d, auto split, int i) {
    return launch_prefill(paged_prefill_kernel<d.value, split.value>, ready[i], ppre::kThreads,
                          ppre::Lay<d.value, split.value>::kAlloc, p, maps, grid, stream);
  };
  auto two = [&](auto d, auto split, int i) {
    return launch_prefill(paged_prefill2_kernel<d.value, split.value>, ready[i], ppre::kThreads2,
                          ppre::Lay2<d.value, split.value>::kAlloc, p, maps, grid, stream);
  };
  constexpr std::integral_constant<int, 64> d64{};
  constexpr std::integral_constant<int, 128> d128{};
  constexpr std::integral_constant<int, 256> d256{};
  constexpr std::true_type split{};
  constexpr std::false_type whole{};
  if (p.D == 64) {
    if (halves == 2) return p.qlo ? two(d64, split, 0) : two(d64, whole, 1);
    return p.qlo ? one(d64, split, 2) : one(d64, whole, 3);
  }
  if (p.D == 128) {
    if (halves == 2) return p.qlo ? two(d128, split, 4) : two(d128, whole, 5);
    return p.qlo ? one(d128, split, 6) : one(d128, whole, 7);
  }
  return p.qlo ? one(d256, split, 8) : one(d256, whole, 9);
}

}  // namespace gqaw
