// gqaw_i4.cuh -- parameters of the operators on paged caches held in 4 bits.
//
// A row of D elements: D / 2 bytes of codes (element 2 i low, 2 i + 1 high in byte i) and D / 32
// bf16 scales; code c stands for (c - 8) scale.  In PagedParams kp and vp are the codes, and sp, sh,
// sr their strides in bytes.
#pragma once

#include "gqaw_i4_rules.cuh"
#include "gqaw_paged.cuh"

namespace gqaw {

constexpr int kI4Group = 32;

struct I4Params : PagedParams {
  uint16_t *kscale, *vscale;    // bf16 bits
  long long tp, th, tr;         // elements between pages, heads, rows of scales
  void *ko, *vo;                // read: rows out, either may be NULL
  long long kos, vos;
  uint32_t div_mul;               // j / page = j div_mul >> div_shift, for j < 2^31
  int div_shift;
  // attention: rows of the cache by 16 bytes of codes and one row's scales
  uint32_t sp16, sr16, tpg, trg;  // strides of pages and rows, in 16 bytes and in rows of scales
  long long to_values, to_value_scales;  // bytes from key codes to value codes, and from key scales to value scales
  bool blocks;                    // i4_blocks()
};

// Where position j of sequence b lies: page and row in it; page -1 when its entry is bad.
struct I4Place {
  long long page;
  int row;
};
__device__ __forceinline__ I4Place i4_place(const I4Params &p, int b, long long j) {
  const uint32_t pg = (uint32_t)(((uint64_t)(uint32_t)j * p.div_mul) >> p.div_shift);
  const int id = p.table[(long long)b * p.width + pg];
  return {(unsigned)id < (unsigned)p.npages ? id : -1, (int)((uint32_t)j - pg * p.page)};
}

}  // namespace gqaw
