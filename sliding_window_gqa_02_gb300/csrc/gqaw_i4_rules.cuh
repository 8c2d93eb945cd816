// gqaw_i4_rules.cuh -- rules of the operators on 4-bit caches that need no GPU, and whose tests compile them for the host.
#pragma once

namespace gqaw {

// Whether a lane of the attention's row kernel finds one block of 1024 / D rows for all: the block lies in one page,
// and a row's offset in it fits 32 bits, in bytes of codes (rows `sr` apart) and in scales (`tr` apart), which
// saves the registers of two 64-bit products.  Else every lane looks up its own rows, in 64 bits (16 contexts of 8192
// keys, 8 kv heads, pages of a multiple of those rows and not: head size 32 50 and 62 us, 64 38 and 56, 128 54 and 83,
// 256 103 and 146).
constexpr bool i4_blocks(long long page, long long D, long long sr, long long tr) {
  const long long rows = 1024 / D;
  return page % rows == 0 && (rows - 1) * sr + D / 2 <= 1ll << 32 && (rows - 1) * tr < 1ll << 32;
}

}  // namespace gqaw
