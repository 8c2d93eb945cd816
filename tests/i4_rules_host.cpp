// The rules of gqaw_i4_rules.cuh, compiled for the host.
#include <stdint.h>

#include "gqaw_i4_rules.cuh"

extern "C" int i4_blocks(long long page, long long D, long long sr, long long tr) { return gqaw::i4_blocks(page, D, sr, tr); }

// Do the kernel's 32-bit offsets of a lane's codes and scales in a block agree with 64 bits, for every lane?
extern "C" int i4_offsets_fit(long long D, long long sr, long long tr) {
  const long long CPR = D / 32, RPC = 32 / CPR, G = D / 32;
  const uint32_t sr16 = (uint32_t)(sr / 16), trg = (uint32_t)(tr / G);
  for (long long lane = 0; lane < 32; ++lane) {
    const uint32_t crow = lane / CPR, cpart = lane % CPR;
    if ((uint32_t)((crow * sr16 + cpart) << 4) != (uint64_t)crow * sr + cpart * 16) return 0;
    if ((uint32_t)(lane % RPC * trg * G) != (uint64_t)(lane % RPC) * tr) return 0;
  }
  return 1;
}
