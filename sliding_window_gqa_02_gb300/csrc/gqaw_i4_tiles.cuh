// gqaw_i4_tiles.cuh -- key and value tiles of a 4-bit cache for the prompt kernel (gqaw_paged_pre.cuh):
// three warps read codes and scales from global memory and write the values as bf16 into the
// 128-byte swizzled operand tiles that TMA fills for a bf16 cache.
//
// A tile of 128 keys is four batches of 32 rows for the keys and four for the values, which the warps
// take in turn, a batch's codes in registers while the one before is written.  A lane has 16 bytes of a
// row, 32 elements with one scale: 128 + c is a nibble in the lower bits of a bf16's mantissa, less 136 it
// is c - 8, times the scale one rounding (none for the scales that the append writes).  A batch takes about
// 450 instructions of a warp and a tile 3600, of three warps; the tile is in use for 4700 cycles, so the
// tensor cores do not wait for it.
#pragma once

#include "gqaw_i4.cuh"
#include "gqaw_tc.cuh"

namespace gqaw {

namespace i4t {

__device__ __forceinline__ uint32_t bf_add2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf_mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t nibble2(uint32_t x, uint32_t s) {  // the lowest nibble of each half, as a value
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xea;" : "=r"(r) : "r"(x));
  return bf_mul2(bf_add2(r, 0xc308c308u), s);
}
// Eight codes as four pairs of values.
__device__ __forceinline__ uint4 values8(uint32_t w, uint32_t s) {
  const uint32_t a = nibble2(w, s), b = nibble2(w >> 4, s), c = nibble2(w >> 8, s), d = nibble2(w >> 12, s);
  return make_uint4(__byte_perm(a, b, 0x5410), __byte_perm(c, d, 0x5410), __byte_perm(a, b, 0x7632), __byte_perm(c, d, 0x7632));
}

// One element of position j, as the prompt kernel rounds it.
__device__ __forceinline__ float element(const I4Params &p, bool value, const I4Place &at, int kvh, int d) {
  const unsigned char *row = static_cast<const unsigned char *>(value ? p.vp : p.kp) + at.page * p.sp + kvh * p.sh + at.row * p.sr;
  const uint16_t s = (value ? p.vscale : p.kscale)[at.page * p.tp + kvh * p.th + at.row * p.tr + d / kI4Group];
  const float c = (float)((int)((row[d / 2] >> (4 * (d & 1))) & 15) - 8);
  return __bfloat162float(__float2bfloat16_rn(c * __uint_as_float((uint32_t)s << 16)));
}

// The rings that the tiles go to, and the barriers of their slots.
struct Rings {
  unsigned char *k, *v;
  uint64_t *k_full, *k_free, *v_full, *v_free;
};

// The batches of warp `cw` of kWarps, over all units of the CTA.  first(): called by warp 0, all lanes, when it
// has reached a unit's first batch (the queries' load).  Returns false when a wait expired or the CTA winds down.
constexpr int kWarps = 3, kBatches = 4;  // of keys in a tile, and of values; arrivals on a slot's barrier

template <int D, int STAGES, int HALF_BYTES, typename First>
__device__ inline bool convert(const I4Params &p, const PShape &shp, const PSched *sched, const Rings &ring, volatile int *abort_flag,
                               int cw, int lane, First first) {
  constexpr int CPR = D / 32, RPC = 32 / CPR, kTile = D / 64 * HALF_BYTES;  // lanes of a row, rows of a load
  const int row = lane / CPR, part = lane % CPR;
  PWalk<128> walk(shp, sched);
  PUnit u;
  int i = cw, tile = 0, gk = 0;  // batch of the tile, tile of the unit's part, tiles before in all
  bool have = walk.next(shp, u), fresh = true;
  auto settle = [&]() {  // to the tile that batch i lies in
    while (have && i >= 2 * kBatches) {
      i -= 2 * kBatches;
      ++gk;
      if (++tile == u.k1 - u.k0) {
        tile = 0;
        fresh = true;
        have = walk.next(shp, u);
      }
    }
  };
  uint4 codes[CPR];
  uint16_t scale[CPR];
  auto fetch = [&]() {  // batch i
    const bool value = i >= kBatches;
    const uint32_t j0 = (uint32_t)(u.kt + u.k0 + tile) * 128 + (i & (kBatches - 1)) * 32 + row;
    const long long lo = p.W > 0 && u.qpos - p.W + 1 > 0 ? u.qpos - p.W + 1 : 0, hi = u.qpos + u.ntok;
    const unsigned char *base = static_cast<const unsigned char *>(value ? p.vp : p.kp) + u.hu * p.sh + part * 16;
    const uint16_t *sbase = (value ? p.vscale : p.kscale) + u.hu * p.th + part;
#pragma unroll
    for (int c = 0; c < CPR; ++c) {
      const uint32_t j = j0 + c * RPC;
      codes[c] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
      scale[c] = 0;
      if (j >= lo && j < hi) {  // a row that some token attends
        const I4Place at = i4_place(p, u.b, j);
        if (at.page >= 0) {
          codes[c] = __ldg(reinterpret_cast<const uint4 *>(base + at.page * p.sp + at.row * p.sr));
          scale[c] = __ldg(sbase + at.page * p.tp + at.row * p.tr);
        } else {
          pflag(p, GQAW_DEV_BAD_PAGE);
        }
      }
    }
  };
  settle();
  if (have) fetch();
  while (have) {
    // what is at hand, before the next batch is asked for
    const bool value = i >= kBatches;
    const int st = gk % STAGES, turn = gk / STAGES, r0 = (i & (kBatches - 1)) * 32 + row;
    if (fresh && cw == 0 && !first()) return false;  // the queries before anything waits for their unit's slots
    fresh = false;
    uint4 now[CPR];
    uint32_t s2[CPR];
#pragma unroll
    for (int c = 0; c < CPR; ++c) now[c] = codes[c], s2[c] = (uint32_t)scale[c] * 0x10001u;
    i += kWarps;
    settle();
    if (have) fetch();
    bool fine = turn == 0 || mbar_wait(value ? &ring.v_free[st] : &ring.k_free[st], (turn & 1) ^ 1);
    fine = __all_sync(0xffffffffu, fine && !*abort_flag);
    if (!fine) return false;
    unsigned char *to = (value ? ring.v : ring.k) + st * kTile;
#pragma unroll
    for (int c = 0; c < CPR; ++c) {
      const int r = r0 + c * RPC;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        // the four parts in an order that keeps the lanes of a store in different banks
        const int w = y ^ (D >= 128 ? (part >> 1 & 1) * 2 : 0), el = part * 4 + w;  // 16-byte part of the row
        const uint32_t word = w == 0 ? now[c].x : w == 1 ? now[c].y : w == 2 ? now[c].z : now[c].w;
        *reinterpret_cast<uint4 *>(to + (el / 8) * HALF_BYTES + r * 128 + (((el & 7) ^ (r & 7)) << 4)) = values8(word, s2[c]);
      }
    }
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(value ? &ring.v_full[st] : &ring.k_full[st]);
  }
  return true;
}

}  // namespace i4t
}  // namespace gqaw
