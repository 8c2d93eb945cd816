// gqaw_i4_tiles.cuh -- key and value tiles of a 4-bit cache for the prompt kernel (gqaw_paged_pre.cuh):
// seven warps read codes and scales from global memory and write the values as bf16 into the
// 128-byte swizzled operand tiles that TMA fills for a bf16 cache.
//
// A tile of 128 keys is taken apart into batches of 1024 / D rows, first of the keys, then of the values,
// which the warps take in turn; the codes of two batches ahead are in registers.  A lane has 16
// bytes of a row, 32 elements with one scale; a value is rounded to bf16 once (not at all with the scales that
// the append writes).
//
// Bound: the latencies of a warp on its own; a batch takes some 130 instructions and a tile 4200, beside
// the softmax warps' code in the instruction cache, so the loop has one batch and not a tile.  With three warps, each
// with four batches unrolled, a tile took 14600 cycles where the tensor cores want one every 5400.
#pragma once

#include <type_traits>

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
__device__ __forceinline__ uint32_t bf_fma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// Nibble k of each half of w as a value.  EXACT: the scale has so few bits, and is so small, that 24 of it
// are a bf16 number: the nibble in the upper bits of the mantissa of 16 is 16 + c, times the scale less 24 of it one multiply-add.  Else in
// the lower bits of 128: less 136, then times the scale.
template <bool EXACT, int K>
__device__ __forceinline__ uint32_t nibble2(uint32_t w, uint32_t s, uint32_t s24) {
  uint32_t r;
  if (EXACT) {
    asm("lop3.b32 %0, %1, 0x00780078, 0x41804180, 0xea;" : "=r"(r) : "r"(K == 0 ? w << 3 : w >> (4 * K - 3)));
    return bf_fma2(r, s, s24);
  }
  asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xea;" : "=r"(r) : "r"(w >> (4 * K)));
  return bf_mul2(bf_add2(r, 0xc308c308u), s);
}
// Eight codes as values: pairs (0, 4), (1, 5), (2, 6), (3, 7), or in their own order.
template <bool EXACT>
__device__ __forceinline__ uint4 values8(uint32_t w, uint32_t s, uint32_t s24, bool order) {
  const uint32_t a = nibble2<EXACT, 0>(w, s, s24), b = nibble2<EXACT, 1>(w, s, s24), c = nibble2<EXACT, 2>(w, s, s24), d = nibble2<EXACT, 3>(w, s, s24);
  return order ? make_uint4(__byte_perm(a, b, 0x5410), __byte_perm(c, d, 0x5410), __byte_perm(a, b, 0x7632), __byte_perm(c, d, 0x7632))
               : make_uint4(a, b, c, d);
}
// Column x of 8 of a value tile holds dimension value_column(x): the pairs are not put in order there,
// but when the outputs leave tensor memory, where that costs nothing.
__host__ __device__ constexpr int value_column(int x) { return (x & ~7) | (x & 1) * 4 | (x >> 1 & 3); }

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

constexpr int kWarps = 7;
template <int D>
constexpr int kBatches = 128 / (1024 / D);  // of keys in a tile, and of values: arrivals on a slot's barrier

// Where a warp's next batch lies; in shared memory, since the walk would take 40 registers.
struct Walker {
  PWalk<128> walk;
  PUnit u;
  uint32_t lo, hi;  // positions that some token attends
  int have;         // a unit
};

// The batches of warp `cw`, over all units of the CTA.  first(): called by warp 0, all lanes, when it has reached a
// unit's first batch (the queries' load).  Returns false when a wait expired or the CTA winds down.
template <int D, int STAGES, int HALF_BYTES, typename First>
__device__ inline bool convert(const I4Params &p, const PShape &shp, const PSched *sched, Walker *wk, const Rings &ring,
                               volatile int *abort_flag, int cw, int lane, First first) {
  constexpr int CPR = D / 32, RPC = 32 / CPR, NB = kBatches<D>, kTile = D / 64 * HALF_BYTES;  // lanes of a row, rows of a load
  const int row = lane / CPR, part = lane % CPR;
  auto advance = [&](bool start) {
    __syncwarp();
    if (lane == 0) {
      if (start) wk->walk = PWalk<128>(shp, sched);
      wk->have = wk->walk.next(shp, wk->u);
      const long long lo = p.W > 0 && wk->u.qpos - p.W + 1 > 0 ? wk->u.qpos - p.W + 1 : 0;
      wk->lo = (uint32_t)lo;
      wk->hi = (uint32_t)(wk->u.qpos + wk->u.ntok);
    }
    __syncwarp();
    return wk->have != 0;
  };
  // The batch whose pages are looked up: number i of tile `tile` of the unit, the gk-th in all.
  int i = cw, tile = 0, gk = 0;
  bool have = advance(true), fresh = true;
  // a batch's place in a word: number in its operand, operand, tile in all; the unit's first tile; none
  constexpr uint32_t kNone = 0xffffffffu, kFresh = 0x80000000u;
  auto settle = [&]() {  // to the tile that batch i lies in
    while (have && i >= 2 * NB) {
      i -= 2 * NB;
      ++gk;
      if (++tile == wk->u.k1 - wk->u.k0) {
        tile = 0;
        fresh = true;
        have = advance(false);
      }
    }
  };
  struct Ids {
    int id;         // this lane's page, or kNotNeeded
    uint32_t row;   // its row in it
    int kvh;
    uint32_t at;    // i | gk << 6 | kFresh, or kNone
  };
  auto look_up = [&]() {
    Ids x{kNotNeeded, 0u, 0, kNone};
    if (!have) return x;
    const uint32_t j = (uint32_t)(wk->u.kt + wk->u.k0 + tile) * 128 + (i & (NB - 1)) * RPC + row;
    const uint32_t page = (uint32_t)(((uint64_t)j * p.div_mul) >> p.div_shift);
    if (j >= wk->lo && j < wk->hi) x.id = needed_page(__ldg(p.table + (long long)wk->u.b * p.width + page));
    x.row = j - page * p.page;
    x.kvh = wk->u.hu;
    x.at = (uint32_t)i | ((uint32_t)gk << 6 & ~kFresh) | (fresh ? kFresh : 0u);
    fresh = false;
    i += kWarps;
    settle();
    return x;
  };
  struct Batch {
    uint4 codes;
    uint32_t scale, at;
  };
  auto fetch = [&](const Ids &x) {
    Batch b{make_uint4(0u, 0u, 0u, 0u), 0u, x.at};
    const bool value = (x.at & 63u) >= (uint32_t)NB;
    if ((unsigned)x.id < (unsigned)p.npages) {
      const uint4 *base = reinterpret_cast<const uint4 *>(static_cast<const unsigned char *>(value ? p.vp : p.kp) + x.kvh * p.sh);
      const uint16_t *sbase = (value ? p.vscale : p.kscale) + x.kvh * p.th + part;
      b.codes = __ldg(base + ((uint64_t)(uint32_t)x.id * p.sp16 + (uint64_t)x.row * p.sr16 + part));
      b.scale = __ldg(sbase + ((uint64_t)(uint32_t)x.id * p.tpg + (uint64_t)x.row * p.trg) * (D / kI4Group));
    } else if (x.id != kNotNeeded) {
      pflag(p, GQAW_DEV_BAD_PAGE);
    }
    return b;
  };
  settle();
  Ids ids = look_up();
  Batch cur = fetch(ids);
  ids = look_up();
  Batch next = fetch(ids);
  ids = look_up();
#pragma unroll 1
  while (cur.at != kNone) {
    const Batch far = fetch(ids);
    ids = look_up();
    if ((cur.at & kFresh) && cw == 0 && !first()) return false;  // the queries before anything waits for their unit's slots
    const uint32_t n = cur.at & 63u, g = (cur.at & ~kFresh) >> 6;
    const bool value = n >= (uint32_t)NB;
    const uint32_t st = g % STAGES, turn = g / STAGES, r = (n & (NB - 1)) * RPC + row;
    bool fine = turn == 0 || mbar_wait(value ? &ring.v_free[st] : &ring.k_free[st], (turn & 1) ^ 1);
    fine = __all_sync(0xffffffffu, fine && !*abort_flag);
    if (!fine) return false;
    unsigned char *to = (value ? ring.v : ring.k) + st * kTile + r * 128;
    const uint32_t s2 = cur.scale * 0x10001u, s24 = bf_mul2(s2, 0xc1c0c1c0u);  // -24 s
    auto put = [&](auto exact, bool order) {
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        // the four parts in an order that keeps the lanes of a store in different banks
        const int w = y ^ (D >= 128 ? (part >> 1 & 1) * 2 : 0), el = part * 4 + w;  // 16-byte part of the row
        const uint32_t word = (y & 1) ? (w & 2 ? cur.codes.w : cur.codes.y) : (w & 2 ? cur.codes.z : cur.codes.x);
        *reinterpret_cast<uint4 *>(to + (el / 8) * HALF_BYTES + (((el & 7) ^ (r & 7)) << 4)) = values8<exact.value>(word, s2, s24, order);
      }
    };
    // more than six bits, not of this library's append; or from 2^123 on, where 24 of it leave bf16 (or not finite)
    if (__any_sync(0xffffffffu, (cur.scale & 3u) != 0u || (cur.scale & 0x7fffu) >= (123u + 127u) << 7))
      put(std::false_type(), !value);
    else if (value)
      put(std::true_type(), false);
    else
      put(std::true_type(), true);
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(value ? &ring.v_full[st] : &ring.k_full[st]);
    cur = next;
    next = far;
  }
  return true;
}

}  // namespace i4t
}  // namespace gqaw
