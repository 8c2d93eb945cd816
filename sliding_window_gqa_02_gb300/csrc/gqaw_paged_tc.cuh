// gqaw_paged_tc.cuh -- what the two tensor-core kernels of the paged attention share: their
// tensor maps, and the TMA loads of a key or value tile through the page table.
//
// A tile is 128 consecutive positions of one sequence and kv head: 128 / page_size pages (or
// a part of one), each a box of min(page_size, 128) rows x 64 dimensions of the 4-dimensional
// cache (dimension, row, kv head, page).  A box lands as whole 8-row groups of the 128-byte
// swizzled operand layout, so the boxes of a tile stacked in row order are the operand; that
// is why page_size must be a multiple of 8 that divides 128 or is divided by it.  Boxes that
// hold no position any row of the unit attends are not loaded (their pages may be gone).
#pragma once

#include "gqaw_paged.cuh"
#include "gqaw_tc.cuh"

namespace gqaw {

struct PagedMaps {
  CUtensorMap q;   // query (N, Nq, D): box (64, group, tokens of a query tile)
  CUtensorMap ql;  // the same of what bf16 left of the queries (PagedParams::qlo); encoded where that is set
  CUtensorMap k;   // key pages (pages, kv heads, rows, D): box (64, box rows, 1, 1)
  CUtensorMap v;   // value pages
};

namespace ptc {

constexpr int kKeys = 128;
constexpr int kHalf = 16384;  // 64 dimensions of a tile: 128 rows of 128 bytes

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, int c0, int c1, int c2, int c3,
                                            uint64_t *bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, "
      "%3, %4, %5}], [%6], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// The maps' own way to the SM, ahead of the first load through them.
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(x) = 1 - 2 / (e^(2x) + 1), absolute error about 1e-7; saturates to the right limits and
// keeps a NaN.
__device__ __forceinline__ float fast_tanh(float x) {
  const float e = fast_exp2(2.8853900817779268f * x);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return fmaf(-2.f, r, 1.f);
}

// What a warp needs to load the tiles of a unit; lane i looks after box i.
struct Boxes {
  int rows, n;          // rows of a box, boxes of a tile
  long long jlo, jhi;   // positions that some row of the unit attends
  int b, kvh;
  int id, row;          // this lane's box of the tile looked up last: page (-1: not loaded), row in it

  __device__ __forceinline__ void unit(const PagedParams &p, const PUnit &u) {
    rows = p.page < kKeys ? p.page : kKeys;
    n = kKeys / rows;
    jlo = p.W > 0 && u.qpos - p.W + 1 > 0 ? u.qpos - p.W + 1 : 0;
    jhi = u.qpos + u.ntok;
    b = u.b;
    kvh = u.hu;
  }
  // page table entries of key tile kt (all lanes)
  __device__ __forceinline__ void look_up(const PagedParams &p, int kt, int lane) {
    const long long j = (long long)kt * kKeys + lane * rows;
    id = -1;
    if (lane < n && j < jhi && j + rows > jlo) {
      const int pg = (int)(j / p.page);
      id = p.table[(long long)b * p.width + pg];
      row = (int)(j - (long long)pg * p.page);
    }
  }
  // drops the boxes whose entry is out of range; returns the boxes to load as a mask
  __device__ __forceinline__ uint32_t valid(const PagedParams &p, int kt, int lane) {
    const long long j = (long long)kt * kKeys + lane * rows;
    const bool want = lane < n && j < jhi && j + rows > jlo, ok = want && (unsigned)id < (unsigned)p.npages;
    if (want && !ok) pflag(p, GQAW_DEV_BAD_PAGE);
    return __ballot_sync(0xffffffffu, ok);
  }
  // issues the loads of one operand tile (all lanes; `mask` from valid()).  One lane issues
  // them all: the instruction takes its operands from uniform registers, and lanes that each
  // issue their own box are serialised at a higher cost.
  template <int HALVES>
  __device__ __forceinline__ void load(const CUtensorMap *map, unsigned char *dst, uint64_t *bar, uint64_t pol,
                                       uint32_t mask, int lane) const {
    for (int i = 0; i < n; ++i) {
      const int bid = __shfl_sync(0xffffffffu, id, i), brow = __shfl_sync(0xffffffffu, row, i);
      if (lane == 0 && ((mask >> i) & 1u)) {
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf)
          tma_load_4d(dst + hf * kHalf + i * rows * 128, map, hf * 64, brow, kvh, bid, bar, pol);
      }
    }
  }
};

}  // namespace ptc
}  // namespace gqaw
