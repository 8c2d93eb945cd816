// gqaw_paged_pre.cuh -- paged attention of many query rows per kv head (prompt chunks, and
// batches that mix them with decoding sequences) on the 5th-generation tensor cores, bf16,
// head sizes 64, 128 and 256.
//
// A query tile is 128 rows, row = token * group + head, of one sequence and kv head; a key
// tile is 128 positions, fetched through the page table (gqaw_paged_tc.cuh):
//   S = Q K^T      M = 128 rows, N = 128 keys, K = D; both operands in shared memory
//   O += P V       M = 128 rows, N = D, K = 128 keys; P (bf16) in tensor memory
// Bound: the softmax of a tile (one 2^x per row and key, and what surrounds it) against 4 D
// multiply-adds per row and key, so both run all the time: S(k + 1) is issued while the softmax
// works on S(k), and O += P(k) V(k) while it works on S(k + 1).
//
// Softmax: sixteen warps, four threads per row (TMEM lane) with 32 keys each, which stay in
// registers from one load to the store of P: a counter run of the form with two threads per row
// and two loads showed the warps waiting for tensor memory (issue slots 25% busy, exponential
// unit 18%).  The four share the row's maximum through shared memory; the reference moves only
// when exceeded by more than 2^8, so O is rarely rescaled.  Sums are fp32 of the unrounded
// weights; P is rounded to bf16 for its product (2^-9 relative, the size of the output's own
// rounding: what bf16 leaves of P would cost a second product).  Queries that the step has turned
// come in two bf16 parts (SPLIT) and S is the sum of two products: error
// of a whole prompt step 0.0025 -> 0.0020 for 8% more time, where the outputs' own rounding is
// 0.0016.  Warps without rows (a decoding sequence among chunks has `group` rows of the 128)
// only keep the barriers turning.
//
// Tensor memory (512 columns), head sizes 64 and 128: S in two buffers [0, 256), O from 256,
// P in two buffers [384, 512).  Head size 256 needs 256 columns for O: S has one buffer
// [0, 128), P two [128, 256), and S(k + 1) waits for P(k).
//
// Warps: 0-15 softmax, 16 MMA issue, 17 loads of Q and K, 18 loads of V (a lane looks up a box).
// Schedule, splits and merges: gqaw_paged.cuh.  A cut unit's partial rows go out column-major
// so that a warp's 32 rows are contiguous.
//
// Keys that some rows attend and others do not lie in the tiles along the diagonal and the
// window's edge.  There the softmax threads zero the value rows that nobody attends, and look
// for rows that are not finite among those that only some attend (0 x inf is NaN): these are
// zeroed too, and added at the unit's end to the rows that attend them, from global memory.
//
// Up to 32 rows (a verify step) lie in one quarter of the lanes, whose warps share one scheduler and
// its exponential unit: that bounds such a step (16 x 8 tokens, window 4096: 53.7 us, 59.7 with a cap,
// whose logits take three of its operations each; 40.6 of memory).
//
// Every wait is bounded; one that expires flags GQAW_DEV_TIMEOUT and the CTA winds down.
#pragma once

#include <atomic>
#include <type_traits>

#include "gqaw_i4_tiles.cuh"
#include "gqaw_paged_tc.cuh"

namespace gqaw {

namespace ppre {

using ptc::kHalf;
using ptc::kKeys;
using ptc::fast_exp2;
constexpr int kRows = 128;
constexpr int kParts = 4, kCols = kKeys / kParts;  // threads per row, and the keys of each
constexpr int kSoft = 32 * 4 * kParts;              // softmax threads
constexpr int kMmaWarp = 4 * kParts, kKWarp = kMmaWarp + 1, kVWarp = kMmaWarp + 2;
constexpr int kThreads = kSoft + 96;
// two query tiles at once
constexpr int kSoft2 = 256, kThreads2 = kSoft2 + 128;
constexpr int kMmaWarp2 = 8, kKWarp2 = 9, kVWarp2 = 10;
template <typename P>
constexpr int threads2 = std::is_same<P, I4Params>::value ? kSoft2 + 256 : kThreads2;
constexpr uint32_t kTmemCols = 512;
constexpr int kUnitCost = 3;   // see gqaw_paged_sched.cuh
constexpr float kRescaleLog2 = 8.0f;  // log2 units
constexpr int kSoftBar = 5;    // named barrier of the softmax warps (1-4: those of a lane quarter)
// Buffers of the bits of values that are not finite.  Unit i (of those with keys that only some rows
// attend) sets bits in buffer i % kOddBufs, its warps meet at a barrier and read them, and behind the
// barrier buffer (i - 1) % kOddBufs is cleared, which every warp has read before it came there.  It is
// next used by unit i + 2, whose bits are set behind the next barrier: with two buffers it would be
// unit i + 1's, and a warp that is ahead could set bits before they are cleared.
constexpr int kOddBufs = 3;

template <int D, bool SPLIT>
struct Lay {
  static constexpr int HALVES = D / 64;
  static constexpr int kTile = HALVES * kHalf;
  static constexpr int kKSt = D == 64 ? 4 : D == 128 ? (SPLIT ? 2 : 3) : 1;
  static constexpr int kVSt = D == 64 ? 4 : D == 128 ? 2 : 1;
  static constexpr int kSBuf = D == 256 ? 1 : 2;
  static constexpr uint32_t kTmemP = D == 256 ? 128 : 384, kTmemO = 256;
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + (SPLIT ? 2 : 1) * kTile;  // Q, and what bf16 left of it
  // Two parts of Q leave head size 256 one slot, which a tile's keys and then its values take
  static constexpr bool kOneSlot = D == 256 && SPLIT;
  static constexpr int kV = kOneSlot ? kK : kK + kKSt * kTile;
  static constexpr int kSched = kV + kVSt * kTile;
  static constexpr int kXch = kSched + (int)((sizeof(PSched) + 15) / 16 * 16);  // float [3][kParts][128]
  // keys attended by some rows only whose values are not finite, as bits: uint32
  // [buffer][part of the dimensions][0: after the first token, 1: before the last token's window][4]
  static constexpr int kOdd = kXch + 3 * kParts * kRows * 4;
  static constexpr int kMisc = kOdd + kOddBufs * kParts * 8 * 4;  // flags
  static constexpr int kStage = (kMisc + 16 + 255) / 256 * 256;  // 32 rows x 16 columns of output per softmax warp
  static constexpr int kBars = kStage + kSoft / 32 * 1024;
  static constexpr int kAlloc = kBars + 32 * 8 + 1024;  // and room to align the base
  static_assert(kAlloc <= 232448, "shared memory");
};

// One thread of the (converged) warp, the same every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
// A wait by the whole warp.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

// Packed pairs of fp32: one instruction computes both lanes.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Bit c set when column c of 32 lies in [c_lo, c_hi).
__device__ __forceinline__ uint32_t col_mask(int c_lo, int c_hi) {
  const uint32_t below_hi = c_hi >= 32 ? 0xffffffffu : (1u << c_hi) - 1u;
  const uint32_t below_lo = c_lo >= 32 ? 0xffffffffu : (1u << c_lo) - 1u;
  return below_hi & ~below_lo;
}

// 128 consecutive 32-bit columns of this thread's lane, loads and wait in one statement.
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, float (&v)[128]) {
  uint32_t r[128];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%128];\n"
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
      "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95, "
      "%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, "
      "%112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%129];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]),
        "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]), "=&r"(r[15]),
        "=&r"(r[16]), "=&r"(r[17]), "=&r"(r[18]), "=&r"(r[19]), "=&r"(r[20]), "=&r"(r[21]), "=&r"(r[22]), "=&r"(r[23]),
        "=&r"(r[24]), "=&r"(r[25]), "=&r"(r[26]), "=&r"(r[27]), "=&r"(r[28]), "=&r"(r[29]), "=&r"(r[30]), "=&r"(r[31]),
        "=&r"(r[32]), "=&r"(r[33]), "=&r"(r[34]), "=&r"(r[35]), "=&r"(r[36]), "=&r"(r[37]), "=&r"(r[38]), "=&r"(r[39]),
        "=&r"(r[40]), "=&r"(r[41]), "=&r"(r[42]), "=&r"(r[43]), "=&r"(r[44]), "=&r"(r[45]), "=&r"(r[46]), "=&r"(r[47]),
        "=&r"(r[48]), "=&r"(r[49]), "=&r"(r[50]), "=&r"(r[51]), "=&r"(r[52]), "=&r"(r[53]), "=&r"(r[54]), "=&r"(r[55]),
        "=&r"(r[56]), "=&r"(r[57]), "=&r"(r[58]), "=&r"(r[59]), "=&r"(r[60]), "=&r"(r[61]), "=&r"(r[62]), "=&r"(r[63]),
        "=&r"(r[64]), "=&r"(r[65]), "=&r"(r[66]), "=&r"(r[67]), "=&r"(r[68]), "=&r"(r[69]), "=&r"(r[70]), "=&r"(r[71]),
        "=&r"(r[72]), "=&r"(r[73]), "=&r"(r[74]), "=&r"(r[75]), "=&r"(r[76]), "=&r"(r[77]), "=&r"(r[78]), "=&r"(r[79]),
        "=&r"(r[80]), "=&r"(r[81]), "=&r"(r[82]), "=&r"(r[83]), "=&r"(r[84]), "=&r"(r[85]), "=&r"(r[86]), "=&r"(r[87]),
        "=&r"(r[88]), "=&r"(r[89]), "=&r"(r[90]), "=&r"(r[91]), "=&r"(r[92]), "=&r"(r[93]), "=&r"(r[94]), "=&r"(r[95]),
        "=&r"(r[96]), "=&r"(r[97]), "=&r"(r[98]), "=&r"(r[99]), "=&r"(r[100]), "=&r"(r[101]), "=&r"(r[102]), "=&r"(r[103]),
        "=&r"(r[104]), "=&r"(r[105]), "=&r"(r[106]), "=&r"(r[107]), "=&r"(r[108]), "=&r"(r[109]), "=&r"(r[110]), "=&r"(r[111]),
        "=&r"(r[112]), "=&r"(r[113]), "=&r"(r[114]), "=&r"(r[115]), "=&r"(r[116]), "=&r"(r[117]), "=&r"(r[118]), "=&r"(r[119]),
        "=&r"(r[120]), "=&r"(r[121]), "=&r"(r[122]), "=&r"(r[123]), "=&r"(r[124]), "=&r"(r[125]), "=&r"(r[126]), "=&r"(r[127])
      : "r"(taddr), "r"(taddr + 64));
#pragma unroll
  for (int i = 0; i < 128; ++i) v[i] = __uint_as_float(r[i]);
}

// P = 2^(z zs - base) of 32 logits as bf16 pairs into 16 columns at tp; returns their sum.
__device__ __forceinline__ float put_p(const float *v, uint32_t tp, float zs, float base) {
  const uint64_t zs2 = pack2(zs, zs), nb2 = pack2(-base, -base);
  uint64_t acc[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
  uint32_t pk[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    float x0, x1;
    unpack2(fma2(pack2(v[2 * c], v[2 * c + 1]), zs2, nb2), x0, x1);
    const float a0 = fast_exp2(x0), a1 = fast_exp2(x1);
    acc[c & 1] = add2(acc[c & 1], pack2(a0, a1));
    pk[c] = tc::pack_bf16x2(a0, a1);
  }
  tc::tmem_st16_async(tp, pk);
  float l0, l1, l2, l3;
  unpack2(acc[0], l0, l1);
  unpack2(acc[1], l2, l3);
  return (l0 + l1) + (l2 + l3);
}

__device__ __forceinline__ bool odd_pair(uint32_t w) {
  return (w & 0x7f800000u) == 0x7f800000u || (w & 0x00007f80u) == 0x00007f80u;
}

}  // namespace ppre

template <int D, bool SPLIT>
__global__ void __launch_bounds__(ppre::kThreads, 1)
    paged_prefill_kernel(const PagedParams p, const __grid_constant__ PagedMaps maps) {
  using namespace ppre;
  using L = Lay<D, SPLIT>;
  constexpr int QP = SPLIT ? 2 : 1;  // parts of the queries
  constexpr int OC = D / kParts;  // output columns of a softmax thread
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  PSched *sched = reinterpret_cast<PSched *>(smem + L::kSched);
  float *xch = reinterpret_cast<float *>(smem + L::kXch);  // [tile & 1 | 2 for the sums][part][row]
  uint32_t *odd = reinterpret_cast<uint32_t *>(smem + L::kOdd);
  volatile int *misc = reinterpret_cast<volatile int *>(smem + L::kMisc);
  volatile int *abort_flag = misc;
  volatile int *s_last = misc + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMisc + 8);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBars);
  uint64_t *q_full = bars, *q_free = bars + 1, *o_free = bars + 2, *mma_done = bars + 3;
  uint64_t *s_full = bars + 4, *p_full = bars + 6, *pv_done = bars + 8;  // two each
  uint64_t *k_full = bars + 10, *k_free = bars + 14, *v_full = bars + 18, *v_free = bars + 22;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    ptc::prefetch_map(&maps.q);
    ptc::prefetch_map(&maps.k);
    ptc::prefetch_map(&maps.v);
    mbar_init(q_full, 1);
    mbar_init(q_free, 1);
    mbar_init(o_free, kSoft / 32);
    mbar_init(mma_done, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kSoft / 32);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < L::kKSt; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_free[i], 1);
    }
    for (int i = 0; i < L::kVSt; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_free[i], 1);
    }
    mbar_fence_init();
    *abort_flag = 0;
    for (int i = 0; i < kOddBufs * kParts * 8; ++i) odd[i] = 0u;
  }
  // query rows past tpt * group stay zero
  for (int e = tid; e < QP * L::kTile / 16; e += kThreads) reinterpret_cast<uint4 *>(smem + L::kQ)[e] = make_uint4(0, 0, 0, 0);
  if (warp == 0) tc::tmem_alloc(tmem_slot, kTmemCols);
  tc::fence_proxy_async_smem();
  pdl_wait();
  const PShape shp = shape_of(p, kUnitCost);
  sched_build<kKeys>(p, shp, sched);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int g = p.group;
  // Key tiles are numbered across the CTA's units (gk), query tiles too (qi), so every ring
  // and barrier phase runs on from unit to unit.

  if (warp == kKWarp || warp == kVWarp) {
    // ------------------------------------------------------------ loads (whole warp)
    const bool value = warp == kVWarp;
    const uint64_t pol = tc::policy_evict_normal(), qpol = policy_evict_first();
    const int nst = value ? L::kVSt : L::kKSt;
    uint64_t *full = value ? v_full : k_full, *empty = value ? v_free : k_free;
    unsigned char *ring = smem + (value ? L::kV : L::kK);
    const CUtensorMap *map = value ? &maps.v : &maps.k;
    PWalk<kKeys> w(shp, sched);
    PUnit u;
    ptc::Boxes bx;
    int gk = 0, qi = 0;
    bool fine = true;
    while (fine && w.next(shp, u)) {
      bx.unit(p, u);
      bx.look_up(p, u.kt + u.k0, lane);
      for (int k = u.k0; k < u.k1; ++k, ++gk) {
        const uint32_t mask = bx.valid(p, u.kt + k, lane);
        const ptc::Boxes cur = bx;
        if (k + 1 < u.k1) bx.look_up(p, u.kt + k + 1, lane);
        const int st = gk % nst;
        if (gk >= nst) fine = mbar_wait(&empty[st], ((gk / nst) & 1) ^ 1);
        // one slot: keys after the last tile's values have been used, values after this tile's keys
        if (L::kOneSlot && fine && (value || gk > 0)) fine = mbar_wait(value ? k_free : v_free, (value ? gk : gk - 1) & 1);
        fine = __all_sync(0xffffffffu, fine && !*abort_flag);
        if (!fine) break;
        if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)(__popc(mask) * bx.rows * 128 * L::HALVES));
        __syncwarp();
        cur.load<L::HALVES>(map, ring + st * L::kTile, &full[st], pol, mask, lane);
        // the query tile after the unit's first K tile, once the last S product with the
        // previous one is done
        if (k == u.k0 && !value) {
          if (qi > 0) fine = mbar_wait(q_free, (qi - 1) & 1);
          fine = __all_sync(0xffffffffu, fine);
          if (!fine) {
            ++gk;
            break;
          }
          if (lane == 0) {
            mbar_arrive_expect_tx(q_full, (uint32_t)(QP * L::HALVES * g * p.tpt * 128));
            for (int h = 0; h < QP * L::HALVES; ++h)
              tc::tma_load_3d(smem + L::kQ + h * kHalf, h < L::HALVES ? &maps.q : &maps.ql, h % L::HALVES * 64, u.hu * g, u.row0, q_full, qpol);
          }
          ++qi;
        }
      }
    }
    if (lane == 0) {
      if (!fine) {
        pflag(p, GQAW_DEV_TIMEOUT);
        *abort_flag = 1;
      }
      // no copy may still be landing in shared memory when the CTA exits
      for (int j = gk > nst ? gk - nst : 0; j < gk; ++j)
        if (!mbar_wait(&full[j % nst], (j / nst) & 1)) pflag(p, GQAW_DEV_TIMEOUT);
      if (!value && qi > 0 && !mbar_wait(q_full, (qi - 1) & 1)) pflag(p, GQAW_DEV_TIMEOUT);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issue
    // The whole warp runs the loop and one elected thread issues: descriptors and addresses are
    // then uniform values, which is what the instruction takes.
    {
      constexpr uint32_t kIdescQK = tc::idesc_bf16_f32(kRows, kKeys, 0, 0);
      constexpr uint32_t kIdescPV = tc::idesc_bf16_f32(kRows, D, 0, 1);
      const uint64_t dq = tc::smem_desc_sw128(smem + L::kQ, 16, 1024);
      const uint64_t dk = tc::smem_desc_sw128(smem + L::kK, 16, 1024);
      const uint64_t dv = tc::smem_desc_sw128(smem + L::kV, kHalf, 1024);
      auto s_product = [&](int gt) -> bool {  // S(gt) into its buffer; K(gt) is waited for
        const int st = gt % L::kKSt;
        if (!warp_wait(&k_full[st], (gt / L::kKSt) & 1)) return false;
        tc::fence_after_sync();
        const uint64_t b0 = dk + (uint64_t)((st * L::kTile) >> 4);
        const uint32_t ds = tmem + (gt % L::kSBuf) * kKeys;
        if (elect_one()) {
#pragma unroll 1
          for (int q = 0; q < QP; ++q) {  // not unrolled: the descriptors of 16 products would spill
            const uint64_t aq = dq + (uint64_t)((q * L::kTile) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t off = (uint64_t)(((kk / 4) * kHalf + (kk % 4) * 32) >> 4);
              tc::mma_bf16_ss(ds, aq + off, b0 + off, kIdescQK, q + kk > 0);
            }
          }
          tc::mma_commit(&s_full[gt & 1]);
          tc::mma_commit(&k_free[st]);
        }
        __syncwarp();
        return true;
      };
      auto pv_product = [&](int gt, bool acc) -> bool {  // P(gt) is waited for by the caller
        const int st = gt % L::kVSt;
        if (!warp_wait(&v_full[st], (gt / L::kVSt) & 1)) return false;
        tc::fence_after_sync();
        // V: keys are K, 64-dimension halves (N) 16 KB apart, 8-key groups 1 KB apart
        const uint64_t b0 = dv + (uint64_t)((st * L::kTile) >> 4);
        const uint32_t pa = tmem + L::kTmemP + (gt & 1) * (kKeys / 2);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            tc::mma_bf16_ts(tmem + L::kTmemO, pa + kk * 8, b0 + (uint64_t)((kk * 16 * 128) >> 4), kIdescPV, acc || kk > 0);
          tc::mma_commit(&pv_done[gt & 1]);
          tc::mma_commit(&v_free[st]);
        }
        __syncwarp();
        return true;
      };
      PWalk<kKeys> w(shp, sched);
      PUnit u;
      int gk = 0, qi = 0;
      bool fine = true;
      while (fine && __all_sync(0xffffffffu, !*abort_flag) && w.next(shp, u)) {
        const int n = u.k1 - u.k0;
        fine = warp_wait(q_full, qi & 1) && s_product(gk);
        if (!fine) break;
        if (n == 1 && elect_one()) tc::mma_commit(q_free);
        for (int k = 0; k < n && fine; ++k) {
          const int gt = gk + k;
          bool have_p = false;
          if (L::kOneSlot) {  // S(k + 1) has its keys only once P(k) V(k) is done
            fine = warp_wait(&p_full[gt & 1], (gt >> 1) & 1) && (k > 0 || qi == 0 || warp_wait(o_free, (qi - 1) & 1)) &&
                   pv_product(gt, k > 0);
            if (fine && k + 1 < n) {
              fine = s_product(gt + 1);
              if (fine && k + 2 == n && elect_one()) tc::mma_commit(q_free);
            }
            continue;
          }
          if (L::kSBuf == 1) {  // the one S buffer is free once P(k) is written
            fine = warp_wait(&p_full[gt & 1], (gt >> 1) & 1);
            have_p = true;
            if (!fine) break;
          }
          if (k + 1 < n) {  // two buffers: P(k - 1), waited for below, freed this one
            fine = s_product(gt + 1);
            if (!fine) break;
            if (k + 2 == n && elect_one()) tc::mma_commit(q_free);  // the unit's last S product
          }
          if (!have_p) fine = warp_wait(&p_full[gt & 1], (gt >> 1) & 1);
          // the first O += P V of a unit overwrites O: the softmax has read the last unit's
          if (fine && k == 0 && qi > 0) fine = warp_wait(o_free, (qi - 1) & 1);
          if (fine) fine = pv_product(gt, k > 0);
        }
        gk += n;
        ++qi;
      }
      if (!fine) {
        if (lane == 0) pflag(p, GQAW_DEV_TIMEOUT);
        *abort_flag = 1;
      }
      if (elect_one()) tc::mma_commit(mma_done);  // every MMA issued has completed before TMEM is released
      if (!warp_wait(mma_done, 0)) if (lane == 0) pflag(p, GQAW_DEV_TIMEOUT);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int wq = warp & 3, hf = warp >> 2;  // TMEM lane quarter, part of the tile's keys
    const int r = wq * 32 + lane;             // query row = TMEM lane
    const int bar_q = 1 + wq;                 // named barrier of the warps of this lane quarter
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t to = tmem + L::kTmemO + hf * OC + lane_off, tp = tmem + L::kTmemP + hf * (kCols / 2) + lane_off;
    const bool plain = p.capmul == 0.f;
    // A cap of at most 64 (log2 units) bounds every logit: P against the reference 0 stays
    // within 2^64 both ways, so no maximum is taken and the threads of a row never meet.
    const bool fixed = p.capmul != 0.f && p.capmul <= 64.f;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out);
    PWalk<kKeys> w(shp, sched);
    PUnit u;
    int gk = 0, odd_at = 0;  // ... and the unit's buffer of odd bits
    // A warp that gives up a tile (an expired wait, an abort elsewhere) still runs every unit's
    // epilogue: the softmax warps meet at its barriers.
    while (w.next(shp, u)) {
      const int rows = u.ntok * g, n = u.k1 - u.k0;
      const bool idle = wq * 32 >= rows;      // no row of this warp exists
      const bool row_ok = r < rows;
      const int rr = row_ok ? r : rows - 1;   // rows past the unit's follow its last one
      const int tok = rr / g, h = u.hu * g + rr - tok * g;
      const long long at = u.qpos + tok;      // absolute position of the row's token
      const long long rlo = p.W > 0 && at - p.W + 1 > 0 ? at - p.W + 1 : 0;
      const long long jlo = p.W > 0 && u.qpos - p.W + 1 > 0 ? u.qpos - p.W + 1 : 0, jhi = u.qpos + u.ntok;
      const long long tile0 = (long long)(u.kt + u.k0) * kKeys;
      // visible columns [lo, hi) of this thread's part, relative to its first column in the
      // tile; both fall by 128 from tile to tile and are kept at -128 once below it
      int lo = (int)min(max(rlo - tile0 - hf * kCols, -128LL), 1LL << 30);
      int hi = (int)min(max(at + 1 - tile0 - hf * kCols, -128LL), 1LL << 30);
      float m_run = fixed ? 0.f : -INFINITY, l_run = 0.f;
      // some key of this CTA's tiles is attended by some of the unit's tokens only
      const bool has_part =
          u.ntok > 1 && (tile0 + (long long)n * kKeys - 1 > u.qpos || (p.W > 0 && tile0 < jhi - p.W));
      int done = 0;
      for (int k = 0; k < n; ++k) {
        const int gt = gk + k;
        const uint32_t ts = tmem + (uint32_t)(gt % L::kSBuf) * kKeys + hf * kCols + lane_off;
        const uint32_t tpk = tp + (uint32_t)(gt & 1) * (kKeys / 2);
        const int c_lo = min(max(lo, 0), kCols), c_hi = min(max(hi, 0), kCols);
        lo = max(lo - kKeys, -kKeys);
        hi = max(hi - kKeys, -kKeys);
        bool okw = __all_sync(0xffffffffu, !*abort_flag && mbar_wait(&s_full[gt & 1], (gt >> 1) & 1));
        tc::fence_after_sync();
        if (!idle && (okw || !fixed)) {
          float v[32];
          tc::tmem_ld32(ts, v);
          if (!plain) {  // cap tanh(z) = cap - 2 cap / (e^(2z) + 1)
            const float z2 = 2.8853900817779268f * p.qscale, c2 = -2.f * p.capmul;
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              float q;
              asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(1.f + fast_exp2(v[c] * z2)));
              v[c] = fmaf(c2, q, p.capmul);
            }
          }
          if (!__all_sync(0xffffffffu, c_lo == 0 && c_hi == kCols)) {
            const uint32_t m = col_mask(c_lo, c_hi);
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = (m >> c) & 1u ? v[c] : -INFINITY;
          }
          const float zs = plain ? p.qscale : 1.f;
          if (fixed) {
            l_run += put_p(v, tpk, 1.f, 0.f);
          } else {
            float m3[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) m3[c] = max3(v[8 * c], v[8 * c + 1], v[8 * c + 2]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              m3[c] = max3(m3[c], v[8 * c + 3], v[8 * c + 4]);
              m3[c] = max3(m3[c], v[8 * c + 5], v[8 * c + 6]);
              m3[c] = fmaxf(m3[c], v[8 * c + 7]);
            }
            // the row's maximum over its four threads (slot gt & 1: everyone has read slot gt & 1
            // of tile gt - 2 before the barrier of tile gt - 1)
            float *x = xch + (gt & 1) * kParts * kRows + r;
            x[hf * kRows] = fmaxf(max3(m3[0], m3[1], m3[2]), m3[3]) * zs;  // zs > 0
            okw = !named_barrier_or(bar_q, 32 * kParts, !okw);
            if (okw) {
              const float mt = fmaxf(max3(x[0], x[kRows], x[2 * kRows]), x[3 * kRows]);
              float alpha = 1.f;
              if (mt > m_run + kRescaleLog2) {  // the four decide alike
                alpha = m_run == -INFINITY ? 0.f : fast_exp2(m_run - mt);
                m_run = mt;
              }
              if (k > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                const bool okv = __all_sync(0xffffffffu, mbar_wait(&pv_done[(gt - 1) & 1], ((gt - 1) >> 1) & 1));
                okw = !named_barrier_or(bar_q, 32 * kParts, !okv);
                tc::fence_after_sync();
                if (okw) {
#pragma unroll 1
                  for (int c = 0; c < OC; c += 16) {
                    float o[16];
                    tc::tmem_ld16(to + c, o);
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] *= alpha;
                    tc::tmem_st16(to + c, o);
                  }
                }
              }
              l_run = l_run * alpha + put_p(v, tpk, zs, m_run == -INFINITY ? 0.f : m_run);
            }
          }
        }
        if (!okw) {
          if (lane == 0) pflag(p, GQAW_DEV_TIMEOUT);
          *abort_flag = 1;
          break;
        }
        // ---- value rows of the tile: key t = tid & 127, a part of its dimensions
        const long long j0 = tile0 + (long long)k * kKeys;
        const bool ends = j0 < jlo || j0 + kKeys > jhi;
        const bool part = u.ntok > 1 && (j0 + kKeys - 1 > u.qpos || (p.W > 0 && j0 < jhi - p.W));
        if (ends || part) {
          const int st = gt % L::kVSt;
          // With one V stage, V(gt - 1) may not have landed yet, and a parity wait cannot tell
          // two phases apart: O += P(gt - 1) V(gt - 1) first.  (With two, S(gt) was issued after
          // the product that waited for V(gt - 2).)
          if (L::kVSt == 1 && gt > 0 && !mbar_wait(&pv_done[(gt - 1) & 1], ((gt - 1) >> 1) & 1)) *abort_flag = 1;
          if (!mbar_wait(&v_full[st], (gt / L::kVSt) & 1)) *abort_flag = 1;
          const int t = tid & 127;
          const long long j = j0 + t;
          unsigned char *row = smem + L::kV + st * L::kTile + t * 128;
          constexpr int C0 = OC / 8;  // 16-byte parts of a row for this thread
          bool zero = j < jlo || j >= jhi;
          if (!zero && part && (j > u.qpos || (p.W > 0 && j < jhi - p.W))) {
            for (int c = hf * C0; c < (hf + 1) * C0; ++c) {
              const uint4 y = *reinterpret_cast<const uint4 *>(row + (c / 8) * kHalf + (((c & 7) ^ (t & 7)) << 4));
              zero |= odd_pair(y.x) || odd_pair(y.y) || odd_pair(y.z) || odd_pair(y.w);
            }
            if (zero) {
              const int kind = j > u.qpos ? 0 : 1, i = (int)(j - (kind ? jlo : u.qpos));
              atomicOr(&odd[(odd_at * kParts + hf) * 8 + kind * 4 + i / 32], 1u << (i & 31));
            }
          }
          if (zero)
            for (int c = hf * C0; c < (hf + 1) * C0; ++c)
              *reinterpret_cast<uint4 *>(row + (c / 8) * kHalf + (((c & 7) ^ (t & 7)) << 4)) = make_uint4(0, 0, 0, 0);
          tc::fence_proxy_async_smem();
        }
        __syncwarp();
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[gt & 1]);
        ++done;
      }
      // the last O += P V; the row sum over its four threads
      const int gl = gk + n - 1;
      const bool okf = done == n && __all_sync(0xffffffffu, mbar_wait(&pv_done[gl & 1], (gl >> 1) & 1));
      float *xs = xch + 2 * kParts * kRows + r;
      xs[hf * kRows] = l_run;
      if (named_barrier_or(bar_q, 32 * kParts, !okf)) {
        if (lane == 0) pflag(p, GQAW_DEV_TIMEOUT);
        *abort_flag = 1;
      }
      l_run = (xs[0] + xs[kRows]) + (xs[2 * kRows] + xs[3 * kRows]);
      tc::fence_after_sync();
      bool any_odd = false;
      const volatile uint32_t *mine = odd + (odd_at * kParts + hf) * 8;
      if (has_part) {
        named_barrier(kSoftBar, kSoft);
        for (int i = 0; i < 8; ++i) any_odd |= mine[i] != 0u;
        if (tid < kParts * 8) odd[(odd_at + kOddBufs - 1) % kOddBufs * kParts * 8 + tid] = 0u;
      }

      // ---- this part's OC columns of (O, m, l), 16 at a time
      const bool cut = u.k0 > 0 || u.k1 < u.nt;
      const int cta = blockIdx.x, cf = cut ? w.owner(u.g0) : cta, cl = cut ? w.owner(u.g0 + u.nt - 1) : cta;
      float4 *const parts = reinterpret_cast<float4 *>(p.partials);
      // partial block of a CTA: D / 4 float4 columns of O and one of (m, l), 128 rows each
      auto part_at = [&](int c, int c4) {
        return parts + (((long long)c * 2 + (c == cf ? 1 : 0)) * (D / 4 + 1) + c4) * kRows + r;
      };
      const float inv = cut ? 1.f : sink_reciprocal(l_run, m_run, paged_sink_log2(p, h));
      // 16 columns of the warp's 32 rows to memory, by way of shared memory: 2 lanes write the 32
      // bytes of a row (a lane writing its own row would touch 32 lines with every store)
      const long long orow = (u.row0 + tok) * p.os + (long long)h * D;  // of this lane's row
      auto put_rows = [&](const float (&v)[16], float f, int d0) {
        unsigned char *st = smem + L::kStage + warp * 1024;
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint4 y;
          y.x = tc::pack_bf16x2(v[8 * c] * f, v[8 * c + 1] * f);
          y.y = tc::pack_bf16x2(v[8 * c + 2] * f, v[8 * c + 3] * f);
          y.z = tc::pack_bf16x2(v[8 * c + 4] * f, v[8 * c + 5] * f);
          y.w = tc::pack_bf16x2(v[8 * c + 6] * f, v[8 * c + 7] * f);
          *reinterpret_cast<uint4 *>(st + lane * 32 + ((c ^ ((lane >> 2) & 1)) << 4)) = y;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = i * 16 + (lane >> 1), c = lane & 1;
          const long long at_ = __shfl_sync(0xffffffffu, orow, row);
          const uint4 y = *reinterpret_cast<const uint4 *>(st + row * 32 + ((c ^ ((row >> 2) & 1)) << 4));
          if (wq * 32 + row < rows) *reinterpret_cast<uint4 *>(out + at_ + d0 + c * 8) = y;
        }
      };
#pragma unroll 1
      for (int c16 = 0; c16 < OC; c16 += 16) {
        float v[16];
        __syncwarp();
        tc::tmem_ld16(to + c16, v);
        if (c16 + 16 == OC) {  // O has left tensor memory: the next unit may overwrite it
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_free);
        }
        const int d0 = hf * OC + c16;
        if (any_odd && row_ok)  // their weights anew, from the cache, for the rows that attend them
          for (int i = 0; i < 8; ++i)
            for (uint32_t bits = mine[i]; bits; bits &= bits - 1u) {
              const long long j = (i < 4 ? u.qpos : jlo) + (i & 3) * 32 + __ffs((int)bits) - 1;
              const long long off = j >= rlo && j <= at ? cache_row(p, u.b, u.hu, (int)j) : -1;
              if (off < 0) continue;
              const __nv_bfloat16 *kr = static_cast<const __nv_bfloat16 *>(p.kp) + off;
              const __nv_bfloat16 *vr = static_cast<const __nv_bfloat16 *>(p.vp) + off + d0;
              const long long q_at = (u.row0 + tok) * p.qs + (long long)h * D;
              const __nv_bfloat16 *qr = static_cast<const __nv_bfloat16 *>(p.q) + q_at;
              const __nv_bfloat16 *ql = static_cast<const __nv_bfloat16 *>(p.qlo) + q_at;
              float z = 0.f;
#pragma unroll 4
              for (int d = 0; d < D; ++d) {
                float x = __bfloat162float(qr[d]);
                if (SPLIT) x += __bfloat162float(ql[d]);
                z = fmaf(x, __bfloat162float(kr[d]), z);
              }
              z *= p.qscale;
              if (!plain) z = p.capmul * ptc::fast_tanh(z);
              const float pr = fast_exp2(z - m_run);
#pragma unroll
              for (int c = 0; c < 16; ++c) v[c] = fmaf(pr, __bfloat162float(vr[c]), v[c]);
            }
        if (cut) {
          if (row_ok)
#pragma unroll
            for (int c = 0; c < 16; c += 4) *part_at(cta, (d0 + c) / 4) = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
        } else {
          put_rows(v, inv, d0);
        }
      }
      if (has_part) odd_at = (odd_at + 1) % kOddBufs;
      if (cut) {
        if (hf == 0 && row_ok) *part_at(cta, D / 4) = make_float4(m_run, l_run, 0.f, 0.f);
        named_barrier(kSoftBar, kSoft);
        if (tid == 0) {
          __threadfence();
          *s_last = atomicAdd(&p.tickets[cf], 1u) == (unsigned)(cl - cf);
        }
        named_barrier(kSoftBar, kSoft);
        if (*s_last) {
          __threadfence();
          float M = -INFINITY, S = 0.f;
#pragma unroll 4
          for (int c = cf; c <= cl; ++c) M = fmaxf(M, row_ok ? __ldcg(part_at(c, D / 4)).x : 0.f);
          const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll 4
          for (int c = cf; c <= cl; ++c) {
            const float4 ml = row_ok ? __ldcg(part_at(c, D / 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
            S = fmaf(fast_exp2(ml.x - ref), ml.y, S);
          }
          const float winv = sink_reciprocal(S, M, paged_sink_log2(p, h));
#pragma unroll 1
          for (int c16 = 0; c16 < OC; c16 += 16) {
            const int d0 = hf * OC + c16;
            float acc[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) acc[c] = 0.f;
            if (row_ok)
#pragma unroll 2
              for (int c = cf; c <= cl; ++c) {
                const float f = fast_exp2(__ldcg(part_at(c, D / 4)).x - ref);
                float4 y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = __ldcg(part_at(c, d0 / 4 + i));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  acc[4 * i] = fmaf(f, y[i].x, acc[4 * i]);
                  acc[4 * i + 1] = fmaf(f, y[i].y, acc[4 * i + 1]);
                  acc[4 * i + 2] = fmaf(f, y[i].z, acc[4 * i + 2]);
                  acc[4 * i + 3] = fmaf(f, y[i].w, acc[4 * i + 3]);
                }
              }
            put_rows(acc, winv, d0);
          }
          if (tid == 0) p.tickets[cf] = 0u;
        }
      }
      gk += n;
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  pdl_launch_dependents();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------------------------------------
// Two query tiles of 128 rows at once (a unit's first and second half of its tokens) against
// the same key tiles: head sizes 64 and 128, where both accumulators fit in tensor memory.
//
// The chain of one tile -- S, softmax, P V -- leaves the tensor cores idle during the softmax
// and the exponential units idle during the products, and its waits are exposed.  With two
// independent chains half a period apart, one's softmax runs during the other's products; the
// key and value tiles are fetched once for 256 rows, and so is every fixed cost of a unit.
// A softmax thread has a whole row, whose 128 logits stay in registers from one load of tensor
// memory to the store of P: a load of 32 columns takes some 500 cycles while eight warps load, and
// a second pass over S cost more than what was done with it.  Tensor memory: S of half x at
// 128 x, P(k) over the first 64 columns of S(k) once they are read, O at 256 + D x.  S(k + 1)
// overwrites P(k), so it is issued after O += P(k) V(k) has completed; meanwhile the other
// half's products run.  That also means O may be rescaled as soon as S(k + 1) is there.
//
// Warps: 0-3 softmax of the first half, 4-7 of the second, 8 MMA issue, 9 loads of Q and K,
// 10 loads of V, 11 idle (whole warpgroups).  A half skips the key tiles that none of its rows
// attends.  The value rows of a tile are checked (see above) by the first half that uses the tile.
// Measured: 8 chunks of 512 tokens with a window of 4096 in 318 us (865 TFLOP/s), a prompt of 8192
// in 0.54 ms (1015 TFLOP/s, 53% of the measured bf16 rate); tensor pipe 39% busy, issue slots
// 31%, exponential unit 20%, DRAM 43%: the chain of a half is the limit, no unit.  The 128 logits do
// not fit beside what else a thread holds: 320 bytes of spill stores and 424 of loads (queries in two
// parts 196 and 272, head size 64 148 and 212, 100 and 140).

namespace ppre {

template <int D, bool SPLIT>
struct Lay2 {
  static constexpr int HALVES = D / 64;
  static constexpr int kTile = HALVES * kHalf;
  // K tiles, and V tiles.  One of each: K(k + 1) is loaded only behind both halves' S(k)
  static constexpr int kSt = D == 64 ? 4 : SPLIT ? 1 : 2;
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + (SPLIT ? 4 : 2) * kTile;  // Q of both halves, and what bf16 left of them
  static constexpr int kV = kK + kSt * kTile;
  static constexpr int kStage = kV + kSt * kTile;  // 32 rows x 32 columns of output per softmax warp
  static constexpr int kSched = kStage + 8 * 2048;
  static constexpr int kOdd = kSched + (int)((sizeof(PSched) + 15) / 16 * 16);  // uint32 [buffer][kind][8]
  static constexpr int kMisc = kOdd + kOddBufs * 16 * 4;
  static constexpr int kBars = kMisc + 16;
  static constexpr int kWalk = kBars + 40 * 8;  // of a cache in 4 bits: the walkers of the warps that write its tiles
  static constexpr int kAlloc = kWalk + (i4t::kWarps + 1) * (int)sizeof(i4t::Walker) + 1024;  // and room to align the base
  static_assert(kAlloc <= 232448, "shared memory");
};

// What each half of a unit does in this CTA: rows, and key tiles [a, b) relative to the unit's.
struct Halves {
  int rows[2], a[2], b[2];
};
__device__ __forceinline__ Halves halves_of(const PagedParams &p, const PUnit &u) {
  Halves h;
  const int t1 = p.tpt / 2;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int s0 = x * t1, s1 = min(u.ntok, s0 + t1);
    h.rows[x] = s1 > s0 ? (s1 - s0) * p.group : 0;
    const long long j = p.W > 0 ? u.qpos + s0 - p.W + 1 : 0;
    h.a[x] = max(u.k0, (int)((j > 0 ? j : 0) / kKeys) - u.kt);
    h.b[x] = s1 > s0 ? min(u.k1, (int)((u.qpos + s1 - 1) / kKeys) + 1 - u.kt) : h.a[x];
    if (h.b[x] < h.a[x]) h.b[x] = h.a[x];
  }
  return h;
}

}  // namespace ppre

// 384 threads launched with 168 registers; the two softmax warpgroups take 208 and the third gives
// back to 88: 256 x 208 + 128 x 88 = 384 x 168.
//
// P: PagedParams, or I4Params for a cache in 4 bits: then warps 9 to 15 write the tiles (gqaw_i4_tiles.cuh), and
// warp 9 loads Q; 512 threads with 128 registers, 2 x 128 x (200 + 56).
template <int D, bool SPLIT, typename P = PagedParams>
__global__ void __launch_bounds__(ppre::threads2<P>, 1)
    paged_prefill2_kernel(const P p, const __grid_constant__ PagedMaps maps) {
  using namespace ppre;
  using L = Lay2<D, SPLIT>;
  constexpr int QP = SPLIT ? 2 : 1;  // parts of the queries
  constexpr bool kI4 = std::is_same<P, I4Params>::value;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  PSched *sched = reinterpret_cast<PSched *>(smem + L::kSched);
  uint32_t *odd = reinterpret_cast<uint32_t *>(smem + L::kOdd);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc), *s_last = abort_flag + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMisc + 8);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBars);
  uint64_t *q_full = bars, *q_free = bars + 1, *mma_done = bars + 2;
  uint64_t *o_free = bars + 4, *s_full = bars + 6, *p_full = bars + 8, *pv_done = bars + 10;  // of each half
  uint64_t *k_full = bars + 12, *k_free = bars + 16, *v_full = bars + 20, *v_free = bars + 24;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    ptc::prefetch_map(&maps.q);
    if (!kI4) {
      ptc::prefetch_map(&maps.k);
      ptc::prefetch_map(&maps.v);
    }
    mbar_init(q_full, 1);
    mbar_init(q_free, 1);
    mbar_init(mma_done, 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&o_free[x], 4);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 4);
      mbar_init(&pv_done[x], 1);
    }
    for (int i = 0; i < L::kSt; ++i) {
      mbar_init(&k_full[i], kI4 ? i4t::kBatches<D> : 1);
      mbar_init(&k_free[i], 1);
      mbar_init(&v_full[i], kI4 ? i4t::kBatches<D> : 1);
      mbar_init(&v_free[i], 1);
    }
    mbar_fence_init();
    *abort_flag = 0;
    for (int i = 0; i < kOddBufs * 16; ++i) odd[i] = 0u;
  }
  // query rows past a half's tokens stay zero
  for (int e = tid; e < 2 * QP * L::kTile / 16; e += threads2<P>) reinterpret_cast<uint4 *>(smem + L::kQ)[e] = make_uint4(0, 0, 0, 0);
  if (warp == 0) tc::tmem_alloc(tmem_slot, kTmemCols);
  tc::fence_proxy_async_smem();
  pdl_wait();
  const PShape shp = shape_of(p, kUnitCost);
  sched_build<kKeys>(p, shp, sched);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int g = p.group, t1 = p.tpt / 2;

  if (warp >= kMmaWarp2) {
    if constexpr (kI4)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (kI4 ? warp != kMmaWarp2 : warp == kKWarp2 || warp == kVWarp2) {
      if constexpr (kI4) {
        // ---------------------------------------------------------- tiles out of codes
        i4t::Walker *const walkers = reinterpret_cast<i4t::Walker *>(smem + L::kWalk);
        i4t::Walker *const qw = walkers + i4t::kWarps;  // of the queries, lane 0 of warp 9 alone
        if (warp == kKWarp2 && lane == 0) qw->walk = PWalk<kKeys>(shp, sched);
        int qi = 0;
        // the queries of the next unit, once the last S product with the previous ones is done
        auto queries = [&]() -> bool {
          if (!__all_sync(0xffffffffu, qi == 0 || mbar_wait(q_free, (qi - 1) & 1))) return false;
          if (lane == 0 && qw->walk.next(shp, qw->u)) {
            const PUnit &u = qw->u;
            const uint64_t qpol = policy_evict_first();
            const int parts = u.ntok > t1 ? 2 : 1;
            mbar_arrive_expect_tx(q_full, (uint32_t)(parts * QP * L::HALVES * g * t1 * 128));
            for (int x = 0; x < parts; ++x)
              for (int h = 0; h < QP * L::HALVES; ++h)
                tc::tma_load_3d(smem + L::kQ + x * QP * L::kTile + h * kHalf, h < L::HALVES ? &maps.q : &maps.ql,
                                h % L::HALVES * 64, u.hu * g, u.row0 + x * t1, q_full, qpol);
          }
          __syncwarp();
          ++qi;
          return true;
        };
        const i4t::Rings rings{smem + L::kK, smem + L::kV, k_full, k_free, v_full, v_free};
        const bool fine = i4t::convert<D, L::kSt, kHalf>(p, shp, sched, walkers + (warp - kKWarp2), rings, abort_flag, warp - kKWarp2,
                                                               lane, queries);
        if (lane == 0) {
          if (!fine) {
            pflag(p, GQAW_DEV_TIMEOUT);
            *abort_flag = 1;
          }
          // no copy may still be landing in shared memory when the CTA exits
          if (qi > 0 && !mbar_wait(q_full, (qi - 1) & 1)) pflag(p, GQAW_DEV_TIMEOUT);
        }
      } else {
        // ------------------------------------------------------------ loads (whole warp)
        const bool value = warp == kVWarp2;
        const uint64_t pol = tc::policy_evict_normal(), qpol = policy_evict_first();
        uint64_t *full = value ? v_full : k_full, *empty = value ? v_free : k_free;
        unsigned char *ring = smem + (value ? L::kV : L::kK);
        const CUtensorMap *map = value ? &maps.v : &maps.k;
        PWalk<kKeys> w(shp, sched);
        PUnit u;
        ptc::Boxes bx;
        int gk = 0, qi = 0;
        bool fine = true;
        while (fine && w.next(shp, u)) {
          bx.unit(p, u);
          bx.look_up(p, u.kt + u.k0, lane);
          for (int k = u.k0; k < u.k1; ++k, ++gk) {
            const uint32_t mask = bx.valid(p, u.kt + k, lane);
            const ptc::Boxes cur = bx;
            if (k + 1 < u.k1) bx.look_up(p, u.kt + k + 1, lane);
            const int st = gk % L::kSt;
            if (gk >= L::kSt) fine = mbar_wait(&empty[st], ((gk / L::kSt) & 1) ^ 1);
            fine = __all_sync(0xffffffffu, fine && !*abort_flag);
            if (!fine) break;
            if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)(__popc(mask) * bx.rows * 128 * L::HALVES));
            __syncwarp();
            cur.load<L::HALVES>(map, ring + st * L::kTile, &full[st], pol, mask, lane);
            // the queries after the unit's first K tile, once the last S product with the previous
            // ones is done
            if (k == u.k0 && !value) {
              if (qi > 0) fine = mbar_wait(q_free, (qi - 1) & 1);
              fine = __all_sync(0xffffffffu, fine);
              if (!fine) {
                ++gk;
                break;
              }
              if (lane == 0) {
                const int parts = u.ntok > t1 ? 2 : 1;
                mbar_arrive_expect_tx(q_full, (uint32_t)(parts * QP * L::HALVES * g * t1 * 128));
                for (int x = 0; x < parts; ++x)
                  for (int h = 0; h < QP * L::HALVES; ++h)
                    tc::tma_load_3d(smem + L::kQ + x * QP * L::kTile + h * kHalf, h < L::HALVES ? &maps.q : &maps.ql,
                                    h % L::HALVES * 64, u.hu * g, u.row0 + x * t1, q_full, qpol);
              }
              ++qi;
            }
          }
        }
        if (lane == 0) {
          if (!fine) {
            pflag(p, GQAW_DEV_TIMEOUT);
            *abort_flag = 1;
          }
          // no copy may still be landing in shared memory when the CTA exits
          for (int j = gk > L::kSt ? gk - L::kSt : 0; j < gk; ++j)
            if (!mbar_wait(&full[j % L::kSt], (j / L::kSt) & 1)) pflag(p, GQAW_DEV_TIMEOUT);
          if (!value && qi > 0 && !mbar_wait(q_full, (qi - 1) & 1)) pflag(p, GQAW_DEV_TIMEOUT);
        }
      }
    } else if (warp == kMmaWarp2) {
      // ------------------------------------------------------------ MMA issue
      // The whole warp runs the loop and one elected thread issues: descriptors and addresses are
      // then uniform values, which is what the instruction takes.
      {
        constexpr uint32_t kIdescQK = tc::idesc_bf16_f32(kRows, kKeys, 0, 0);
        constexpr uint32_t kIdescPV = tc::idesc_bf16_f32(kRows, D, 0, 1);
        const uint64_t dq = tc::smem_desc_sw128(smem + L::kQ, 16, 1024);
        const uint64_t dk = tc::smem_desc_sw128(smem + L::kK, 16, 1024);
        const uint64_t dv = tc::smem_desc_sw128(smem + L::kV, kHalf, 1024);
        PWalk<kKeys> w(shp, sched);
        PUnit u;
        Halves hv{};
        int gk = 0, qi = 0, pvs[2] = {0, 0}, outs[2] = {0, 0};  // products O += P V issued, units finished
        // S of half x for tile k of the unit, once the half's last P V has completed
        auto s_product = [&](int x, int k) -> bool {
          const int kt = gk + k - u.k0, st = kt % L::kSt;
          if (!warp_wait(&k_full[st], (kt / L::kSt) & 1)) return false;
          if (pvs[x] > 0 && !warp_wait(&pv_done[x], (pvs[x] - 1) & 1)) return false;
          tc::fence_after_sync();
          const uint64_t a0 = dq + (uint64_t)((x * QP * L::kTile) >> 4), b0 = dk + (uint64_t)((st * L::kTile) >> 4);
          const bool second = hv.a[1] <= k && k < hv.b[1];
          if (elect_one()) {
#pragma unroll 1
            for (int q = 0; q < QP; ++q) {  // not unrolled: the descriptors of 16 products would spill
              const uint64_t aq = a0 + (uint64_t)((q * L::kTile) >> 4);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t off = (uint64_t)(((kk / 4) * kHalf + (kk % 4) * 32) >> 4);
                tc::mma_bf16_ss(tmem + x * kKeys, aq + off, b0 + off, kIdescQK, q + kk > 0);
              }
            }
            tc::mma_commit(&s_full[x]);
            if (x == 1 || !second) tc::mma_commit(&k_free[st]);
            // the unit's last S product: the second half's, if it has any tile here
            if (k + 1 == hv.b[x] && x == (hv.a[1] < hv.b[1] ? 1 : 0)) tc::mma_commit(q_free);
          }
          __syncwarp();
          return true;
        };
        bool fine = true;
        while (fine && __all_sync(0xffffffffu, !*abort_flag) && w.next(shp, u)) {
          hv = halves_of(p, u);
          fine = warp_wait(q_full, qi & 1);
          for (int x = 0; x < 2 && fine; ++x)
            if (hv.a[x] == u.k0 && hv.a[x] < hv.b[x]) fine = s_product(x, u.k0);
          for (int k = u.k0; k < u.k1 && fine; ++k) {
            const int kt = gk + k - u.k0, st = kt % L::kSt;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (!fine) break;
              if (hv.a[x] <= k && k < hv.b[x]) {
                const bool first = k == hv.a[x];
                fine = warp_wait(&p_full[x], pvs[x] & 1) &&
                       // the first P V of a unit overwrites O: the softmax has read the last unit's
                       (!first || outs[x] == 0 || warp_wait(&o_free[x], (outs[x] - 1) & 1)) &&
                       warp_wait(&v_full[st], (kt / L::kSt) & 1);
                if (!fine) break;
                tc::fence_after_sync();
                const uint64_t b0 = dv + (uint64_t)((st * L::kTile) >> 4);
                const bool second = hv.a[1] <= k && k < hv.b[1];
                if (elect_one()) {
#pragma unroll
                  for (int kk = 0; kk < kKeys / 16; ++kk)
                    tc::mma_bf16_ts(tmem + 256 + x * D, tmem + x * kKeys + kk * 8, b0 + (uint64_t)((kk * 16 * 128) >> 4), kIdescPV,
                                    !first || kk > 0);
                  tc::mma_commit(&pv_done[x]);
                  if (x == 1 || !second) tc::mma_commit(&v_free[st]);
                }
                __syncwarp();
                ++pvs[x];
                if (k + 1 < hv.b[x]) fine = s_product(x, k + 1);
              } else if (k + 1 == hv.a[x] && hv.a[x] < hv.b[x]) {
                fine = s_product(x, k + 1);
              }
            }
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) outs[x] += hv.a[x] < hv.b[x] ? 1 : 0;
          gk += u.k1 - u.k0;
          ++qi;
        }
        if (!fine) {
          if (lane == 0) pflag(p, GQAW_DEV_TIMEOUT);
          *abort_flag = 1;
        }
        if (elect_one()) tc::mma_commit(mma_done);  // every MMA issued has completed before TMEM is released
        if (!warp_wait(mma_done, 0)) if (lane == 0) pflag(p, GQAW_DEV_TIMEOUT);
      }
    }
  } else {
    if constexpr (kI4)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ------------------------------------------------------------ softmax (warps 0-7)
    const int wq = warp & 3, x = warp >> 2;  // TMEM lane quarter, half
    const int r = wq * 32 + lane;            // row of the half = TMEM lane
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t ts = tmem + x * kKeys + lane_off, to = tmem + 256 + x * D + lane_off;
    const bool plain = p.capmul == 0.f, fixed = !plain && p.capmul <= 64.f;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out);
    PWalk<kKeys> w(shp, sched);
    PUnit u;
    int gk = 0, cnt = 0, odd_at = 0;  // key tiles of the CTA's units so far, and of this half; buffer of odd bits
    // A warp that gives up a tile (an expired wait, an abort elsewhere) still runs every unit's
    // epilogue: the softmax warps meet at its barriers.
    while (w.next(shp, u)) {
      const Halves hv = halves_of(p, u);
      const int rows = hv.rows[x], a = hv.a[x], b = hv.b[x];
      const bool idle = wq * 32 >= rows;        // no row of this warp exists
      const bool row_ok = r < rows;
      const int rr = row_ok ? r : max(rows - 1, 0);  // rows past the half's follow its last one
      const int tok = x * t1 + rr / g, h = u.hu * g + rr % g;
      const long long at = u.qpos + tok;        // absolute position of the row's token
      const long long rlo = p.W > 0 && at - p.W + 1 > 0 ? at - p.W + 1 : 0;
      const long long jlo = p.W > 0 && u.qpos - p.W + 1 > 0 ? u.qpos - p.W + 1 : 0, jhi = u.qpos + u.ntok;
      const long long unit0 = (long long)u.kt * kKeys;
      // some key of this CTA's tiles is attended by some of the unit's tokens only
      const bool has_part = u.ntok > 1 && (unit0 + (long long)u.k1 * kKeys - 1 > u.qpos ||
                                           (p.W > 0 && unit0 + (long long)u.k0 * kKeys < jhi - p.W));
      float m_run = fixed ? 0.f : -INFINITY, l_run = 0.f;
      bool dead = false;
      for (int k = a; k < b; ++k, ++cnt) {
        const long long j0 = unit0 + (long long)k * kKeys;
        if (!__all_sync(0xffffffffu, !*abort_flag && mbar_wait(&s_full[x], cnt & 1))) {
          if (lane == 0) pflag(p, GQAW_DEV_TIMEOUT);
          *abort_flag = 1;
          dead = true;
          break;
        }
        tc::fence_after_sync();
        if (!idle) {
          const int c_lo = (int)min(max(rlo - j0, 0LL), (long long)kKeys), c_hi = (int)min(max(at + 1 - j0, 0LL), (long long)kKeys);
          float v[128];  // the row's logits stay here from one load to the store of P
          tmem_ld128(ts, v);
          if (!plain) {  // cap tanh(z) = cap - 2 cap / (e^(2z) + 1)
            const float z2 = 2.8853900817779268f * p.qscale, c2 = -2.f * p.capmul;
#pragma unroll
            for (int c = 0; c < 128; ++c) {
              float q;
              asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(1.f + fast_exp2(v[c] * z2)));
              v[c] = fmaf(c2, q, p.capmul);
            }
          }
          if (!__all_sync(0xffffffffu, c_lo == 0 && c_hi == kKeys)) {
#pragma unroll
            for (int c32 = 0; c32 < 4; ++c32) {
              const uint32_t m = col_mask(min(max(c_lo - c32 * 32, 0), 32), min(max(c_hi - c32 * 32, 0), 32));
#pragma unroll
              for (int c = 0; c < 32; ++c) v[c32 * 32 + c] = (m >> c) & 1u ? v[c32 * 32 + c] : -INFINITY;
            }
          }
          const float zs = plain ? p.qscale : 1.f;  // > 0
          float alpha = 1.f;
          if (!fixed) {
            float m4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
            for (int c = 4; c < 124; c += 8) {
#pragma unroll
              for (int i = 0; i < 4; ++i) m4[i] = max3(m4[i], v[c + 2 * i], v[c + 2 * i + 1]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) m4[i] = fmaxf(m4[i], v[124 + i]);
            const float mt = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]) * zs;
            // the reference moves only when exceeded by more than 2^8; O holds the tiles before
            // this one (S was issued after their last product had completed)
            if (mt > m_run + kRescaleLog2) {
              alpha = m_run == -INFINITY ? 0.f : fast_exp2(m_run - mt);
              m_run = mt;
            }
            if (k > a && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                float o[16];
                tc::tmem_ld16(to + c, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= alpha;
                tc::tmem_st16(to + c, o);
              }
            }
          }
          const float base = m_run == -INFINITY ? 0.f : m_run;
          l_run = l_run * alpha + ((put_p(v, ts, zs, base) + put_p(v + 32, ts + 16, zs, base)) +
                                   (put_p(v + 64, ts + 32, zs, base) + put_p(v + 96, ts + 48, zs, base)));
        }
        // ---- value rows of the tile, by the first half that uses it: key t = row r
        const bool ends = j0 < jlo || j0 + kKeys > jhi;
        const bool part = u.ntok > 1 && (j0 + kKeys - 1 > u.qpos || (p.W > 0 && j0 < jhi - p.W));
        if ((ends || part) && (x == 0 || k < hv.a[0] || k >= hv.b[0])) {
          const int vt = gk + k - u.k0, st = vt % L::kSt;
          if (!mbar_wait(&v_full[st], (vt / L::kSt) & 1)) *abort_flag = 1;
          const long long j = j0 + r;
          unsigned char *row = smem + L::kV + st * L::kTile + r * 128;
          constexpr int C = D / 8;  // 16-byte parts of a row
          bool zero = j < jlo || j >= jhi;
          if (!zero && part && (j > u.qpos || (p.W > 0 && j < jhi - p.W))) {
            for (int c = 0; c < C; ++c) {
              const uint4 v = *reinterpret_cast<const uint4 *>(row + (c / 8) * kHalf + (((c & 7) ^ (r & 7)) << 4));
              zero |= odd_pair(v.x) || odd_pair(v.y) || odd_pair(v.z) || odd_pair(v.w);
            }
            // a unit has up to 256 tokens: bits of keys after its first token, or of those before
            // its last token's window
            if (zero) {
              const int kind = j > u.qpos ? 0 : 1, i = (int)(j - (kind ? jlo : u.qpos));
              atomicOr(&odd[odd_at * 16 + kind * 8 + i / 32], 1u << (i & 31));
            }
          }
          if (zero)
            for (int c = 0; c < C; ++c)
              *reinterpret_cast<uint4 *>(row + (c / 8) * kHalf + (((c & 7) ^ (r & 7)) << 4)) = make_uint4(0, 0, 0, 0);
          tc::fence_proxy_async_smem();
        }
        __syncwarp();
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
      }
      // the half's last O += P V
      bool have = a < b && !dead;
      if (have && !__all_sync(0xffffffffu, mbar_wait(&pv_done[x], (cnt - 1) & 1))) {
        if (lane == 0) pflag(p, GQAW_DEV_TIMEOUT);
        *abort_flag = 1;
        have = false;
      }
      tc::fence_after_sync();
      bool any_odd = false;
      const volatile uint32_t *mine = odd + odd_at * 16;
      if (has_part) {  // both halves' checks are in
        named_barrier(kSoftBar, kSoft2);
        for (int i = 0; i < 16; ++i) any_odd |= mine[i] != 0u;
        if (tid < 16) odd[(odd_at + kOddBufs - 1) % kOddBufs * 16 + tid] = 0u;
      }

      // ---- the row's D columns of O, and (m, l), 32 at a time
      const bool cut = u.k0 > 0 || u.k1 < u.nt;
      const int cta = blockIdx.x, cf = cut ? w.owner(u.g0) : cta, cl = cut ? w.owner(u.g0 + u.nt - 1) : cta;
      float4 *const parts = reinterpret_cast<float4 *>(p.partials);
      // partial block of a CTA: D / 4 float4 columns of O and one of (m, l), 256 rows each
      auto part_at = [&](int c, int c4) {
        return parts + (((long long)c * 2 + (c == cf ? 1 : 0)) * (D / 4 + 1) + c4) * (2 * kRows) + x * kRows + r;
      };
      const float inv = cut ? 1.f : sink_reciprocal(l_run, m_run, paged_sink_log2(p, h));
      // 32 columns of the warp's 32 rows to memory, by way of shared memory: 4 lanes write the 64
      // bytes of a row (a lane writing its own row would touch 32 lines with every store)
      const long long orow = (u.row0 + tok) * p.os + (long long)h * D;  // of this lane's row
      auto put_rows = [&](const float (&v)[32], float f, int d0) {
        unsigned char *st = smem + L::kStage + warp * 2048;
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint4 y;
          y.x = tc::pack_bf16x2(v[8 * c] * f, v[8 * c + 1] * f);
          y.y = tc::pack_bf16x2(v[8 * c + 2] * f, v[8 * c + 3] * f);
          y.z = tc::pack_bf16x2(v[8 * c + 4] * f, v[8 * c + 5] * f);
          y.w = tc::pack_bf16x2(v[8 * c + 6] * f, v[8 * c + 7] * f);
          *reinterpret_cast<uint4 *>(st + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) = y;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = i * 8 + (lane >> 2), c = lane & 3;
          const long long at_ = __shfl_sync(0xffffffffu, orow, row);
          const uint4 y = *reinterpret_cast<const uint4 *>(st + row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
          if (wq * 32 + row < rows) *reinterpret_cast<uint4 *>(out + at_ + d0 + c * 8) = y;
        }
      };
      if (!idle || a < b) {
#pragma unroll 1
        for (int c32 = 0; c32 < D / 32; ++c32) {
          float v[32];
          const int d0 = c32 * 32;
          __syncwarp();
          if (have) {
            tc::tmem_ld32(to + d0, v);
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = 0.f;
          }
          if constexpr (kI4) {  // the columns as the value tiles hold the dimensions
            float y[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) y[i4t::value_column(c)] = v[c];
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = y[c];
          }
          if (c32 == D / 32 - 1 && a < b) {  // O has left tensor memory: the next unit may overwrite it
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_free[x]);
          }
          if (any_odd && row_ok)  // their weights anew, from the cache, for the rows that attend them
            for (int i = 0; i < 16; ++i)
              for (uint32_t bits = mine[i]; bits; bits &= bits - 1u) {
                const long long j = (i < 8 ? u.qpos : jlo) + (i & 7) * 32 + __ffs((int)bits) - 1;
                if constexpr (kI4) {
                  const I4Place place = j >= rlo && j <= at ? i4_place(p, u.b, j) : I4Place{-1, 0};
                  if (place.page < 0) continue;
                  const long long q_at = (u.row0 + tok) * p.qs + (long long)h * D;
                  float z = 0.f;
#pragma unroll 1
                  for (int d = 0; d < D; ++d) {
                    float y = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.q)[q_at + d]);
                    if (SPLIT) y += __bfloat162float(static_cast<const __nv_bfloat16 *>(p.qlo)[q_at + d]);
                    z = fmaf(y, i4t::element(p, false, place, u.hu, d), z);
                  }
                  z *= p.qscale;
                  if (!plain) z = p.capmul * ptc::fast_tanh(z);
                  const float pr = fast_exp2(z - m_run);
#pragma unroll
                  for (int c = 0; c < 32; ++c) v[c] = fmaf(pr, i4t::element(p, true, place, u.hu, d0 + c), v[c]);
                } else {
                  const long long off = j >= rlo && j <= at ? cache_row(p, u.b, u.hu, (int)j) : -1;
                  if (off < 0) continue;
                  const __nv_bfloat16 *kr = static_cast<const __nv_bfloat16 *>(p.kp) + off;
                  const __nv_bfloat16 *vr = static_cast<const __nv_bfloat16 *>(p.vp) + off + d0;
                  const long long q_at = (u.row0 + tok) * p.qs + (long long)h * D;
                  const __nv_bfloat16 *qr = static_cast<const __nv_bfloat16 *>(p.q) + q_at;
                  const __nv_bfloat16 *ql = static_cast<const __nv_bfloat16 *>(p.qlo) + q_at;
                  float z = 0.f;
#pragma unroll 4
                  for (int d = 0; d < D; ++d) {
                    float x = __bfloat162float(qr[d]);
                    if (SPLIT) x += __bfloat162float(ql[d]);
                    z = fmaf(x, __bfloat162float(kr[d]), z);
                  }
                  z *= p.qscale;
                  if (!plain) z = p.capmul * ptc::fast_tanh(z);
                  const float pr = fast_exp2(z - m_run);
#pragma unroll
                  for (int c = 0; c < 32; ++c) v[c] = fmaf(pr, __bfloat162float(vr[c]), v[c]);
                }
              }
          if (cut) {
            if (row_ok)
#pragma unroll
              for (int c = 0; c < 32; c += 4) *part_at(cta, (d0 + c) / 4) = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
          } else {
            put_rows(v, inv, d0);
          }
        }
      }
      if (has_part) odd_at = (odd_at + 1) % kOddBufs;
      if (cut) {
        if (row_ok) *part_at(cta, D / 4) = make_float4(have ? m_run : -INFINITY, have ? l_run : 0.f, 0.f, 0.f);
        named_barrier(kSoftBar, kSoft2);
        if (tid == 0) {
          __threadfence();
          *s_last = atomicAdd(&p.tickets[cf], 1u) == (unsigned)(cl - cf);
        }
        named_barrier(kSoftBar, kSoft2);
        if (*s_last) {
          __threadfence();
          float M = -INFINITY, S = 0.f;
#pragma unroll 4
          for (int c = cf; c <= cl; ++c) M = fmaxf(M, row_ok ? __ldcg(part_at(c, D / 4)).x : 0.f);
          const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll 4
          for (int c = cf; c <= cl; ++c) {
            const float4 ml = row_ok ? __ldcg(part_at(c, D / 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
            S = fmaf(fast_exp2(ml.x - ref), ml.y, S);
          }
          const float winv = sink_reciprocal(S, M, paged_sink_log2(p, h));
#pragma unroll 1
          for (int d0 = 0; d0 < D; d0 += 32) {
            float acc[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) acc[c] = 0.f;
            if (row_ok)
              for (int c = cf; c <= cl; ++c) {
                const float f = fast_exp2(__ldcg(part_at(c, D / 4)).x - ref);
                float4 y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = __ldcg(part_at(c, d0 / 4 + i));
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  acc[4 * i] = fmaf(f, y[i].x, acc[4 * i]);
                  acc[4 * i + 1] = fmaf(f, y[i].y, acc[4 * i + 1]);
                  acc[4 * i + 2] = fmaf(f, y[i].z, acc[4 * i + 2]);
                  acc[4 * i + 3] = fmaf(f, y[i].w, acc[4 * i + 3]);
                }
              }
            put_rows(acc, winv, d0);
          }
          if (tid == 0) p.tickets[cf] = 0u;
        }
      }
      gk += u.k1 - u.k0;
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  pdl_launch_dependents();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

constexpr int kPrefillDevices = 64;

template <typename K, typename P>
cudaError_t launch_prefill(K kernel, std::atomic<bool> *ready, int threads, int smem, const P &p, const PagedMaps &maps,
                           int grid, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kPrefillDevices || !ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < kPrefillDevices) ready[dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see pdl_wait()
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, p, maps);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace gqaw
