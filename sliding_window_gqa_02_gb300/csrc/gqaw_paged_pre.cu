// gqaw_paged_pre.cu -- paged attention of many query rows per kv head (prompt chunks, and
// batches that mix them with decoding sequences) on the 5th-generation tensor cores, bf16,
// head sizes 64, 128 and 256.
//
// A query tile is 128 rows, row = token * group + head, of one sequence and kv head; a key
// tile is 128 positions, fetched through the page table (gqaw_paged_tc.cuh):
//   S = Q K^T      M = 128 rows, N = 128 keys, K = D; both operands in shared memory
//   O += P V       M = 128 rows, N = D, K = 128 keys; P (bf16) in tensor memory
// Bound: the exponentials and the tensor cores about alike (4 D multiply-adds and one 2^x
// per row and key), so both run all the time: S(k + 1) is issued while the softmax works on
// S(k), and O += P(k) V(k) while it works on S(k + 1).
//
// Softmax: two threads per row (TMEM lane), half the keys each.  The reference maximum moves
// only when exceeded by more than 2^8, so O is rarely rescaled; in a tile that every row of
// the warp attends whole, P is computed against the running reference in the same pass as the
// tile's maximum, and the factor is owed to O if it has to move after all.  Sums are fp32 of
// the unrounded weights; P is rounded to bf16 for its product (2^-9 relative, the size of the
// output's own rounding).  Warps without rows (a decoding sequence among chunks has `group`
// rows of the 128) only keep the barriers turning.
//
// Tensor memory (512 columns), head sizes 64 and 128: S in two buffers [0, 256), O from 256,
// P in two buffers [384, 512).  Head size 256 needs 256 columns for O: S has one buffer
// [0, 128), P two [128, 256), and S(k + 1) waits for P(k).
//
// Warps: 0-7 softmax, 8 MMA issue, 9 loads of Q and K, 10 loads of V (one lane per box).
// Schedule, splits and merges: gqaw_paged.cuh.  A cut unit's partial rows go out column-major
// so that a warp's 32 rows are contiguous.
//
// Keys that some rows attend and others do not lie in the tiles along the diagonal and the
// window's edge.  There the softmax threads zero the value rows that nobody attends, and look
// for rows that are not finite among those that only some attend (0 x inf is NaN): these are
// zeroed too, and added at the unit's end to the rows that attend them, from global memory.
//
// Every wait is bounded; one that expires flags GQAW_DEV_TIMEOUT and the CTA winds down.
#include <atomic>

#include "gqaw_paged_tc.cuh"

namespace gqaw {

namespace ppre {

using ptc::kHalf;
using ptc::kKeys;
using ptc::fast_exp2;
constexpr int kRows = 128;
constexpr int kHalfKeys = 64;
constexpr int kMmaWarp = 8, kKWarp = 9, kVWarp = 10;
constexpr int kThreads = 352;
constexpr uint32_t kTmemCols = 512;
constexpr int kUnitCost = 3;   // see gqaw_paged_sched.cuh
constexpr float kRescaleLog2 = 8.0f, kDangerLog2 = 16.0f;  // log2 units
constexpr int kSoftBar = 5;    // named barrier of the 8 softmax warps (1-4: pairs of warps)

template <int D>
struct Lay {
  static constexpr int HALVES = D / 64;
  static constexpr int kTile = HALVES * kHalf;
  static constexpr int kKSt = D == 64 ? 4 : D == 128 ? 3 : 1;
  static constexpr int kVSt = D == 64 ? 4 : D == 128 ? 2 : 1;
  static constexpr int kSBuf = D == 256 ? 1 : 2;
  static constexpr uint32_t kTmemP = D == 256 ? 128 : 384, kTmemO = 256;
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + kTile;
  static constexpr int kV = kK + kKSt * kTile;
  static constexpr int kSched = kV + kVSt * kTile;
  static constexpr int kXch = kSched + (int)((sizeof(PSched) + 15) / 16 * 16);  // float [3][2][128]
  // keys attended by some rows only whose values are not finite, as bits: uint32
  // [unit & 1][column half][0: after the first token, 1: before the last token's window][4]
  static constexpr int kOdd = kXch + 3 * 2 * kRows * 4;
  static constexpr int kMisc = kOdd + 2 * 16 * 4;  // flags
  static constexpr int kStage = (kMisc + 128 + 255) / 256 * 256;  // 32 rows x 32 columns of output per softmax warp
  static constexpr int kBars = kStage + 8 * 2048;
  static constexpr int kAlloc = kBars + 32 * 8 + 1024;  // and room to align the base
  static_assert(kAlloc <= 232448, "shared memory");
};

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

// Bit c set when column 32 * c32 + c lies in [c_lo, c_hi).
__device__ __forceinline__ uint32_t chunk_mask(int c32, int c_lo, int c_hi) {
  const int lo = min(max(c_lo - c32 * 32, 0), 32), hi = min(max(c_hi - c32 * 32, 0), 32);
  const uint32_t below_hi = hi >= 32 ? 0xffffffffu : (1u << hi) - 1u;
  const uint32_t below_lo = lo >= 32 ? 0xffffffffu : (1u << lo) - 1u;
  return below_hi & ~below_lo;
}

// The largest logit of this thread's row among its 64 columns (kMasked: of [c_lo, c_hi)).
template <bool kMasked>
__device__ __forceinline__ float tile_max(uint32_t ts, int c_lo, int c_hi) {
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int c32 = 0; c32 < kHalfKeys / 32; ++c32) {
    float v[32];
    tc::tmem_ld32(ts + c32 * 32, v);
    if (kMasked) {
      const uint32_t m = chunk_mask(c32, c_lo, c_hi);
#pragma unroll
      for (int c = 0; c < 32; ++c) mx[c & 3] = fmaxf(mx[c & 3], (m >> c) & 1u ? v[c] : -INFINITY);
    } else {
#pragma unroll
      for (int c = 0; c < 32; c += 2) mx[(c / 2) & 3] = max3(mx[(c / 2) & 3], v[c], v[c + 1]);
    }
  }
  return max3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
}

// P = 2^(z zs - base) of this thread's 64 logits at ts, as bf16 pairs into 32 columns at tp;
// returns the sum of the fp32 values.  With kMax the largest raw logit is left in *mx.
template <bool kMasked, bool kMax = false>
__device__ __forceinline__ float tile_p(uint32_t ts, uint32_t tp, int c_lo, int c_hi, float zs, float base,
                                        float *mx = nullptr) {
  if (kMasked) {
    float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c32 = 0; c32 < kHalfKeys / 32; ++c32) {
      float v[32];
      tc::tmem_ld32(ts + c32 * 32, v);
      const uint32_t m = chunk_mask(c32, c_lo, c_hi);
      uint32_t pk[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const float a0 = (m >> (2 * c)) & 1u ? fast_exp2(fmaf(v[2 * c], zs, -base)) : 0.f;
        const float a1 = (m >> (2 * c + 1)) & 1u ? fast_exp2(fmaf(v[2 * c + 1], zs, -base)) : 0.f;
        ls[c & 3] += a0 + a1;
        pk[c] = tc::pack_bf16x2(a0, a1);
      }
      tc::tmem_st16_async(tp + c32 * 16, pk);
    }
    return (ls[0] + ls[1]) + (ls[2] + ls[3]);
  }
  const uint64_t zs2 = pack2(zs, zs), nb2 = pack2(-base, -base);
  uint64_t acc[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
  float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int c32 = 0; c32 < kHalfKeys / 32; ++c32) {
    float v[32];
    tc::tmem_ld32(ts + c32 * 32, v);
    uint32_t pk[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      if (kMax) m4[c & 3] = max3(m4[c & 3], v[2 * c], v[2 * c + 1]);
      float x0, x1;
      unpack2(fma2(pack2(v[2 * c], v[2 * c + 1]), zs2, nb2), x0, x1);
      const float a0 = fast_exp2(x0), a1 = fast_exp2(x1);
      acc[c & 1] = add2(acc[c & 1], pack2(a0, a1));
      pk[c] = tc::pack_bf16x2(a0, a1);
    }
    tc::tmem_st16_async(tp + c32 * 16, pk);
  }
  if (kMax) *mx = max3(m4[0], m4[1], fmaxf(m4[2], m4[3]));
  float l0, l1, l2, l3;
  unpack2(acc[0], l0, l1);
  unpack2(acc[1], l2, l3);
  return (l0 + l1) + (l2 + l3);
}

// Capped logits against a fixed reference of 0: P = 2^(cap tanh(z zs)), |cap| <= 64, of this
// thread's 64 logits, as bf16 pairs into 32 columns at tp; returns their sum.
template <bool kMasked>
__device__ __forceinline__ float tile_p_cap(uint32_t ts, uint32_t tp, int c_lo, int c_hi, float zs, float cap) {
  // tanh(x) = 1 - 2 / (e^(2x) + 1), which saturates to the right limits and keeps a NaN
  const float z2 = 2.8853900817779268f * zs, c2 = -2.f * cap;
  float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c32 = 0; c32 < kHalfKeys / 32; ++c32) {
    float v[32];
    tc::tmem_ld32(ts + c32 * 32, v);
    const uint32_t m = kMasked ? chunk_mask(c32, c_lo, c_hi) : 0xffffffffu;
    uint32_t pk[16];
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      float r;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + fast_exp2(v[c] * z2)));
      v[c] = fast_exp2(fmaf(c2, r, cap));
      if (kMasked && !((m >> c) & 1u)) v[c] = 0.f;
      ls[c & 3] += v[c];
    }
#pragma unroll
    for (int c = 0; c < 16; ++c) pk[c] = tc::pack_bf16x2(v[2 * c], v[2 * c + 1]);
    tc::tmem_st16_async(tp + c32 * 16, pk);
  }
  return (ls[0] + ls[1]) + (ls[2] + ls[3]);
}

__device__ __forceinline__ bool odd_pair(uint32_t w) {
  return (w & 0x7f800000u) == 0x7f800000u || (w & 0x00007f80u) == 0x00007f80u;
}

}  // namespace ppre

template <int D>
__global__ void __launch_bounds__(ppre::kThreads, 1)
    paged_prefill_kernel(const PagedParams p, const __grid_constant__ PagedMaps maps) {
  using namespace ppre;
  using L = Lay<D>;
  constexpr int OC = D / 2;  // output columns of a softmax thread
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  PSched *sched = reinterpret_cast<PSched *>(smem + L::kSched);
  float *xch = reinterpret_cast<float *>(smem + L::kXch);  // [tile & 1 | 2 for the sums][column half][row]
  uint32_t *odd = reinterpret_cast<uint32_t *>(smem + L::kOdd);
  volatile int *misc = reinterpret_cast<volatile int *>(smem + L::kMisc);
  volatile int *abort_flag = misc;
  volatile int *s_last = misc + 1;
  volatile int *xok = misc + 8;                                               // [tile & 1][column half][lane quarter]
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMisc + 4 * 24);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBars);
  uint64_t *q_full = bars, *q_free = bars + 1, *o_free = bars + 2, *mma_done = bars + 3;
  uint64_t *s_full = bars + 4, *p_full = bars + 6, *pv_done = bars + 8;  // two each
  uint64_t *k_full = bars + 10, *k_free = bars + 14, *v_full = bars + 18, *v_free = bars + 22;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_free, 1);
    mbar_init(o_free, 8);
    mbar_init(mma_done, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 8);
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
    for (int i = 0; i < 32; ++i) odd[i] = 0u;
  }
  // query rows past tpt * group stay zero
  for (int e = tid; e < L::kTile / 16; e += kThreads) reinterpret_cast<uint4 *>(smem + L::kQ)[e] = make_uint4(0, 0, 0, 0);
  if (warp == 0) tc::tmem_alloc(tmem_slot, kTmemCols);
  tc::fence_proxy_async_smem();
  pdl_wait();
  const PShape shp = shape_of(p, kUnitCost);
  sched_build<kKeys>(p, shp, sched, kThreads);
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
            mbar_arrive_expect_tx(q_full, (uint32_t)(L::HALVES * g * p.tpt * 128));
            for (int h = 0; h < L::HALVES; ++h)
              tc::tma_load_3d(smem + L::kQ + h * kHalf, &maps.q, h * 64, u.hu * g, u.row0, q_full, qpol);
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
    if (lane == 0) {
      constexpr uint32_t kIdescQK = tc::idesc_bf16_f32(kRows, kKeys, 0, 0);
      constexpr uint32_t kIdescPV = tc::idesc_bf16_f32(kRows, D, 0, 1);
      const uint64_t dq = tc::smem_desc_sw128(smem + L::kQ, 16, 1024);
      const uint64_t dk = tc::smem_desc_sw128(smem + L::kK, 16, 1024);
      const uint64_t dv = tc::smem_desc_sw128(smem + L::kV, kHalf, 1024);
      auto s_product = [&](int gt) -> bool {  // S(gt) into its buffer; K(gt) is waited for
        const int st = gt % L::kKSt;
        if (!mbar_wait(&k_full[st], (gt / L::kKSt) & 1)) return false;
        tc::fence_after_sync();
        const uint64_t b0 = dk + (uint64_t)((st * L::kTile) >> 4);
        const uint32_t ds = tmem + (gt % L::kSBuf) * kKeys;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = (uint64_t)(((kk / 4) * kHalf + (kk % 4) * 32) >> 4);
          tc::mma_bf16_ss(ds, dq + off, b0 + off, kIdescQK, kk > 0);
        }
        tc::mma_commit(&s_full[gt & 1]);
        tc::mma_commit(&k_free[st]);
        return true;
      };
      auto pv_product = [&](int gt, bool acc) -> bool {  // P(gt) is waited for by the caller
        const int st = gt % L::kVSt;
        if (!mbar_wait(&v_full[st], (gt / L::kVSt) & 1)) return false;
        tc::fence_after_sync();
        // V: keys are K, 64-dimension halves (N) 16 KB apart, 8-key groups 1 KB apart
        const uint64_t b0 = dv + (uint64_t)((st * L::kTile) >> 4);
        const uint32_t pa = tmem + L::kTmemP + (gt & 1) * (kKeys / 2);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          tc::mma_bf16_ts(tmem + L::kTmemO, pa + kk * 8, b0 + (uint64_t)((kk * 16 * 128) >> 4), kIdescPV, acc || kk > 0);
        tc::mma_commit(&pv_done[gt & 1]);
        tc::mma_commit(&v_free[st]);
        return true;
      };
      PWalk<kKeys> w(shp, sched);
      PUnit u;
      int gk = 0, qi = 0;
      bool fine = true;
      while (fine && !*abort_flag && w.next(shp, u)) {
        const int n = u.k1 - u.k0;
        fine = mbar_wait(q_full, qi & 1) && s_product(gk);
        if (!fine) break;
        if (n == 1) tc::mma_commit(q_free);
        for (int k = 0; k < n && fine; ++k) {
          const int gt = gk + k;
          bool have_p = false;
          if (L::kSBuf == 1) {  // the one S buffer is free once P(k) is written
            fine = mbar_wait(&p_full[gt & 1], (gt >> 1) & 1);
            have_p = true;
            if (!fine) break;
          }
          if (k + 1 < n) {  // two buffers: P(k - 1), waited for below, freed this one
            fine = s_product(gt + 1);
            if (!fine) break;
            if (k + 2 == n) tc::mma_commit(q_free);  // the unit's last S product
          }
          if (!have_p) fine = mbar_wait(&p_full[gt & 1], (gt >> 1) & 1);
          // the first O += P V of a unit overwrites O: the softmax has read the last unit's
          if (fine && k == 0 && qi > 0) fine = mbar_wait(o_free, (qi - 1) & 1);
          if (fine) fine = pv_product(gt, k > 0);
        }
        gk += n;
        ++qi;
      }
      if (!fine) {
        pflag(p, GQAW_DEV_TIMEOUT);
        *abort_flag = 1;
      }
      tc::mma_commit(mma_done);  // every MMA issued has completed before TMEM is released
      if (!mbar_wait(mma_done, 0)) pflag(p, GQAW_DEV_TIMEOUT);
    }
  } else {
    // ------------------------------------------------------------ softmax (warps 0-7)
    const int wq = warp & 3, hf = warp >> 2;  // TMEM lane quarter, column half
    const int r = wq * 32 + lane;             // query row = TMEM lane
    const int bar_pair = 1 + wq;              // named barrier of warps wq and wq + 4
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t to = tmem + L::kTmemO + hf * OC + lane_off, tp = tmem + L::kTmemP + hf * 32 + lane_off;
    const bool plain = p.capmul == 0.f;
    // A cap of at most 64 (log2 units) bounds every logit: P against the reference 0 stays
    // within 2^64 both ways, so no maximum is taken and the two halves of a row never meet.
    const bool fixed = p.capmul != 0.f && p.capmul <= 64.f;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out);
    PWalk<kKeys> w(shp, sched);
    PUnit u;
    int gk = 0, odd_par = 0;
    // A warp that gives up a tile (an expired wait, an abort elsewhere) still runs every unit's
    // epilogue: the 8 warps meet at its barriers.
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
      // visible columns [lo, hi) of this row's half, relative to the tile's half; both fall by
      // 128 from tile to tile and are kept at -128 once below it
      int lo = (int)min(max(rlo - tile0 - hf * kHalfKeys, -128LL), 1LL << 30);
      int hi = (int)min(max(at + 1 - tile0 - hf * kHalfKeys, -128LL), 1LL << 30);
      float m_run = fixed ? 0.f : -INFINITY, l_run = 0.f;
      float pend = 1.f;  // the factor O in tensor memory still owes
      // some key of this CTA's tiles is attended by some of the unit's tokens only
      const bool has_part =
          u.ntok > 1 && (tile0 + (long long)n * kKeys - 1 > u.qpos || (p.W > 0 && tile0 < jhi - p.W));
      int done = 0;
      for (int k = 0; k < n; ++k) {
        const int gt = gk + k;
        const uint32_t ts = tmem + (uint32_t)(gt % L::kSBuf) * kKeys + hf * kHalfKeys + lane_off;
        const uint32_t tpk = tp + (uint32_t)(gt & 1) * (kKeys / 2);
        const int c_lo = min(max(lo, 0), kHalfKeys), c_hi = min(max(hi, 0), kHalfKeys);
        lo = max(lo - kKeys, -kKeys);
        hi = max(hi - kKeys, -kKeys);
        const bool okw = __all_sync(0xffffffffu, !*abort_flag && mbar_wait(&s_full[gt & 1], (gt >> 1) & 1));
        tc::fence_after_sync();
        bool okp = true;
        if (idle || (fixed && !okw)) {
          okp = okw;
        } else if (fixed) {
          const bool whole = __all_sync(0xffffffffu, c_lo == 0 && c_hi == kHalfKeys);
          l_run += whole ? tile_p_cap<false>(ts, tpk, 0, kHalfKeys, p.qscale, p.capmul)
                         : tile_p_cap<true>(ts, tpk, c_lo, c_hi, p.qscale, p.capmul);
        } else {
          const bool whole = __all_sync(0xffffffffu, c_lo == 0 && c_hi == kHalfKeys);
          // Fast: a plain, wholly visible tile of rows that have a reference already: P against
          // it in the same pass as the maximum.  Else the maximum first (capped logits are
          // written back transformed, invisible columns as -inf).
          const bool fast = okw && plain && whole && __all_sync(0xffffffffu, m_run > -INFINITY);
          float mt = -INFINITY, lt = 0.f;
          if (fast) {
            lt = tile_p<false, true>(ts, tpk, 0, kHalfKeys, p.qscale, m_run, &mt);
            mt *= p.qscale;
          } else if (okw && plain) {
            mt = (whole ? tile_max<false>(ts, c_lo, c_hi) : tile_max<true>(ts, c_lo, c_hi)) * p.qscale;
          } else if (okw) {
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c32 = 0; c32 < kHalfKeys / 32; ++c32) {
              float v[32];
              tc::tmem_ld32(ts + c32 * 32, v);
              const uint32_t m = chunk_mask(c32, c_lo, c_hi);
#pragma unroll
              for (int c = 0; c < 32; ++c) {
                v[c] = (m >> c) & 1u ? p.capmul * ptc::fast_tanh(v[c] * p.qscale) : -INFINITY;
                mx[c & 3] = fmaxf(mx[c & 3], v[c]);
              }
              tc::tmem_st32(ts + c32 * 32, v);
            }
            mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          }
          // Exchange with the other half (slot gt & 1: it has read slot gt & 1 of tile gt - 2
          // before it reached the barrier of tile gt - 1).  Careful when either half was not
          // fast or saw a logit more than 2^16 above the reference.
          xch[((gt & 1) * 2 + hf) * kRows + r] = mt;
          if (lane == 0) xok[((gt & 1) * 2 + hf) * 4 + wq] = okw;
          const bool careful = named_barrier_or(bar_pair, 64, !fast || mt > m_run + kDangerLog2);
          okp = okw && xok[((gt & 1) * 2 + (hf ^ 1)) * 4 + wq];
          if (okp) {
            mt = fmaxf(mt, xch[((gt & 1) * 2 + (hf ^ 1)) * kRows + r]);
            const bool need = mt > m_run + kRescaleLog2;  // both halves decide alike
            float alpha = 1.f;
            if (need) {
              alpha = m_run == -INFINITY ? 0.f : fast_exp2(m_run - mt);
              m_run = mt;
            }
            const float oscale = careful ? pend * alpha : pend;
            if (k > 0 && __any_sync(0xffffffffu, oscale != 1.f)) {
              const bool okv = __all_sync(0xffffffffu, mbar_wait(&pv_done[(gt - 1) & 1], ((gt - 1) >> 1) & 1));
              okp = !named_barrier_or(bar_pair, 64, !okv);
              tc::fence_after_sync();
              if (okp) {
#pragma unroll
                for (int c32 = 0; c32 < OC / 32; ++c32) {
                  float v[32];
                  tc::tmem_ld32(to + c32 * 32, v);
#pragma unroll
                  for (int c = 0; c < 32; ++c) v[c] *= oscale;
                  tc::tmem_st32(to + c32 * 32, v);
                }
              }
            }
            if (careful) {
              const float base = m_run == -INFINITY ? 0.f : m_run, zs = plain ? p.qscale : 1.f;
              l_run = l_run * alpha + (plain && !whole ? tile_p<true>(ts, tpk, c_lo, c_hi, zs, base)
                                                       : tile_p<false>(ts, tpk, c_lo, c_hi, zs, base));
              pend = 1.f;
            } else {
              l_run = (l_run + lt) * alpha;
              pend = alpha;
            }
          }
        }
        if (!okp) {
          if (lane == 0) pflag(p, GQAW_DEV_TIMEOUT);
          *abort_flag = 1;
          break;
        }
        // ---- value rows of the tile: key t = tid & 127, half of its dimensions
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
          constexpr int C0 = D / 16;  // 16-byte parts of half a row
          bool zero = j < jlo || j >= jhi;
          if (!zero && part && (j > u.qpos || (p.W > 0 && j < jhi - p.W))) {
            for (int c = hf * C0; c < (hf + 1) * C0; ++c) {
              const uint4 x = *reinterpret_cast<const uint4 *>(row + (c / 8) * kHalf + (((c & 7) ^ (t & 7)) << 4));
              zero |= odd_pair(x.x) || odd_pair(x.y) || odd_pair(x.z) || odd_pair(x.w);
            }
            if (zero) {
              const int kind = j > u.qpos ? 0 : 1, i = (int)(j - (kind ? jlo : u.qpos));
              atomicOr(&odd[odd_par * 16 + hf * 8 + kind * 4 + i / 32], 1u << (i & 31));
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
      // the last O += P V; the row sum from both halves
      const int gl = gk + n - 1;
      const bool okf = done == n && __all_sync(0xffffffffu, mbar_wait(&pv_done[gl & 1], (gl >> 1) & 1));
      xch[(4 + hf) * kRows + r] = l_run;
      if (named_barrier_or(bar_pair, 64, !okf)) {
        if (lane == 0) pflag(p, GQAW_DEV_TIMEOUT);
        *abort_flag = 1;
      }
      l_run += xch[(4 + (hf ^ 1)) * kRows + r];
      tc::fence_after_sync();
      bool any_odd = false;
      if (has_part) {  // also orders the bits of units two apart
        named_barrier(kSoftBar, 256);
        const volatile uint32_t *mine = odd + odd_par * 16 + hf * 8;
        for (int i = 0; i < 8; ++i) any_odd |= mine[i] != 0u;
        if (tid < 16) odd[(odd_par ^ 1) * 16 + tid] = 0u;
      }

      // ---- this half's OC columns of (O, m, l), 32 at a time
      const bool cut = u.k0 > 0 || u.k1 < u.nt;
      const int cta = blockIdx.x, cf = cut ? w.owner(u.g0) : cta, cl = cut ? w.owner(u.g0 + u.nt - 1) : cta;
      float4 *const parts = reinterpret_cast<float4 *>(p.partials);
      // partial block of a CTA: D / 4 float4 columns of O and one of (m, l), 128 rows each
      auto part_at = [&](int c, int c4) {
        return parts + (((long long)c * 2 + (c == cf ? 1 : 0)) * (D / 4 + 1) + c4) * kRows + r;
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
          uint4 x;
          x.x = tc::pack_bf16x2(v[8 * c] * f, v[8 * c + 1] * f);
          x.y = tc::pack_bf16x2(v[8 * c + 2] * f, v[8 * c + 3] * f);
          x.z = tc::pack_bf16x2(v[8 * c + 4] * f, v[8 * c + 5] * f);
          x.w = tc::pack_bf16x2(v[8 * c + 6] * f, v[8 * c + 7] * f);
          *reinterpret_cast<uint4 *>(st + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) = x;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = i * 8 + (lane >> 2), c = lane & 3;
          const long long at_ = __shfl_sync(0xffffffffu, orow, row);
          const uint4 x = *reinterpret_cast<const uint4 *>(st + row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
          if (wq * 32 + row < rows) *reinterpret_cast<uint4 *>(out + at_ + d0 + c * 8) = x;
        }
      };
#pragma unroll
      for (int c32 = 0; c32 < OC / 32; ++c32) {
        float v[32];
        __syncwarp();
        tc::tmem_ld32(to + c32 * 32, v);
        if (c32 == OC / 32 - 1) {  // O has left tensor memory: the next unit may overwrite it
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_free);
        }
        const int d0 = hf * OC + c32 * 32;
        if (row_ok) {
#pragma unroll
        for (int c = 0; c < 32; ++c) v[c] *= pend;
        if (any_odd) {  // their weights anew, from the cache, for the rows that attend them
          const volatile uint32_t *mine = odd + odd_par * 16 + hf * 8;
          for (int i = 0; i < 8; ++i)
            for (uint32_t bits = mine[i]; bits; bits &= bits - 1u) {
              const long long j = (i < 4 ? u.qpos : jlo) + (i & 3) * 32 + __ffs((int)bits) - 1;
              const long long off = j >= rlo && j <= at ? cache_row(p, u.b, u.hu, (int)j) : -1;
              if (off < 0) continue;
              const __nv_bfloat16 *kr = static_cast<const __nv_bfloat16 *>(p.kp) + off;
              const __nv_bfloat16 *vr = static_cast<const __nv_bfloat16 *>(p.vp) + off + d0;
              const __nv_bfloat16 *qr = static_cast<const __nv_bfloat16 *>(p.q) + (u.row0 + tok) * p.qs + (long long)h * D;
              float z = 0.f;
              for (int d = 0; d < D; ++d) z = fmaf(__bfloat162float(qr[d]), __bfloat162float(kr[d]), z);
              z *= p.qscale;
              if (!plain) z = p.capmul * ptc::fast_tanh(z);
              const float pr = fast_exp2(z - m_run);
#pragma unroll
              for (int c = 0; c < 32; ++c) v[c] = fmaf(pr, __bfloat162float(vr[c]), v[c]);
            }
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
      if (has_part) odd_par ^= 1;
      if (cut) {
        if (hf == 0 && row_ok) *part_at(cta, D / 4) = make_float4(m_run, l_run, 0.f, 0.f);
        named_barrier(kSoftBar, 256);
        if (tid == 0) {
          __threadfence();
          *s_last = atomicAdd(&p.tickets[cf], 1u) == (unsigned)(cl - cf);
        }
        named_barrier(kSoftBar, 256);
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
          for (int c32 = 0; c32 < OC / 32; ++c32) {
            const int d0 = hf * OC + c32 * 32;
            float acc[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) acc[c] = 0.f;
            if (row_ok)
              for (int c = cf; c <= cl; ++c) {
                const float f = fast_exp2(__ldcg(part_at(c, D / 4)).x - ref);
                float4 x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = __ldcg(part_at(c, d0 / 4 + i));
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  acc[4 * i] = fmaf(f, x[i].x, acc[4 * i]);
                  acc[4 * i + 1] = fmaf(f, x[i].y, acc[4 * i + 1]);
                  acc[4 * i + 2] = fmaf(f, x[i].z, acc[4 * i + 2]);
                  acc[4 * i + 3] = fmaf(f, x[i].w, acc[4 * i + 3]);
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

template <int D>
cudaError_t launch_paged_prefill_one(const PagedParams &p, const PagedMaps &maps, int grid, cudaStream_t stream) {
  constexpr int kMaxDevices = 64, kSmem = ppre::Lay<D>::kAlloc;
  static std::atomic<bool> ready[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(paged_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) ready[dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(ppre::kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see pdl_wait()
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged_prefill_kernel<D>, p, maps);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_paged_prefill(const PagedParams &p, const PagedMaps &maps, int grid, cudaStream_t stream) {
  switch (p.D) {
    case 64: return launch_paged_prefill_one<64>(p, maps, grid, stream);
    case 128: return launch_paged_prefill_one<128>(p, maps, grid, stream);
    default: return launch_paged_prefill_one<256>(p, maps, grid, stream);
  }
}

}  // namespace gqaw
