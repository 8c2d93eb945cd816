// gqaw_paged_dec.cu -- paged attention of few query rows per kv head (decode: at most 8 rows,
// tokens x query heads of a kv head) on the 5th-generation tensor cores, bf16, head sizes 64,
// 128 and 256.
//
// Bound: HBM.  Every attended key and value row is read once; the arithmetic is 2 x 16 padded
// rows wide.  So the products run transposed, the 128 keys of a tile as the
// MMA's M dimension, and little work is left per key:
//   S^T = K Q^T        M = 128 keys, N = 16 query rows, K = D dimensions
//   O^T += V^T P^T     M = 128 dimensions (two blocks for 256), N = 16 rows, K = 128 keys
// With head size 64 the second 64 of V^T's M rows repeat the first (a leading offset of 0);
// their results are not read.
// A softmax thread owns one key (a TMEM lane) and NC of the query rows.  The rows keep a
// reference maximum, uniform over the CTA, that moves only when a logit exceeds it by more
// than 2^8 (one vote per tile), so P = 2^(z - ref) stays within fp32 and bf16 range, the
// common tile needs no reduction across threads, and each thread sums its own keys' weights
// in fp32.  The MMA has 16 rows and a unit at most 8, so the other 8 are put to use: row n + 8 of
// P^T holds what bf16 left of row n's weights, and the two rows of O^T are added at the end.  The
// weights so enter the product with 16 bits instead of 8, at no cost in time, and the output's
// only rounding is its own (error against 64 bits 0.0023 -> 0.0017 relative).  Likewise rows 8 to 15
// of Q hold what bf16 left of queries that the step has turned, and the two logits are added.
//
// Measured: 64 contexts of 4096 to 32768 keys (3.6 GB) in 506 to 515 us on different machines, 7.0 to
// 7.1 TB/s, 105 to 107% of the measured copy rate; one sequence of 131 keys 8.0 us.  Head sizes 64
// and 256 reach 6.5 and 7.0 TB/s with pages of 64 rows, 4.7 and 5.0 with pages of 16 (copies of 2 KB).
//
// Warps: 4 CG softmax warps, a TMA warp for Q and K and one for V (a lane looks up each box of
// a tile), one warp issuing S^T and one issuing P.V.  K and V tiles alternate through one ring of
// kSlots tiles, so the loads run up to kSlots tiles ahead of the products, over the ends of units.  The schedule
// is that of gqaw_paged.cuh.
//
// Keys that some rows attend and others do not (several new tokens) sit in the last tiles:
// there a value row that is not finite would spoil the rows that do not attend it, 0 x inf
// being NaN.  Such rows are looked for, zeroed for the product, and added on the CUDA cores to
// the rows that do attend them.
//
// Every wait is bounded; one that expires flags GQAW_DEV_TIMEOUT and the CTA winds down.
#include <atomic>

#include "gqaw_paged_tc.cuh"

namespace gqaw {

namespace pdec {

using ptc::kHalf;
using ptc::kKeys;
constexpr float kRescale = 8.0f;  // log2 units
constexpr int kBar = 1;           // named barrier of the softmax warps
constexpr int kUnitCost = 2;      // see gqaw_paged_sched.cuh

constexpr int NPAD = 16;   // rows of the MMA: 8 of a unit, and what is left of their weights
constexpr int CG = 2;      // column groups of softmax warps: more warps to overlap than the rows need
constexpr int kThreads = 32 * (4 * CG + 4);

template <int D>
struct Lay {
  static constexpr int HALVES = D / 64;
  static constexpr int DM = D > 128 ? D / 128 : 1;  // 128-dimension blocks of O^T
  static constexpr int kTile = HALVES * kHalf;
  // as many tiles in flight as fit beside Q and P: at 44 bytes per ns and SM, a load that
  // takes 2 us needs 90 KB under way
  static constexpr int kSlots = D == 64 ? 10 : D == 128 ? 6 : 2;
  // Even, so that a slot holds keys only or values only: the one thread that consumes them
  // has waited for the slot's last tile before it waits for the next.  (An odd count puts K
  // where V was; the S^T thread could then take V's pending phase for K's completed one.)
  static_assert(kSlots % 2 == 0, "slots alternate between K and V");
  static constexpr int kQHalf = NPAD * 128;           // 64 columns of Q or P^T
  static constexpr int kQBuf = HALVES * kQHalf;
  static constexpr int kQ = kSlots * kTile;           // two Q buffers
  static constexpr int kP = kQ + 2 * kQBuf;           // two P^T buffers
  static constexpr int kSched = kP + 4 * kQHalf;
  static constexpr int kRed = kSched + (int)((sizeof(PSched) + 15) / 16 * 16);  // float [4][NPAD]
  static constexpr int kFin = kRed + 4 * NPAD * 4;    // float m, l [2][NPAD]
  static constexpr int kBars = kFin + 2 * NPAD * 4;
  static constexpr int kNumBars = 2 * kSlots + 14;
  static constexpr int kMisc = kBars + kNumBars * 8;  // TMEM address, flags
  static constexpr int kAlloc = kMisc + 64 + 1024;    // and room to align the base
  static constexpr uint32_t kCols = 64;  // S^T twice, O^T
  static_assert((2 + DM) * NPAD <= (int)kCols, "tensor memory columns");
  static_assert(kAlloc <= 232448, "shared memory");
};

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[N]);
template <>
__device__ __forceinline__ void tmem_ld<2>(uint32_t taddr, float (&v)[2]) {
  uint32_t r[2];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];\ntcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]) : "r"(taddr));
  v[0] = __uint_as_float(r[0]);
  v[1] = __uint_as_float(r[1]);
}
template <>
__device__ __forceinline__ void tmem_ld<4>(uint32_t taddr, float (&v)[4]) {
  uint32_t r[4];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\ntcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const float (&v)[N]);
template <>
__device__ __forceinline__ void tmem_st<2>(uint32_t taddr, const float (&v)[2]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(taddr), "r"(__float_as_uint(v[0])),
               "r"(__float_as_uint(v[1])) : "memory");
  tc::tmem_wait_st();
}
template <>
__device__ __forceinline__ void tmem_st<4>(uint32_t taddr, const float (&v)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(__float_as_uint(v[0])),
               "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])) : "memory");
  tc::tmem_wait_st();
}
// Does a pair of bf16 in a word hold an infinity or a NaN?
__device__ __forceinline__ bool odd_pair(uint32_t w) {
  return (w & 0x7f800000u) == 0x7f800000u || (w & 0x00007f80u) == 0x00007f80u;
}

}  // namespace pdec

// NVT: rows the softmax warps work on (4 or 8), NC = NVT / CG of them a thread.
template <int D, int NVT>
__global__ void __launch_bounds__(pdec::kThreads, 1)
    paged_decode_kernel(const PagedParams p, const __grid_constant__ PagedMaps maps) {
  using namespace pdec;
  using ptc::fast_exp2;
  using L = Lay<D>;
  constexpr int NC = NVT / CG, kSoft = 128 * CG, DM = L::DM, kSlots = L::kSlots;
  constexpr int kSoftWarps = 4 * CG, kKWarp = kSoftWarps, kVWarp = kKWarp + 1, kSWarp = kKWarp + 2, kPVWarp = kKWarp + 3;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  PSched *sched = reinterpret_cast<PSched *>(smem + L::kSched);
  float *red = reinterpret_cast<float *>(smem + L::kRed);
  float *fin_m = reinterpret_cast<float *>(smem + L::kFin), *fin_l = fin_m + NPAD;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBars);
  uint64_t *full = bars, *empty = bars + kSlots, *s_full = bars + 2 * kSlots, *s_free = s_full + 2;
  // two barriers each where one side may run a tile ahead: a parity wait cannot tell two
  // phases apart
  uint64_t *p_full = s_free + 2, *o_done = p_full + 2, *q_full = o_done + 2, *q_free = q_full + 2;
  uint64_t *o_free = q_free + 2, *mma_done = o_free + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMisc);
  int *s_abort = reinterpret_cast<int *>(smem + L::kMisc + 4), *s_last = s_abort + 1;
  uint32_t *s_odd = reinterpret_cast<uint32_t *>(smem + L::kMisc + 16);  // [4] keys with a value that is not finite

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    ptc::prefetch_map(&maps.q);
    ptc::prefetch_map(&maps.k);
    ptc::prefetch_map(&maps.v);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], kSoftWarps);
      mbar_init(&p_full[i], kSoftWarps);
      mbar_init(&o_done[i], 1);
      mbar_init(&q_full[i], 1);
      mbar_init(&q_free[i], 1);
    }
    mbar_init(o_free, kSoftWarps);
    mbar_init(mma_done, 2);
    mbar_fence_init();
    *s_abort = 0;
  }
  // rows of Q and P^T past the unit's stay zero, or hold finite leftovers of other units
  for (int e = tid; e < (2 * L::kQBuf + 4 * L::kQHalf) / 16; e += blockDim.x)
    reinterpret_cast<uint4 *>(smem + L::kQ)[e] = make_uint4(0, 0, 0, 0);
  if (warp == 0) tc::tmem_alloc(tmem_slot, L::kCols);
  tc::fence_proxy_async_smem();
  pdl_wait();
  const PShape shp = shape_of(p, kUnitCost);
  sched_build<kKeys>(p, shp, sched);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot, tmem_s = tmem, tmem_o = tmem + 2 * NPAD;
  const int g = p.group;
  volatile int *abort_flag = s_abort;

  // K of tile kc (counted over the CTA's units) is load 2 kc, V load 2 kc + 1; load n sits in
  // slot n % kSlots, phase (n / kSlots) & 1
  auto slot = [&](int n) { return smem + (n % kSlots) * L::kTile; };
  auto phase = [&](int n) { return (uint32_t)(n / kSlots) & 1u; };
  auto qbuf = [&](int ui) { return smem + L::kQ + (ui & 1) * L::kQBuf; };
  auto pbuf = [&](int kc) { return smem + L::kP + (kc & 1) * 2 * L::kQHalf; };

  if (warp == kKWarp || warp == kVWarp) {
    // ------------------------------------------------------------ loads: Q and K | V (whole warps)
    const bool value = warp == kVWarp;
    const uint64_t pol = policy_evict_first(), qpol = tc::policy_evict_last();
    PWalk<kKeys> w(shp, sched);
    PUnit u;
    ptc::Boxes bx;
    int n = value ? 1 : 0, ui = 0;  // this warp's loads are n, n + 2, ...
    bool alive = true;
    while (alive && w.next(shp, u)) {
      bx.unit(p, u);
      bx.look_up(p, u.kt + u.k0, lane);
      if (!value) {
        if (ui >= 2) alive = __all_sync(0xffffffffu, mbar_wait(&q_free[ui & 1], ((ui - 2) >> 1) & 1));
        if (!alive) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&q_full[ui & 1], (uint32_t)((p.qlo ? 2 : 1) * L::HALVES * g * p.tpt * 128));
          for (int h = 0; h < L::HALVES; ++h) {
            tc::tma_load_3d(qbuf(ui) + h * L::kQHalf, &maps.q, h * 64, u.hu * g, u.row0, &q_full[ui & 1], qpol);
            if (p.qlo) tc::tma_load_3d(qbuf(ui) + h * L::kQHalf + 1024, &maps.ql, h * 64, u.hu * g, u.row0, &q_full[ui & 1], qpol);
          }
        }
        ++ui;
      }
      for (int k = u.k0; k < u.k1 && alive; ++k) {
        const uint32_t mask = bx.valid(p, u.kt + k, lane);
        const uint32_t bytes = (uint32_t)(__popc(mask) * bx.rows * 128 * L::HALVES);
        const ptc::Boxes cur = bx;
        if (k + 1 < u.k1) bx.look_up(p, u.kt + k + 1, lane);  // in flight while the slot is waited for
        const int s = n % kSlots;
        if (n >= kSlots) alive = mbar_wait(&empty[s], phase(n) ^ 1u);
        alive = __all_sync(0xffffffffu, alive && !*abort_flag);
        if (!alive) break;
        if (lane == 0) mbar_arrive_expect_tx(&full[s], bytes);
        cur.load<L::HALVES>(value ? &maps.v : &maps.k, slot(n), &full[s], pol, mask, lane);
        n += 2;
      }
    }
    if (lane == 0) {
      if (!alive) {
        pflag(p, GQAW_DEV_TIMEOUT);
        *abort_flag = 1;
      }
      // no copy may still be landing in shared memory when the CTA exits
      const int first = value ? 1 : 0;
      for (int i = n - kSlots > first ? n - kSlots : first; i < n; i += 2)
        if (!mbar_wait(&full[i % kSlots], phase(i))) pflag(p, GQAW_DEV_TIMEOUT);
      for (int i = ui > 2 ? ui - 2 : 0; i < ui; ++i)
        if (!mbar_wait(&q_full[i & 1], (i >> 1) & 1)) pflag(p, GQAW_DEV_TIMEOUT);
    }
  } else if (warp == kSWarp) {
    // ------------------------------------------------------------ S^T = K Q^T
    if (lane == 0) {
      constexpr uint32_t kIdesc = tc::idesc_bf16_f32(kKeys, NPAD, 0, 0);
      PWalk<kKeys> w(shp, sched);
      PUnit u;
      int kc = 0, ui = 0;
      bool fine = true;
      while (fine && !*abort_flag && w.next(shp, u)) {
        fine = mbar_wait(&q_full[ui & 1], (ui >> 1) & 1);
        const uint64_t qd = tc::smem_desc_sw128(qbuf(ui), 16, 1024);
        for (int k = u.k0; k < u.k1 && fine; ++k, ++kc) {
          fine = mbar_wait(&full[(2 * kc) % kSlots], phase(2 * kc)) &&
                 (kc < 2 || mbar_wait(&s_free[kc & 1], ((kc - 2) >> 1) & 1));
          if (!fine) break;
          tc::fence_after_sync();
          const uint64_t kd = tc::smem_desc_sw128(slot(2 * kc), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc::mma_bf16_ss(tmem_s + (kc & 1) * NPAD, kd + (uint64_t)(((kk / 4) * kHalf + (kk % 4) * 32) >> 4),
                            qd + (uint64_t)(((kk / 4) * L::kQHalf + (kk % 4) * 32) >> 4), kIdesc, kk > 0);
          tc::mma_commit(&s_full[kc & 1]);
          tc::mma_commit(&empty[(2 * kc) % kSlots]);
        }
        ++ui;
      }
      if (!fine) {
        pflag(p, GQAW_DEV_TIMEOUT);
        *abort_flag = 1;
      }
      tc::mma_commit(mma_done);  // every MMA issued has completed before TMEM is released
      if (!mbar_wait(mma_done, 0)) pflag(p, GQAW_DEV_TIMEOUT);
    }
  } else if (warp == kPVWarp) {
    // ------------------------------------------------------------ O^T += V^T P^T
    if (lane == 0) {
      constexpr uint32_t kIdesc = tc::idesc_bf16_f32(128, NPAD, 1, 0);
      PWalk<kKeys> w(shp, sched);
      PUnit u;
      int kc = 0, ui = 0;
      bool fine = true;
      while (fine && !*abort_flag && w.next(shp, u)) {
        for (int k = u.k0; k < u.k1 && fine; ++k, ++kc) {
          fine = mbar_wait(&full[(2 * kc + 1) % kSlots], phase(2 * kc + 1)) && mbar_wait(&p_full[kc & 1], (kc >> 1) & 1) &&
                 (k > u.k0 || ui == 0 || mbar_wait(o_free, (ui - 1) & 1));
          if (!fine) break;
          tc::fence_after_sync();
          // V^T: 64-dimension halves 16 KB apart (head size 64: the one half twice), 8-key
          // groups 1 KB apart
          const uint64_t vd = tc::smem_desc_sw128(slot(2 * kc + 1), D == 64 ? 0 : kHalf, 1024);
          const uint64_t pd = tc::smem_desc_sw128(pbuf(kc), 16, 1024);
#pragma unroll
          for (int m = 0; m < DM; ++m)
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              tc::mma_bf16_ss(tmem_o + m * NPAD, vd + (uint64_t)((m * 2 * kHalf + kk * 16 * 128) >> 4),
                              pd + (uint64_t)(((kk / 4) * L::kQHalf + (kk % 4) * 32) >> 4), kIdesc, k > u.k0 || kk > 0);
          tc::mma_commit(&o_done[kc & 1]);
          tc::mma_commit(&empty[(2 * kc + 1) % kSlots]);
          if (k + 1 == u.k1) tc::mma_commit(&q_free[ui & 1]);
        }
        ++ui;
      }
      if (!fine) {
        pflag(p, GQAW_DEV_TIMEOUT);
        *abort_flag = 1;
      }
      tc::mma_commit(mma_done);
      if (!mbar_wait(mma_done, 0)) pflag(p, GQAW_DEV_TIMEOUT);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int t = tid & 127;            // key of a tile (S^T lane), dimension of O^T (lane)
    const int col0 = (tid >> 7) * NC;   // first query row of this thread
    const int wq = warp & 3;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out);
    PWalk<kKeys> w(shp, sched);
    PUnit u;
    int kc = 0;
    bool stop = false;
    while (!stop && w.next(shp, u)) {
      const int NV = u.ntok * g;
      const long long jlo = p.W > 0 && u.qpos - p.W + 1 > 0 ? u.qpos - p.W + 1 : 0, jhi = u.qpos + u.ntok;
      float m_ref[NC], lsum[NC], ext[DM][NC];
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        m_ref[i] = -INFINITY;
        lsum[i] = 0.f;
#pragma unroll
        for (int m = 0; m < DM; ++m) ext[m][i] = 0.f;
      }
      bool any_ext = false;
      // tiles [ka, kb) hold only keys that every token attends
      const int ka = (int)(((p.W > 0 ? max(0LL, jhi - p.W) : 0LL) + kKeys - 1) / kKeys) - u.kt;
      const int kb = (int)((u.qpos + 1) / kKeys) - u.kt;
      for (int k = u.k0; k < u.k1; ++k, ++kc) {
        const bool inner = k >= ka && k < kb;
        const long long j0 = (long long)(u.kt + k) * kKeys, j = j0 + t;
        // tokens [ta, tz) of the unit attend key j; their rows are [ta g, tz g)
        int ta = 0, tz = u.ntok;
        if (!inner) {
          tz = 0;
          if (j >= jlo && j < jhi) {
            ta = j > u.qpos ? (int)(j - u.qpos) : 0;
            tz = p.W > 0 ? (int)min((long long)u.ntok, j - u.qpos + p.W) : u.ntok;
          }
        }
        const int nlo = ta * g - col0, nhi = tz * g - col0;
        bool ok = mbar_wait(&s_full[kc & 1], (kc >> 1) & 1);
        __syncwarp();
        tc::fence_after_sync();
        float z[NC];
        tmem_ld<NC>(tmem_s + (kc & 1) * NPAD + col0 + lane_off, z);
        if (p.qlo) {  // an infinite logit stays what it is
          float rest[NC];
          tmem_ld<NC>(tmem_s + (kc & 1) * NPAD + 8 + col0 + lane_off, rest);
#pragma unroll
          for (int i = 0; i < NC; ++i) z[i] = fabsf(z[i]) < INFINITY ? z[i] + rest[i] : z[i];
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[kc & 1]);
        bool exceed = false;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          float v = z[i] * p.qscale;
          if (p.capmul != 0.f) v = p.capmul * ptc::fast_tanh(v);
          z[i] = i >= nlo && i < nhi ? v : -INFINITY;
          exceed |= z[i] > m_ref[i] + kRescale;
        }
        const bool fail = !ok || *abort_flag;
        const bool any = named_barrier_or(kBar, kSoft, exceed || fail);
        if (any && named_barrier_or(kBar, kSoft, fail)) {
          stop = true;
          break;
        }
        // P^T buffer kc & 1 is free once the P.V of tile kc - 2 has completed
        if (kc >= 2) ok = mbar_wait(&o_done[kc & 1], ((kc - 2) >> 1) & 1);
        tc::fence_after_sync();
        if (any) {
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            float mx = z[i];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            if (lane == 0) red[wq * NPAD + col0 + i] = mx;
          }
          named_barrier(kBar, kSoft);
          float alpha[NC];
          bool resc = false;
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            const int n = col0 + i;
            const float mt = fmaxf(fmaxf(red[n], red[NPAD + n]), fmaxf(red[2 * NPAD + n], red[3 * NPAD + n]));
            alpha[i] = 1.f;
            if (mt > m_ref[i] + kRescale) {
              alpha[i] = m_ref[i] == -INFINITY ? 0.f : fast_exp2(m_ref[i] - mt);
              m_ref[i] = mt;
              lsum[i] *= alpha[i];
              if (any_ext) {
#pragma unroll
                for (int m = 0; m < DM; ++m) ext[m][i] *= alpha[i];
              }
              resc = true;
            }
          }
          // O^T holds earlier tiles of this unit (the decision is uniform within a column group)
          if (resc && k > u.k0) {
            if (!mbar_wait(&o_done[(kc - 1) & 1], ((kc - 1) >> 1) & 1)) ok = false;
            __syncwarp();
            tc::fence_after_sync();
#pragma unroll
            for (int m = 0; m < DM; ++m) {
#pragma unroll
              for (int lo = 0; lo < 16; lo += 8) {
                float o[NC];
                tmem_ld<NC>(tmem_o + m * NPAD + lo + col0 + lane_off, o);
#pragma unroll
                for (int i = 0; i < NC; ++i) o[i] *= alpha[i];
                tmem_st<NC>(tmem_o + m * NPAD + lo + col0 + lane_off, o);
              }
            }
          }
        }
        {  // P^T: row n, key t, 128-byte swizzled, K-major
          unsigned char *pb = pbuf(kc) + (t >> 6) * L::kQHalf + (t & 7) * 2;
          const int c = (t & 63) >> 3;
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            const int n = col0 + i;
            const float pr = fast_exp2(z[i] - (m_ref[i] == -INFINITY ? 0.f : m_ref[i]));
            lsum[i] += pr;
            const __nv_bfloat16 hi = __float2bfloat16_rn(pr);
            unsigned char *at = pb + n * 128 + ((c ^ (n & 7)) << 4);  // row n + 8: 1 KB on, the same swizzle
            *reinterpret_cast<__nv_bfloat16 *>(at) = hi;
            *reinterpret_cast<__nv_bfloat16 *>(at + 1024) = __float2bfloat16_rn(pr - __bfloat162float(hi));
          }
        }
        // value rows outside [jlo, jhi) were not loaded, or may hold anything: zero them
        if (!inner) {
          const int z0 = (int)max(0LL, jlo - j0), z1 = (int)min((long long)kKeys, jhi - j0);
          // some key of the tile is attended by some tokens only
          const bool part = u.ntok > 1 && (j0 + kKeys - 1 > u.qpos || (p.W > 0 && j0 < jhi - p.W));
          // With two slots, V(kc - 1) may not have landed yet, and a parity wait cannot tell two
          // phases apart: its product first.  (With more, the slot's last tile is behind the
          // o_done waited for above.)
          if (kSlots == 2 && kc > 0 && !mbar_wait(&o_done[(kc - 1) & 1], ((kc - 1) >> 1) & 1)) ok = false;
          if (!mbar_wait(&full[(2 * kc + 1) % kSlots], phase(2 * kc + 1))) ok = false;
          unsigned char *vb = slot(2 * kc + 1);
          for (int e = tid; e < (kKeys - (z1 - z0)) * (D / 8); e += kSoft) {
            const int q = e / (D / 8), row = q < z0 ? q : z1 + q - z0, c = e % (D / 8);
            *reinterpret_cast<uint4 *>(vb + (c / 8) * kHalf + row * 128 + (c % 8) * 16) = make_uint4(0, 0, 0, 0);
          }
          if (part) {
            bool odd = false;
            if (tid < kKeys && tz > ta && (ta > 0 || tz < u.ntok)) {
              for (int c = 0; c < D / 8; ++c) {
                const uint4 x = *reinterpret_cast<const uint4 *>(vb + (c / 8) * kHalf + t * 128 + (c % 8) * 16);
                odd |= odd_pair(x.x) || odd_pair(x.y) || odd_pair(x.z) || odd_pair(x.w);
              }
            }
            if (named_barrier_or(kBar, kSoft, odd)) {
              if (tid < kKeys) {
                const uint32_t bal = __ballot_sync(0xffffffffu, odd);
                if (lane == 0) s_odd[warp] = bal;
              }
              named_barrier(kBar, kSoft);  // the keys, and P^T
              any_ext = true;
              for (int q = 0; q < 4; ++q)
                for (uint32_t bits = s_odd[q]; bits; bits &= bits - 1u) {
                  const int jj = q * 32 + __ffs((int)bits) - 1;
                  const long long ja = j0 + jj;
                  const int ra = (ja > u.qpos ? (int)(ja - u.qpos) : 0) * g;
                  const int rz = (p.W > 0 ? (int)min((long long)u.ntok, ja - u.qpos + p.W) : u.ntok) * g;
#pragma unroll
                  for (int m = 0; m < DM; ++m) {
                    const int d = m * 128 + t;
                    if (d < D) {
                      const float v = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(
                          vb + (d / 64) * kHalf + jj * 128 + ((((d & 63) >> 3) ^ (jj & 7)) << 4) + (d & 7) * 2));
#pragma unroll
                      for (int i = 0; i < NC; ++i) {
                        const int n = col0 + i;
                        const __nv_bfloat16 *pp = reinterpret_cast<const __nv_bfloat16 *>(
                            pbuf(kc) + (jj >> 6) * L::kQHalf + n * 128 + ((((jj & 63) >> 3) ^ (n & 7)) << 4) + (jj & 7) * 2);
                        const float pr = __bfloat162float(pp[0]) + __bfloat162float(pp[512]);
                        if (n >= ra && n < rz) ext[m][i] = fmaf(pr, v, ext[m][i]);
                      }
                    }
                  }
                }
              named_barrier(kBar, kSoft);  // every thread has read them
              if (odd)
                for (int c = 0; c < D / 8; ++c)
                  *reinterpret_cast<uint4 *>(vb + (c / 8) * kHalf + t * 128 + (c % 8) * 16) = make_uint4(0, 0, 0, 0);
            }
          }
        }
        if (!ok) {
          pflag(p, GQAW_DEV_TIMEOUT);
          *abort_flag = 1;
        }
        tc::fence_proxy_async_smem();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[kc & 1]);
      }
      if (stop) break;

      // ---- the unit's state in this CTA
      named_barrier(kBar, kSoft);  // every thread is done with the last maxima in red
      const bool okd = mbar_wait(&o_done[(kc - 1) & 1], ((kc - 1) >> 1) & 1);
      tc::fence_after_sync();
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float v = lsum[i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) red[wq * NPAD + col0 + i] = v;
        if (t == 0) fin_m[col0 + i] = m_ref[i];
      }
      float o[DM][NC];
      __syncwarp();
#pragma unroll
      for (int m = 0; m < DM; ++m) {
        float rest[NC];
        tmem_ld<NC>(tmem_o + m * NPAD + col0 + lane_off, o[m]);
        tmem_ld<NC>(tmem_o + m * NPAD + 8 + col0 + lane_off, rest);
#pragma unroll
        for (int i = 0; i < NC; ++i) o[m][i] += rest[i];
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);  // the next unit may overwrite O^T
      if (named_barrier_or(kBar, kSoft, !okd)) {
        pflag(p, GQAW_DEV_TIMEOUT);
        *abort_flag = 1;
        break;
      }
      if (tid < NVT) fin_l[tid] = red[tid] + red[NPAD + tid] + red[2 * NPAD + tid] + red[3 * NPAD + tid];
      if (any_ext) {
#pragma unroll
        for (int m = 0; m < DM; ++m)
#pragma unroll
          for (int i = 0; i < NC; ++i) o[m][i] += ext[m][i];
      }
      named_barrier(kBar, kSoft);
      if (u.k0 == 0 && u.k1 == u.nt) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int n = col0 + i;
          if (n < NV) {
            const int tok = n / g, h = u.hu * g + n - tok * g;
            const float inv = sink_reciprocal(fin_l[n], fin_m[n], paged_sink_log2(p, h));
            __nv_bfloat16 *row = out + (u.row0 + tok) * p.os + (long long)h * D;
#pragma unroll
            for (int m = 0; m < DM; ++m)
              if (m * 128 + t < D) row[m * 128 + t] = __float2bfloat16_rn(o[m][i] * inv);
          }
        }
      } else {
        constexpr int PS = D + 2;
        const int cf = w.owner(u.g0), cl = w.owner(u.g0 + u.nt - 1), cta = blockIdx.x;
        float *part = p.partials + ((long long)cta * 2 + (cta == cf ? 1 : 0)) * NPAD * PS;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int n = col0 + i;
          if (n < NV) {
#pragma unroll
            for (int m = 0; m < DM; ++m)
              if (m * 128 + t < D) part[n * PS + m * 128 + t] = o[m][i];
            if (t == 0) {
              part[n * PS + D] = fin_m[n];
              part[n * PS + D + 1] = fin_l[n];
            }
          }
        }
        named_barrier(kBar, kSoft);
        if (tid == 0) {
          __threadfence();
          *s_last = atomicAdd(&p.tickets[cf], 1u) == (unsigned)(cl - cf);
        }
        named_barrier(kBar, kSoft);
        if (*reinterpret_cast<volatile int *>(s_last)) {
          __threadfence();
          auto at = [&](int c) { return p.partials + ((long long)c * 2 + (c == cf ? 1 : 0)) * NPAD * PS; };
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            const int n = col0 + i;
            if (n < NV) {
              float M, S, A[DM];
              merge_row<D, DM>(cf, cl, t, [&](int c) { return at(c) + n * PS; }, M, S, A);
              const int tok = n / g, h = u.hu * g + n - tok * g;
              const float inv = sink_reciprocal(S, M, paged_sink_log2(p, h));
              __nv_bfloat16 *row = out + (u.row0 + tok) * p.os + (long long)h * D;
#pragma unroll
              for (int m = 0; m < DM; ++m)
                if (m * 128 + t < D) row[m * 128 + t] = __float2bfloat16_rn(A[m] * inv);
            }
          }
          if (tid == 0) p.tickets[cf] = 0u;
        }
      }
      named_barrier(kBar, kSoft);  // fin and red are reused by the next unit
    }
    if (stop) pflag(p, GQAW_DEV_TIMEOUT);
  }

  tc::fence_before_sync();
  __syncthreads();
  pdl_launch_dependents();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, L::kCols);
  }
}

template <int D, int NVT>
cudaError_t launch_paged_decode_one(const PagedParams &p, const PagedMaps &maps, int grid, cudaStream_t stream) {
  constexpr int kMaxDevices = 64, kSmem = pdec::Lay<D>::kAlloc;
  static std::atomic<bool> ready[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(paged_decode_kernel<D, NVT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) ready[dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(pdec::kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see pdl_wait()
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged_decode_kernel<D, NVT>, p, maps);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// rows: tokens of a query tile times group, at most 8.
template <int D>
cudaError_t launch_paged_decode_d(const PagedParams &p, const PagedMaps &maps, int rows, int grid, cudaStream_t stream) {
  return rows <= 4 ? launch_paged_decode_one<D, 4>(p, maps, grid, stream)
                   : launch_paged_decode_one<D, 8>(p, maps, grid, stream);
}

cudaError_t launch_paged_decode(const PagedParams &p, const PagedMaps &maps, int rows, int grid, cudaStream_t stream) {
  switch (p.D) {
    case 64: return launch_paged_decode_d<64>(p, maps, rows, grid, stream);
    case 128: return launch_paged_decode_d<128>(p, maps, rows, grid, stream);
    default: return launch_paged_decode_d<256>(p, maps, rows, grid, stream);
  }
}

}  // namespace gqaw
