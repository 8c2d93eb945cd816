// gqaw_i4_attend.cuh -- attention over a paged cache held in 4 bits, up to 32 query rows of a kv
// head at once.
//
//     o_i = sum_j softmax_j(cap(scale q_i k_j)) v_j,  j <= i (and j > i - W), with sinks,
// k = (c - 8) s and v likewise, c the code of an element and s the scale of its 32 elements.
//
// Bound: HBM (72 bytes a row of 128), if what a byte costs in instructions stays below what the SM
// issues meanwhile: at 44 bytes a ns and SM a warp instruction is there for every 2 codes.  So
//   - codes go from shared memory to registers once and are matrix operands as they are: a nibble
//     in the low bits of an fp16 is the subnormal number c 2^-24, one in the next four bits 16 c 2^-24,
//     which the tensor cores take exactly; one AND makes two operands of two nibbles of a word, and the
//     factor of 16 goes to the query (keys) or to the end (values).  Converting to bf16 through shared
//     memory, as the 5th-generation tensor cores would need it, costs four bytes there for every
//     byte of codes, written and read again: more than its 128 bytes a cycle.  Hence mma.sync with the
//     keys (dimensions) as M, whose operands are registers, 8 query rows as N; its rate, a product of 16 x 8
//     x 16 every 2 cycles of an SM, is 2.4 times what the memory feeds;
//   - z = sum over groups g of s_g (sum_d c_d q_d - 8 sum_d q_d): the scale multiplies a group's sum in fp32,
//     and the sum of the queries is where the accumulator starts;
//   - o = sum_j (p_j s_j) (c_j - 8): with 8 rows the weights take the scales, one operand for each group,
//     and the values are subnormal numbers less 8 2^-24 (kFold).  With more rows there are more weights
//     than values: then the values are (c - 8) s in fp16, which holds them exactly.  (Here the 8 does not
//     wait for the end as with the keys: 8 sum p s beside a small result would take its last bits.)
//
// Queries come as one or two parts of fp16 (QP; fp32, or turned bf16: two), after a power of two per
// row that puts the largest element at 2^13; weights (times scales) as one part, or two for fp32 (PP).
// A weight is at most 4, since the row's reference maximum moves when exceeded by more than that, and a
// scale is taken relative to the largest power of two of its group so far: products stay below 2^15,
// and whatever the scales' size none is lost beside 2^-25.  Sums and statistics are fp32.
//
// Each warp works on its own, on tiles of 32 keys through a ring of its own (cp.async through the page
// table, any page size and strides); no barrier of the CTA falls inside a unit.  Schedule, splits and
// merges: gqaw_paged.cuh.
//
// Rows that nobody of a unit attends are not loaded and read as zeros.  A value scale that is not
// finite counts as zero in the products, and the tokens that attend it are marked: their outputs of
// that group are NaN, nobody else's.
#pragma once

#include <atomic>

#include "gqaw_i4.cuh"
#include "gqaw_paged_tc.cuh"

namespace gqaw {

namespace i4a {

constexpr int kKeys = 32;      // a warp's tile
constexpr int kUnitCost = 24;  // see gqaw_paged_sched.cuh
constexpr float kLazy = 2.f;   // log2 units

template <int D, int NT, int QP>
struct Lay {
  static constexpr int G = D / kI4Group;                 // groups of a row
  static constexpr int R = 8 * NT;                       // query rows
  static constexpr int kRow = D / 2;                     // bytes of a row's codes
  static constexpr int kCodes = kKeys * kRow;            // of a tile
  static constexpr int kScales = kKeys * G * 2;
  static constexpr int kStage = 2 * kCodes + 2 * kScales;  // K, V, their scales
  static constexpr int W = D <= 128 && NT == 1 ? 12 : 8;
  static constexpr int S = D == 32 ? 8 : D == 64 ? 6 : D == 128 ? (W == 12 ? 3 : 4) : 2;
  static constexpr int kThreads = 32 * W;
  static constexpr int PS = D + 4;                       // a row of a warp's state: D sums, maximum, sum of weights
  static constexpr int kRing = S * kStage > R * PS * 4 ? S * kStage : R * PS * 4;  // the state takes the ring's place
  static constexpr int kNorm = W * kRing;                // per warp: scales as the products take them
  static constexpr int kNormBytes = 2 * kKeys * G * 4;
  static constexpr int kQ = kNorm + W * kNormBytes;      // query operands [QP][NT][2 G][32 lanes] of 8 bytes
  static constexpr int kQsum = kQ + QP * NT * 2 * G * 32 * 8;  // [R][G] fp32: where accumulators start
  static constexpr int kQexp = kQsum + R * G * 4;        // [R]: power of two of a row
  static constexpr int kTotal = (kQexp + R * 4 + 15) / 16 * 16;
  static_assert(kTotal + 12 * 1024 <= 232448, "shared memory");
};

// Where 16-byte part `part` of row r's codes lies in a tile: parts are exchanged so that 8 rows of one
// part, and the 4 even or 4 odd rows of 8, lie in different banks.
template <int D>
__device__ __forceinline__ int at_part(int r, int part) {
  const int x = D == 256 ? r & 7 : D == 128 ? (r >> 1) & 3 : D == 64 ? (r >> 2) & 1 : 0;
  return r * (D / 2) + ((part ^ x) << 4);
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit elements over the warp, transposed.
__device__ __forceinline__ uint32_t transpose(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 floats_of(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2 *>(&h)); }
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// (x & mask) | bits
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(x), "r"(mask), "r"(bits));
  return r;
}
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^e for any e, as what fp32 holds of it
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(min(max(e, -126), 127) + 127) << 23); }
// the same, and 0 where that is too small for fp32's normal numbers
__device__ __forceinline__ float pow2_or_0(int e) { return e < -126 ? 0.f : pow2(e); }
// x 2^e without leaving fp32 on the way
__device__ __forceinline__ float times_pow2(float x, int e) {
  const int a = e / 2;
  return x * pow2(a) * pow2(e - a);
}

// The scales of a key, as the products take them: N groups, four floats a load.
template <int N>
__device__ __forceinline__ void lds_scales(const float *p, int key, float (&s)[N]) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 x = *reinterpret_cast<const float4 *>(p + (i / 4) * (kKeys * 4) + key * 4);
      s[i] = x.x, s[i + 1] = x.y, s[i + 2] = x.z, s[i + 3] = x.w;
    }
  } else if constexpr (N == 2) {
    const float2 x = *reinterpret_cast<const float2 *>(p + key * 2);
    s[0] = x.x, s[1] = x.y;
  } else {
    s[0] = p[key];
  }
}

__device__ __forceinline__ uint32_t lds32(const unsigned char *p) { return *reinterpret_cast<const uint32_t *>(p); }
__device__ __forceinline__ uint32_t lds16(const unsigned char *p) { return *reinterpret_cast<const uint16_t *>(p); }

template <int N>
__device__ __forceinline__ void cp_async(void *dst, const void *src, bool ok) {
  const int n = ok ? N : 0;  // 0: zeros
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src), "n"(N), "r"(n) : "memory");
}

}  // namespace i4a

// NT: operands of 8 query rows.  T: type of the rows outside the cache.
template <typename T, int D, int NT, int QP>
__global__ void __launch_bounds__(i4a::Lay<D, NT, QP>::kThreads, 1) i4_attend_kernel(const I4Params p) {
  using namespace i4a;
  using L = Lay<D, NT, QP>;
  constexpr int W = L::W, S = L::S, G = L::G, R = L::R, PS = L::PS;
  constexpr int PP = sizeof(T) == 4 ? 2 : 1;         // parts of a weight
  constexpr bool kFold = NT == 1;                    // the weights take the value scales
  constexpr bool kQreg = NT * QP * G <= 8;           // query operands in registers
  constexpr int SB = NT == 1 ? 2 : 1;                // blocks of 16 keys at once
  constexpr int kTop = kFold ? 12 : 11;              // a scale's largest power of two becomes 2^kTop
  constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ PSched sched;
  __shared__ int s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, t4 = lane & 3;
  unsigned char *ring = smem + warp * L::kRing;
  float *nk = reinterpret_cast<float *>(smem + L::kNorm + warp * L::kNormBytes);
  float *nv = nk + kKeys * G;                        // kFold: [key][group] fp32, else [group][key] fp16
  uint16_t *nvh = reinterpret_cast<uint16_t *>(nv);
  const uint2 *sq = reinterpret_cast<const uint2 *>(smem + L::kQ);
  float *sqsum = reinterpret_cast<float *>(smem + L::kQsum);
  int *sqexp = reinterpret_cast<int *>(smem + L::kQexp);
  pdl_wait();
  const PShape shp = shape_of(p, kUnitCost);
  sched_build<kKeys>(p, shp, &sched);
  PWalk<kKeys> walk(shp, &sched);
  PUnit u;
  while (walk.next(shp, u)) {
    const int kvh = u.hu / p.hblocks, hb = u.hu - kvh * p.hblocks;
    const int h0 = kvh * p.group + hb * p.gb, g = min(p.gb, p.group - hb * p.gb);
    const int rows = u.ntok * g;
    const long long jlo = p.W > 0 && u.qpos - p.W + 1 > 0 ? u.qpos - p.W + 1 : 0, jhi = u.qpos + u.ntok;
    const int n = (u.k1 - u.k0 - warp + W - 1) / W;  // tiles of this warp: k0 + warp, k0 + warp + W, ...
    auto key0 = [&](int i) { return (long long)(u.kt + u.k0 + warp + i * W) * kKeys; };
    auto look_up = [&](int i) {  // this lane's page of the warp's tile i: -2 when not needed
      const long long j = key0(i) + lane;
      return i < n && j >= jlo && j < jhi ? p.table[(long long)u.b * p.width + (int)j / p.page] : -2;
    };
    auto load = [&](int i, int id) {
      if (i < n) {  // uniform over the warp
        constexpr int CPR = D / 32;  // 16-byte parts of a row
        const int j = (int)key0(i) + lane, row = j - j / p.page * p.page;
        long long off = -1, soff = 0;
        if (id != -2) {
          if ((unsigned)id < (unsigned)p.npages) {
            off = id * p.sp + kvh * p.sh + row * p.sr;
            soff = id * p.tp + kvh * p.th + row * p.tr;
          } else {
            pflag(p, GQAW_DEV_BAD_PAGE);
          }
        }
        unsigned char *kb = ring + (i % S) * L::kStage, *sb = kb + 2 * L::kCodes;
#pragma unroll
        for (int c0 = 0; c0 < CPR; ++c0) {
          const int c = c0 * 32 + lane, r = c / CPR, part = c % CPR;
          const long long o = __shfl_sync(0xffffffffu, off, r);
          const bool ok = o >= 0;
          const unsigned char *k = static_cast<const unsigned char *>(p.kp) + (ok ? o : 0) + part * 16;
          const unsigned char *v = static_cast<const unsigned char *>(p.vp) + (ok ? o : 0) + part * 16;
          cp_async<16>(kb + at_part<D>(r, part), k, ok);
          cp_async<16>(kb + L::kCodes + at_part<D>(r, part), v, ok);
        }
        if constexpr (G >= 2) {
          cp_async<2 * G>(sb + lane * 2 * G, p.kscale + soff, off >= 0);
          cp_async<2 * G>(sb + L::kScales + lane * 2 * G, p.vscale + soff, off >= 0);
        } else {  // two bytes: too few for a copy
          reinterpret_cast<uint16_t *>(sb)[lane] = off >= 0 ? p.kscale[soff] : (uint16_t)0;
          reinterpret_cast<uint16_t *>(sb + L::kScales)[lane] = off >= 0 ? p.vscale[soff] : (uint16_t)0;
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int id = look_up(0);
    for (int i = 0; i < S - 1; ++i) {
      const int next = look_up(i + 1);
      load(i, id);
      id = next;
    }

    // ---- queries: a warp has a row, a lane one element of every group
    for (int r = warp; r < R; r += W) {
      const int tok = r / g, hh = r - tok * g;
      float x[G];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < G; ++i) {
        x[i] = 0.f;
        if (r < rows) {
          const long long at = (u.row0 + tok) * p.qs + (long long)(h0 + hh) * D + i * 32 + lane;
          x[i] = Elem<T>::load(static_cast<const T *>(p.q)[at]);
          if (QP == 2 && sizeof(T) == 2) x[i] += Elem<T>::load(static_cast<const T *>(p.qlo)[at]);
        }
        top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
      }
      top = __reduce_max_sync(0xffffffffu, top);
      const int e = top ? min(140 - (int)(top >> 23), 126) : 0;  // x 2^e: the largest at 2^13
      const int nib = lane & 7, step = (nib >> 1) & 1;
      const float f = nib & 1 ? 0.0625f : 1.f;                   // a code of an odd nibble counts 16 times
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const float y = times_pow2(x[i], e) * f;
        const __half h1 = __float2half_rn(y);
        float sum = __half2float(h1);
        const int slot = ((r / 8) * 2 * G + 2 * i + step) * 32 + (r & 7) * 4 + (lane >> 3);
        __half *q = reinterpret_cast<__half *>(smem + L::kQ) + slot * 4 + (nib & 1) * 2 + (nib >> 2);
        q[0] = h1;
        if (QP == 2) {
          const __half h2 = __float2half_rn(y - sum);
          q[NT * 2 * G * 32 * 4] = h2;
          sum += __half2float(h2);
        }
        sum /= f;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        if (lane == 0) sqsum[r * G + i] = sum * (-8.f / 16777216.f);
      }
      if (lane == 0) sqexp[r] = e;
    }
    __syncthreads();
    uint2 qr[kQreg ? QP * NT * 2 * G : 1];
    float qs[kQreg ? NT * G * 2 : 1];  // of this lane's two rows of each operand
    if constexpr (kQreg) {
#pragma unroll
      for (int i = 0; i < QP * NT * 2 * G; ++i) qr[i] = sq[i * 32 + lane];
#pragma unroll
      for (int i = 0; i < NT * G * 2; ++i) qs[i] = sqsum[((i / 2 / G) * 8 + 2 * t4 + (i & 1)) * G + i / 2 % G];
    }
    // z = (sum s 2^se acc) 2^(24 - se - e) qscale, e the row's power of two; se is not 0 where queries are
    // so large (e < 0) that the keys' scales may be too small for fp32 beside acc < 1
    const int se = -min(0, __reduce_min_sync(0xffffffffu, lane < rows ? sqexp[min(lane, R - 1)] : 0));
    const float sfac = pow2(se);
    float qf[NT][2], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        qf[nt][c] = p.qscale * pow2_or_0(24 - se - sqexp[nt * 8 + 2 * t4 + c]);
        m[nt][c] = -INFINITY;
        l[nt][c] = 0.f;
      }
    float o[NT][2 * G][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2 * G; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[nt][i][c] = 0.f;
    // of each group: the largest scale (bf16 bits) of the power of two seen so far, and the factor that
    // takes that power to 2^kTop
    uint32_t thr[(G + 1) / 2];
    float vf[G];
#pragma unroll
    for (int i = 0; i < (G + 1) / 2; ++i) thr[i] = 0u;
#pragma unroll
    for (int i = 0; i < G; ++i) vf[i] = pow2(127);
    uint32_t marked = 0;  // groups of row `lane` that attend a scale that is not finite

    for (int i = 0; i < n; ++i) {
      const int next = look_up(i + S);
      load(i + S - 1, id);
      id = next;
      asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
      __syncwarp();
      const unsigned char *kb = ring + (i % S) * L::kStage, *vb = kb + L::kCodes, *sb = vb + L::kCodes;
      const long long j0 = key0(i);
      const bool inner = j0 >= jlo && j0 + kKeys - 1 <= u.qpos && (p.W == 0 || j0 >= jhi - p.W);

      // ---- scales: a lane has a key
      {
        uint32_t kw[(G + 1) / 2], vw[(G + 1) / 2];
        if constexpr (G == 1) {
          kw[0] = reinterpret_cast<const uint16_t *>(sb)[lane];
          vw[0] = reinterpret_cast<const uint16_t *>(sb + L::kScales)[lane];
        } else {
#pragma unroll
          for (int x = 0; x < G / 2; ++x) {
            kw[x] = reinterpret_cast<const uint32_t *>(sb)[lane * (G / 2) + x];
            vw[x] = reinterpret_cast<const uint32_t *>(sb + L::kScales)[lane * (G / 2) + x];
          }
        }
        bool above = false, odd = false;
#pragma unroll
        for (int x = 0; x < (G + 1) / 2; ++x) {
          const uint32_t a = vw[x] & 0x7fff7fffu;
          above |= __vmaxu2(a, thr[x]) != thr[x];
        }
        if (__any_sync(0xffffffffu, above)) {
#pragma unroll
          for (int x = 0; x < (G + 1) / 2; ++x) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint32_t half = 0xffffu << (16 * hf), inf = 0x7f800000u >> (16 - 16 * hf);
              if (2 * x + hf < G && (vw[x] & 0x7fff7fffu & half) >= inf) {
                odd = true;
                vw[x] &= ~half;
              }
            }
            uint32_t mx = vw[x] & 0x7fff7fffu;
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, s));
            mx = __vmaxu2(mx | 0x007f007fu, thr[x]);
            thr[x] = mx;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              constexpr int kG = G;
              const int gr = 2 * x + hf;
              if (gr < kG) {
                const float f = pow2(kTop + 127 - (int)((mx >> (16 * hf + 7)) & 0xffu));
                const float down = f / vf[gr];
                vf[gr] = f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int c = 0; c < 4; ++c) {
                    o[nt][2 * gr][c] *= down;
                    o[nt][2 * gr + 1][c] *= down;
                  }
              }
            }
          }
          uint32_t who = __ballot_sync(0xffffffffu, odd);
          while (who) {  // a key with scales that are not finite: mark the rows that attend it
            const int k = __ffs((int)who) - 1;
            who &= who - 1u;
            const long long j = j0 + k, at = u.qpos + lane / g;
            const bool sees = lane < rows && j <= at && j >= jlo && (p.W == 0 || j > at - p.W);
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
              const uint32_t bits = reinterpret_cast<const uint16_t *>(sb + L::kScales)[k * G + gr] & 0x7f80u;
              if (sees && bits == 0x7f80u) marked |= 1u << gr;
            }
          }
        }
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
          const uint32_t ka = gr & 1 ? kw[gr / 2] & 0xffff0000u : kw[gr / 2] << 16;
          const uint32_t va = gr & 1 ? vw[gr / 2] & 0xffff0000u : vw[gr / 2] << 16;
          const float ks = __uint_as_float(ka) * sfac, vs = __uint_as_float(va) * vf[gr];
          const int at = (gr / 4) * (kKeys * 4) + lane * (G < 4 ? G : 4) + gr % 4;
          nk[at] = ks;
          if (kFold)
            nv[at] = vs;
          else
            nvh[gr * kKeys + lane] = __half_as_ushort(__float2half_rn(vs));
        }
      }
      __syncwarp();

#pragma unroll
      for (int b0 = 0; b0 < 2; b0 += SB) {
        // ---- logits of SB blocks of 16 keys: this lane has keys gid and gid + 8, rows 2 t4 and 2 t4 + 1
        float z[SB][NT][4];
#pragma unroll
        for (int b = 0; b < SB; ++b) {
          const int k0 = (b0 + b) * 16 + gid;
          float s0[G], s1[G];
          lds_scales<G>(nk, k0, s0);
          lds_scales<G>(nk, k0 + 8, s1);
#pragma unroll
          for (int gr = 0; gr < G; ++gr) {
            const uint32_t w0 = lds32(kb + at_part<D>(k0, gr) + t4 * 4), w1 = lds32(kb + at_part<D>(k0 + 8, gr) + t4 * 4);
            const uint32_t x0 = w0 >> 8, x1 = w1 >> 8;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float c[4];
              if constexpr (kQreg) {
                c[0] = c[2] = qs[(nt * G + gr) * 2];
                c[1] = c[3] = qs[(nt * G + gr) * 2 + 1];
              } else {
                c[0] = c[2] = sqsum[(nt * 8 + 2 * t4) * G + gr];
                c[1] = c[3] = sqsum[(nt * 8 + 2 * t4 + 1) * G + gr];
              }
#pragma unroll
              for (int q = 0; q < QP; ++q) {
                const int at = (q * NT + nt) * 2 * G + 2 * gr;
                const uint2 qa = kQreg ? qr[kQreg ? at : 0] : sq[at * 32 + lane], qb = kQreg ? qr[kQreg ? at + 1 : 0] : sq[(at + 1) * 32 + lane];
                mma(c, w0 & kLow, w1 & kLow, w0 & kHigh, w1 & kHigh, qa.x, qa.y);
                mma(c, x0 & kLow, x1 & kLow, x0 & kHigh, x1 & kHigh, qb.x, qb.y);
              }
              z[b][nt][0] = gr ? fmaf(s0[gr], c[0], z[b][nt][0]) : s0[gr] * c[0];
              z[b][nt][1] = gr ? fmaf(s0[gr], c[1], z[b][nt][1]) : s0[gr] * c[1];
              z[b][nt][2] = gr ? fmaf(s1[gr], c[2], z[b][nt][2]) : s1[gr] * c[2];
              z[b][nt][3] = gr ? fmaf(s1[gr], c[3], z[b][nt][3]) : s1[gr] * c[3];
            }
          }
        }
        // ---- softmax
        bool up = false;
#pragma unroll
        for (int b = 0; b < SB; ++b)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              float x = z[b][nt][c] * qf[nt][c & 1];
              if (p.capmul != 0.f) x = sizeof(T) == 4 ? cap_logit(p, x) : p.capmul * ptc::fast_tanh(x);
              if (!inner) {
                const int r = nt * 8 + 2 * t4 + (c & 1);
                const long long j = j0 + (b0 + b) * 16 + gid + (c & 2 ? 8 : 0), at = u.qpos + r / g;
                if (r >= rows || j > at || j < jlo || (p.W > 0 && j <= at - p.W)) x = -INFINITY;
              }
              z[b][nt][c] = x;
              up |= x > m[nt][c & 1] + kLazy;
            }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float mx = fmaxf(z[0][nt][c], z[0][nt][c + 2]);
              if (SB == 2) mx = fmaxf(mx, fmaxf(z[SB - 1][nt][c], z[SB - 1][nt][c + 2]));
#pragma unroll
              for (int s = 4; s < 32; s <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
              if (mx > m[nt][c] + kLazy) {
                const float f = fast_exp2(m[nt][c] - mx);  // 0 while nothing was seen
                m[nt][c] = mx;
                l[nt][c] *= f;
#pragma unroll
                for (int x = 0; x < 2 * G; ++x) o[nt][x][c] *= f, o[nt][x][c + 2] *= f;
              }
            }
        }
#pragma unroll
        for (int b = 0; b < SB; ++b) {
          // ---- weights
          const int kc = (b0 + b) * 16;
          uint32_t pb[NT][PP][kFold ? G : 1][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float pr[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float base = m[nt][c & 1] == -INFINITY ? 0.f : m[nt][c & 1];
              pr[c] = fast_exp2(z[b][nt][c] - base);
              l[nt][c & 1] += pr[c];
            }
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              float s[kFold ? G : 1] = {8192.f};
              if constexpr (kFold) lds_scales<G>(nv, kc + gid + 8 * hf, s);
#pragma unroll
              for (int gr = 0; gr < (kFold ? G : 1); ++gr) {
                const float w0 = pr[2 * hf] * s[gr], w1 = pr[2 * hf + 1] * s[gr];
                const uint32_t h = half2_of(w0, w1);
                pb[nt][0][gr][hf] = transpose(h);
                if (PP == 2) {
                  const float2 back = floats_of(h);
                  pb[nt][PP - 1][gr][hf] = transpose(half2_of(w0 - back.x, w1 - back.y));
                }
              }
            }
          }
          // ---- values: this lane has dimensions 4 gid .. 4 gid + 3 of every group, keys 2 t4, + 1, + 8, + 9
          const unsigned char *r0 = vb + 2 * gid;
          const int ka = kc + 2 * t4;
#pragma unroll
          for (int gr = 0; gr < G; ++gr) {
            const uint32_t xa = __byte_perm(lds16(r0 + at_part<D>(ka, gr)), lds16(r0 + at_part<D>(ka + 1, gr)), 0x5410);
            const uint32_t xb = __byte_perm(lds16(r0 + at_part<D>(ka + 8, gr)), lds16(r0 + at_part<D>(ka + 9, gr)), 0x5410);
            const uint32_t ya = xa >> 8, yb = xb >> 8;
            uint32_t v[2][4] = {{xa & kLow, xa & kHigh, xb & kLow, xb & kHigh}, {ya & kLow, ya & kHigh, yb & kLow, yb & kHigh}};
            if constexpr (kFold) {  // c - 8 (16 times) in units of 2^-24
#pragma unroll
              for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int c = 0; c < 4; ++c) v[x][c] = hadd2(v[x][c], c & 1 ? 0x80808080u : 0x80088008u);
            } else {  // (1024 + c) - 1032 and (1024 + 16 c) / 16 - 72: c - 8, then times its scale
              const uint32_t sa = *reinterpret_cast<const uint32_t *>(nvh + gr * kKeys + ka), sc = *reinterpret_cast<const uint32_t *>(nvh + gr * kKeys + ka + 8);
#pragma unroll
              for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  uint32_t y = v[x][c] | 0x64006400u;
                  y = c & 1 ? hfma2(y, 0x2c002c00u, 0xd480d480u) : hadd2(y, 0xe408e408u);
                  v[x][c] = hmul2(y, c & 2 ? sc : sa);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int q = 0; q < PP; ++q) {
                const uint32_t *w = pb[nt][q][kFold ? gr : 0];
#pragma unroll
                for (int x = 0; x < 2; ++x) mma(o[nt][2 * gr + x], v[x][0], v[x][1], v[x][2], v[x][3], w[0], w[1]);
              }
          }
        }
      }
      __syncwarp();  // the stage and the scales are free
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();

    // ---- the warp's state into its ring: [R][D + 4]
    float *mine = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = nt * 8 + 2 * t4 + c;
        float x = l[nt][c];
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
        const uint32_t bad = __shfl_sync(0xffffffffu, marked, r);
        if (gid == 0) {
          mine[r * PS + D] = m[nt][c];
          mine[r * PS + D + 1] = x;
        }
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
          // vf is a power of two, and its reciprocal one
          const int e = 127 - (int)(__float_as_uint(vf[gr]) >> 23) + (kFold ? 24 : -13);
          float y[4];
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const float a = o[nt][2 * gr + d / 2][c + 2 * (d & 1)];
            y[d] = times_pow2(kFold && (d & 1) ? a * 0.0625f : a, e);
            if ((bad >> gr) & 1u) y[d] = NAN;
          }
          *reinterpret_cast<float4 *>(mine + r * PS + gr * 32 + gid * 4) = make_float4(y[0], y[1], y[2], y[3]);
        }
      }
    __syncthreads();
    // ---- the warps' states joined
    const bool cut = u.k0 > 0 || u.k1 < u.nt;
    const int cta = blockIdx.x, cf = cut ? walk.owner(u.g0) : cta, cl = cut ? walk.owner(u.g0 + u.nt - 1) : cta;
    T *out = static_cast<T *>(p.out);
    float *part = p.partials + ((long long)cta * 2 + (cta == cf ? 1 : 0)) * R * PS;
    for (int e = tid; e < rows * D; e += L::kThreads) {
      const int r = e / D, d = e - r * D, tok = r / g, h = h0 + r - tok * g;
      float M = -INFINITY, A = 0.f, Z = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) M = fmaxf(M, reinterpret_cast<const float *>(smem + w * L::kRing)[r * PS + D]);
      const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float *x = reinterpret_cast<const float *>(smem + w * L::kRing) + r * PS;
        const float f = exp2f(x[D] - ref);
        Z = fmaf(f, x[D + 1], Z);
        A = fmaf(f, x[d], A);
      }
      if (cut) {
        part[r * PS + d] = A;
        if (d == 0) {
          part[r * PS + D] = M;
          part[r * PS + D + 1] = Z;
        }
      } else {
        out[(u.row0 + tok) * p.os + (long long)h * D + d] = Elem<T>::store(A * sink_reciprocal(Z, M, paged_sink_log2(p, h)));
      }
    }
    if (cut) {
      __syncthreads();
      if (tid == 0) {
        __threadfence();
        s_last = atomicAdd(&p.tickets[cf], 1u) == (unsigned)(cl - cf);
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        for (int e = tid; e < rows * D; e += L::kThreads) {
          const int r = e / D, d = e - r * D, tok = r / g, h = h0 + r - tok * g;
          float M, Z, A[1];
          merge_row<D, 1>(cf, cl, d, [&](int c) { return p.partials + ((long long)c * 2 + (c == cf)) * R * PS + r * PS; }, M, Z, A);
          out[(u.row0 + tok) * p.os + (long long)h * D + d] = Elem<T>::store(A[0] * sink_reciprocal(Z, M, paged_sink_log2(p, h)));
        }
        if (tid == 0) p.tickets[cf] = 0u;
      }
    }
    __syncthreads();  // queries and rings are reused by the next unit
  }
  pdl_launch_dependents();
}

template <typename T, int D, int NT, int QP>
cudaError_t launch_i4_attend_one(const I4Params &p, int sms, cudaStream_t stream) {
  using L = i4a::Lay<D, NT, QP>;
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> ready[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(i4_attend_kernel<T, D, NT, QP>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kTotal);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) ready[dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms);
  cfg.blockDim = dim3(L::kThreads);
  cfg.dynamicSmemBytes = L::kTotal;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see pdl_wait()
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, i4_attend_kernel<T, D, NT, QP>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// nt: 1, 2 or 4 (head size 256: 1 or 2) operands of 8 rows.
template <typename T, int QP>
cudaError_t launch_i4_attend_t(const I4Params &p, int nt, int sms, cudaStream_t stream) {
#define GQAW_I4_D(D)                                                                      \
  return nt == 1   ? launch_i4_attend_one<T, D, 1, QP>(p, sms, stream)                    \
         : nt == 2 ? launch_i4_attend_one<T, D, 2, QP>(p, sms, stream)                    \
                   : launch_i4_attend_one<T, D, D == 256 ? 2 : 4, QP>(p, sms, stream)
  switch (p.D) {
    case 32: GQAW_I4_D(32);
    case 64: GQAW_I4_D(64);
    case 128: GQAW_I4_D(128);
    default: GQAW_I4_D(256);
  }
#undef GQAW_I4_D
}

}  // namespace gqaw
