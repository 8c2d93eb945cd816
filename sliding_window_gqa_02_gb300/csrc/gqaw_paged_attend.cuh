// gqaw_paged_attend.cuh -- attention over a paged cache on the CUDA cores: fp32 caches, and
// bf16 ones that the tensor-core kernels do not take (head sizes 8, 16 and 32, pages whose
// rows do not tile 128 keys, more than 128 query heads per kv head).
//
// The formula: row (token i, head h) of a query tile keeps the running maximum m, the
// sum l and the accumulator o of its softmax, in fp32,
//     m' = max(m, z_j),  l' = l 2^(m - m') + sum_j 2^(z_j - m'),  o' = o 2^(m - m') + sum_j 2^(z_j - m') v_j
// over tiles of kKeys keys, z in log2 units; the output is o / l (with the sink's term).
//
// Layout: BM query rows.  Thread (ty, tx) owns 4 rows and, of a tile, every TX-th key and every
// TX-th vector of dimensions, so a row's statistics are a butterfly over TX lanes of one warp and
// its probabilities never leave the warp.  Products are packed pairs of fp32 (one instruction for
// two multiply-adds).  K and V tiles come by 16-byte cp.async from wherever the page table says,
// kStages - 1 tiles ahead, and the table entries a tile before that; rows that no row of the tile
// may see are zero-filled and not read.  K rows are padded by 16 bytes: eight lanes read eight
// consecutive keys without a bank conflict.
//
// BM = 16 (decode and short verify, 128 threads): a warp owns 4 rows, and one without rows sits
// out, so the kernel stays bound by memory up to about 8 rows.  BM = 128 (more rows; 64 for head
// size 256; 256 threads): bound by the FMA pipe, 64 packed multiply-adds for 8 shared loads in
// Q.K^T.
#pragma once

#include "gqaw_paged.cuh"

namespace gqaw {

namespace prow {
constexpr int kKeys = 32;
constexpr int kUnitCost = 4;  // see gqaw_paged_sched.cuh

template <typename T, int D, int BM>
struct Lay {
  static constexpr int kThreads = BM == 16 ? 128 : 256;
  static constexpr int RM = 4;
  static constexpr int TY = BM / RM, TX = kThreads / TY;
  static constexpr int kStages = D * (int)sizeof(T) <= 512 ? 3 : 2;
  static constexpr int KT = kKeys / TX > 0 ? kKeys / TX : 1;        // keys per thread and tile
  static constexpr int VW = D / TX >= 4 ? 4 : (D / TX >= 2 ? 2 : 1);  // dimensions per vector
  static constexpr int NV = D / (TX * VW) > 0 ? D / (TX * VW) : 1;    // vectors per thread
  static constexpr int kRowK = D * (int)sizeof(T) + 16;  // padded K row, bytes
  static constexpr int kRowV = D * (int)sizeof(T);
  static constexpr int kK = 0;
  static constexpr int kV = kK + kStages * kKeys * kRowK;
  static constexpr int kQ = kV + kStages * kKeys * kRowV;      // fp32, scaled
  static constexpr int kPS = kKeys + 4;                  // row stride of P
  static constexpr int kP = kQ + BM * D * 4;
  static constexpr int kTotal = kP + BM * kPS * 4;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}

// N consecutive elements of a shared row as floats
template <int N>
__device__ __forceinline__ void lds(const float *s, float (&f)[N]) {
  if constexpr (N == 4) {
    const float4 v = *reinterpret_cast<const float4 *>(s);
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
  } else if constexpr (N == 2) {
    const float2 v = *reinterpret_cast<const float2 *>(s);
    f[0] = v.x, f[1] = v.y;
  } else {
    f[0] = *s;
  }
}
template <int N>
__device__ __forceinline__ void lds(const __nv_bfloat16 *s, float (&f)[N]) {
  if constexpr (N == 4) {
    const uint2 v = *reinterpret_cast<const uint2 *>(s);
    f[0] = __uint_as_float(v.x << 16), f[1] = __uint_as_float(v.x & 0xffff0000u);
    f[2] = __uint_as_float(v.y << 16), f[3] = __uint_as_float(v.y & 0xffff0000u);
  } else if constexpr (N == 2) {
    const uint32_t v = *reinterpret_cast<const uint32_t *>(s);
    f[0] = __uint_as_float(v << 16), f[1] = __uint_as_float(v & 0xffff0000u);
  } else {
    f[0] = __bfloat162float(*s);
  }
}

// Packed pairs of fp32.
__device__ __forceinline__ uint64_t pk(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpk(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
}  // namespace prow

template <typename T, int D, int BM>
__global__ void __launch_bounds__(prow::Lay<T, D, BM>::kThreads) paged_rows_attend_kernel(const PagedParams p) {
  using namespace prow;
  using L = Lay<T, D, BM>;
  constexpr int kThreads = L::kThreads, kStages = L::kStages, RM = L::RM, TX = L::TX, KT = L::KT, VW = L::VW, NV = L::NV;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ PSched sched;
  __shared__ long long rowoff[kStages][kKeys];
  __shared__ int s_last;
  const int tid = threadIdx.x, ty = tid / TX, tx = tid % TX;
  const int warp_row = (tid & ~31) / TX * RM;  // first row of this warp
  float *sq = reinterpret_cast<float *>(smem + L::kQ);
  float *sp = reinterpret_cast<float *>(smem + L::kP);
  pdl_wait();
  const PShape shp = shape_of(p, kUnitCost);
  sched_build<kKeys>(p, shp, &sched);
  PWalk<kKeys> walk(shp, &sched);
  PUnit u;
  while (walk.next(shp, u)) {
    const int kvh = u.hu / p.hblocks, hb = u.hu - kvh * p.hblocks;
    const int h0 = kvh * p.group + hb * p.gb, g = min(p.gb, p.group - hb * p.gb);
    const int rows = u.ntok * g;
    // this unit's first attended key, and one past its last
    const long long jlo = p.W > 0 && u.qpos - p.W + 1 > 0 ? u.qpos - p.W + 1 : 0;
    const long long jhi = u.qpos + u.ntok;

    // Tile k (relative to the unit) sits in stage k % kStages.  Its table entries are read by
    // the last warp, which seldom has rows where time matters, a tile before its loads go out.
    auto look_up = [&](int k) {  // this thread's page of tile k: -2 when not needed
      const long long j = (long long)(u.kt + k) * kKeys + (tid & 31);
      return k < u.k1 && j >= jlo && j < jhi ? p.table[(long long)u.b * p.width + (int)j / p.page] : -2;
    };
    auto put_rows = [&](int k, int id) {
      const int j = (u.kt + k) * kKeys + (tid & 31);
      long long off = -1;
      if (id != -2) {
        if ((unsigned)id < (unsigned)p.npages)
          off = id * p.sp + kvh * p.sh + (long long)(j - j / p.page * p.page) * p.sr;
        else
          pflag(p, GQAW_DEV_BAD_PAGE);
      }
      rowoff[k % kStages][tid & 31] = off;
    };
    auto load = [&](int k) {
      if (k < u.k1) {
        constexpr int CPR = D * (int)sizeof(T) / 16;  // 16-byte parts of a row
        const int st = k % kStages;
        for (int c = tid; c < kKeys * CPR; c += kThreads) {
          const int r = c / CPR, part = c % CPR;
          const long long off = rowoff[st][r];
          const T *ks = static_cast<const T *>(p.kp) + (off < 0 ? 0 : off), *vs = static_cast<const T *>(p.vp) + (off < 0 ? 0 : off);
          cp_async16(smem_u32(smem + L::kK + (st * kKeys + r) * L::kRowK + part * 16),
                     reinterpret_cast<const char *>(ks) + part * 16, off >= 0);
          cp_async16(smem_u32(smem + L::kV + (st * kKeys + r) * L::kRowV + part * 16),
                     reinterpret_cast<const char *>(vs) + part * 16, off >= 0);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const bool finder = tid >= kThreads - 32;
    int id = -2;
    if (finder)
      for (int k = 0; k < kStages; ++k) put_rows(u.k0 + k, look_up(u.k0 + k));
    // the query rows, scaled
    for (int e = tid; e < BM * D; e += kThreads) {
      const int r = e / D, d = e - r * D, tok = r / g, hh = r - tok * g;
      float x = 0.f;
      if (r < rows) {
        const long long at = (u.row0 + tok) * p.qs + (long long)(h0 + hh) * D + d;
        x = Elem<T>::load(static_cast<const T *>(p.q)[at]);
        if (p.qlo) x += Elem<T>::load(static_cast<const T *>(p.qlo)[at]);
      }
      sq[e] = x * p.qscale;
    }
    __syncthreads();
    for (int k = 0; k < kStages - 1; ++k) load(u.k0 + k);

    constexpr int NO = (NV * VW + 1) / 2;  // accumulators of a row, in pairs
    float m[RM], l[RM];
    uint64_t o[RM][NO];
    long long vlo[RM], vhi[RM];  // keys [vlo, vhi) that each row attends
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
      const int r = ty * RM + i;
      const long long at = u.qpos + r / g;
      vhi[i] = r < rows ? at + 1 : 0;
      vlo[i] = p.W > 0 && at - p.W + 1 > 0 ? at - p.W + 1 : 0;
#pragma unroll
      for (int d = 0; d < NO; ++d) o[i][d] = 0ull;
    }
    for (int k = u.k0; k < u.k1; ++k) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      // tile k and the rows of tile k + kStages - 1 are there; tile k - 1 is done with
      __syncthreads();
      load(k + kStages - 1);
      if (finder) id = look_up(k + kStages);
      if (warp_row < rows) {  // uniform over the warp, whose lanes exchange values below
        const int st = k % kStages;
        const unsigned char *kb = smem + L::kK + st * kKeys * L::kRowK;
        const T *vb = reinterpret_cast<const T *>(smem + L::kV + st * kKeys * L::kRowV);
        uint64_t z2[RM][KT];
#pragma unroll
        for (int i = 0; i < RM; ++i)
#pragma unroll
          for (int c = 0; c < KT; ++c) z2[i][c] = 0ull;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
          uint64_t qf[RM][2], kf[KT][2];
#pragma unroll
          for (int i = 0; i < RM; ++i) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(sq + (ty * RM + i) * D + d);
            qf[i][0] = v.x, qf[i][1] = v.y;
          }
#pragma unroll
          for (int c = 0; c < KT; ++c) {
            const T *kr = reinterpret_cast<const T *>(kb + (tx + c * TX) * L::kRowK) + d;
            if constexpr (sizeof(T) == 4) {
              const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(kr);
              kf[c][0] = v.x, kf[c][1] = v.y;
            } else {
              float f[4];
              lds<4>(kr, f);
              kf[c][0] = pk(f[0], f[1]), kf[c][1] = pk(f[2], f[3]);
            }
          }
#pragma unroll
          for (int i = 0; i < RM; ++i)
#pragma unroll
            for (int c = 0; c < KT; ++c) {
              z2[i][c] = fma2(qf[i][0], kf[c][0], z2[i][c]);
              z2[i][c] = fma2(qf[i][1], kf[c][1], z2[i][c]);
            }
        }
        float z[RM][KT];
#pragma unroll
        for (int i = 0; i < RM; ++i)
#pragma unroll
          for (int c = 0; c < KT; ++c) {
            const float2 f = unpk(z2[i][c]);
            z[i][c] = f.x + f.y;
          }
        const long long j0 = (long long)(u.kt + k) * kKeys;
        bool hidden = false;  // some key of the tile is hidden from some row of this thread
#pragma unroll
        for (int i = 0; i < RM; ++i) {
          hidden |= j0 < vlo[i] || j0 + kKeys > vhi[i];
          float mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < KT; ++c) {
            const long long j = j0 + tx + c * TX;
            if (p.capmul != 0.f) z[i][c] = cap_logit(p, z[i][c]);
            if (j < vlo[i] || j >= vhi[i]) z[i][c] = -INFINITY;
            mx = fmaxf(mx, z[i][c]);
          }
#pragma unroll
          for (int s = TX < 32 ? TX / 2 : 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
          const float mn = fmaxf(m[i], mx), ref = mn == -INFINITY ? 0.f : mn;
          const float f = exp2f(m[i] - ref);  // 0 while nothing was seen
          float sum = 0.f;
#pragma unroll
          for (int c = 0; c < KT; ++c) {
            const long long j = j0 + tx + c * TX;
            float pr = exp2f(z[i][c] - ref);
            sum += pr;
            if (j < vlo[i] || j >= vhi[i]) pr = -1.f;  // hidden: its value row is not touched
            sp[(ty * RM + i) * L::kPS + tx + c * TX] = pr;
          }
#pragma unroll
          for (int s = TX < 32 ? TX / 2 : 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
          l[i] = fmaf(l[i], f, sum);
          m[i] = mn;
          const uint64_t f2 = pk(f, f);
#pragma unroll
          for (int d = 0; d < NO; ++d) o[i][d] = fma2(o[i][d], f2, 0ull);
        }
        __syncwarp();
        hidden = __any_sync(0xffffffffu, hidden);
        if (tx * VW < D) {
#pragma unroll 2
          for (int c = 0; c < kKeys; c += 4) {
            float pf[RM][4];
#pragma unroll
            for (int i = 0; i < RM; ++i) lds<4>(sp + (ty * RM + i) * L::kPS + c, pf[i]);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint64_t vf[NO];
#pragma unroll
              for (int n = 0; n < NV; ++n) {
                float f[VW];
                lds<VW>(vb + (c + x) * D + (tx + n * TX) * VW, f);
                if constexpr (VW == 4) {
                  vf[2 * n] = pk(f[0], f[1]);
                  vf[2 * n + 1] = pk(f[2], f[3]);
                } else {  // VW < 4: one vector
                  vf[n] = pk(f[0], VW > 1 ? f[VW - 1] : 0.f);
                }
              }
#pragma unroll
              for (int i = 0; i < RM; ++i)
                if (!hidden || pf[i][x] >= 0.f) {
                  const uint64_t p2 = pk(pf[i][x], pf[i][x]);
#pragma unroll
                  for (int n = 0; n < NO; ++n) o[i][n] = fma2(p2, vf[n], o[i][n]);
                }
            }
          }
        }
        __syncwarp();
      }
      if (finder) put_rows(k + kStages, id);  // into the slot of tile k, whose loads went out long ago
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    float of[RM][2 * NO];
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
      for (int d = 0; d < NO; ++d) {
        const float2 f = unpk(o[i][d]);
        of[i][2 * d] = f.x;
        of[i][2 * d + 1] = f.y;
      }
    // ---- the unit's rows, or this CTA's part of them
    const bool cut = u.k0 > 0 || u.k1 < u.nt;
    T *out = static_cast<T *>(p.out);
    if (!cut) {
      if (tx * VW < D) {
#pragma unroll
        for (int i = 0; i < RM; ++i) {
          const int r = ty * RM + i;
          if (r < rows) {
            const int tok = r / g, h = h0 + r - tok * g;
            const float inv = sink_reciprocal(l[i], m[i], paged_sink_log2(p, h));
            T *row = out + (u.row0 + tok) * p.os + (long long)h * D;
#pragma unroll
            for (int n = 0; n < NV; ++n)
#pragma unroll
              for (int y = 0; y < VW; ++y) row[(tx + n * TX) * VW + y] = Elem<T>::store(of[i][n * VW + y] * inv);
          }
        }
      }
    } else {
      constexpr int PS = D + 2;
      const int cf = walk.owner(u.g0), cl = walk.owner(u.g0 + u.nt - 1);
      float *part = p.partials + ((long long)blockIdx.x * 2 + ((int)blockIdx.x == cf ? 1 : 0)) * BM * PS;
#pragma unroll
      for (int i = 0; i < RM; ++i) {
        const int r = ty * RM + i;
        if (r < rows) {
          if (tx * VW < D) {
#pragma unroll
            for (int n = 0; n < NV; ++n)
#pragma unroll
              for (int y = 0; y < VW; ++y) part[r * PS + (tx + n * TX) * VW + y] = of[i][n * VW + y];
          }
          if (tx == 0) {
            part[r * PS + D] = m[i];
            part[r * PS + D + 1] = l[i];
          }
        }
      }
      __syncthreads();
      if (tid == 0) {
        __threadfence();
        s_last = atomicAdd(&p.tickets[cf], 1u) == (unsigned)(cl - cf);
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        for (int e = tid; e < rows * D; e += kThreads) {
          const int r = e / D, d = e - r * D, tok = r / g, h = h0 + r - tok * g;
          float M, S, A[1];
          merge_row<D, 1>(cf, cl, d, [&](int c) { return p.partials + ((long long)c * 2 + (c == cf)) * BM * PS + r * PS; }, M, S, A);
          out[(u.row0 + tok) * p.os + (long long)h * D + d] =
              Elem<T>::store(A[0] * sink_reciprocal(S, M, paged_sink_log2(p, h)));
        }
        if (tid == 0) p.tickets[cf] = 0u;
      }
    }
    __syncthreads();  // sq, rowoff and the tiles are reused by the next unit
  }
  pdl_launch_dependents();
}

}  // namespace gqaw
