// gqaw_paged_attend.cuh -- attention over a paged cache on the CUDA cores: fp32 caches, and
// bf16 ones that the tensor-core kernels do not take (head sizes 8, 16 and 32, pages whose
// rows do not tile 128 keys, more than 128 query heads per kv head).
//
// The formula: row (token i, head h) of a query tile keeps the running maximum m, the
// sum l and the accumulator o of its softmax, in fp32,
//     m' = max(m, z_j),  l' = l 2^(m - m') + sum_j 2^(z_j - m'),  o' = o 2^(m - m') + sum_j 2^(z_j - m') v_j
// over tiles of kKeys keys, z in log2 units; the output is o / l (with the sink's term).
//
// Layout: 128 threads; BM query rows.  Thread (ty, tx) owns 4 rows and, of a tile, every
// TX-th key and every TX-th vector of dimensions, so a row's statistics are a butterfly over
// TX lanes of one warp and its probabilities never leave the warp.  K and V tiles come by
// 16-byte cp.async from wherever the page table says, one tile ahead; rows that no row of the
// tile may see are zero-filled and not read.  K rows are padded by 16 bytes: eight lanes read
// eight consecutive keys without a bank conflict.
//
// BM = 16 (decode and short verify): a warp owns 4 rows, and one without rows sits out, so
// the kernel stays bound by memory up to about 8 rows.  BM = 64 (more rows; 32 for head
// size 256): bound by the FMA pipe, 128 multiply-adds for 12 shared loads in Q.K^T.
#pragma once

#include "gqaw_paged.cuh"

namespace gqaw {

namespace prow {
constexpr int kKeys = 32;
constexpr int kThreads = 128;

template <typename T, int D, int BM>
struct Lay {
  static constexpr int RM = 4;
  static constexpr int TY = BM / RM, TX = kThreads / TY;
  static constexpr int KT = kKeys / TX > 0 ? kKeys / TX : 1;        // keys per thread and tile
  static constexpr int VW = D / TX >= 4 ? 4 : (D / TX >= 2 ? 2 : 1);  // dimensions per vector
  static constexpr int NV = D / (TX * VW) > 0 ? D / (TX * VW) : 1;    // vectors per thread
  static constexpr int kRowK = D * (int)sizeof(T) + 16;  // padded K row, bytes
  static constexpr int kRowV = D * (int)sizeof(T);
  static constexpr int kK = 0;
  static constexpr int kV = kK + 2 * kKeys * kRowK;
  static constexpr int kQ = kV + 2 * kKeys * kRowV;      // fp32, scaled
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
}  // namespace prow

template <typename T, int D, int BM>
__global__ void __launch_bounds__(prow::kThreads) paged_rows_attend_kernel(const PagedParams p) {
  using namespace prow;
  using L = Lay<T, D, BM>;
  constexpr int RM = L::RM, TX = L::TX, KT = L::KT, VW = L::VW, NV = L::NV;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ PSched sched;
  __shared__ long long rowoff[2][kKeys];
  __shared__ int s_last;
  const int tid = threadIdx.x, ty = tid / TX, tx = tid % TX;
  const int warp_row = (tid & ~31) / TX * RM;  // first row of this warp
  float *sq = reinterpret_cast<float *>(smem + L::kQ);
  float *sp = reinterpret_cast<float *>(smem + L::kP);
  pdl_wait();
  sched_build<kKeys>(p, &sched, kThreads);
  PWalk<kKeys> walk(p, &sched);
  PUnit u;
  while (walk.next(p, u)) {
    const int kvh = u.hu / p.hblocks, hb = u.hu - kvh * p.hblocks;
    const int h0 = kvh * p.group + hb * p.gb, g = min(p.gb, p.group - hb * p.gb);
    const int rows = u.ntok * g;
    // this unit's first attended key, and one past its last
    const long long jlo = p.W > 0 && u.qpos - p.W + 1 > 0 ? u.qpos - p.W + 1 : 0;
    const long long jhi = u.qpos + u.ntok;

    auto find_rows = [&](int k) {  // row offsets of tile k (relative to the unit), into slot k & 1
      if (tid < kKeys) {
        const long long j = (long long)(u.kt + k) * kKeys + tid;
        long long off = -1;
        if (k < u.k1 && j >= jlo && j < jhi) {
          off = cache_row(p, u.b, kvh, (int)j);
          if (off < 0) pflag(p, GQAW_DEV_BAD_PAGE);
        }
        rowoff[k & 1][tid] = off;
      }
    };
    auto load = [&](int k) {
      if (k < u.k1) {
        constexpr int CPR = D * (int)sizeof(T) / 16;  // 16-byte parts of a row
        for (int c = tid; c < kKeys * CPR; c += kThreads) {
          const int r = c / CPR, part = c % CPR;
          const long long off = rowoff[k & 1][r];
          const T *ks = static_cast<const T *>(p.kp) + (off < 0 ? 0 : off), *vs = static_cast<const T *>(p.vp) + (off < 0 ? 0 : off);
          cp_async16(smem_u32(smem + L::kK + (k & 1) * kKeys * L::kRowK + r * L::kRowK + part * 16),
                     reinterpret_cast<const char *>(ks) + part * 16, off >= 0);
          cp_async16(smem_u32(smem + L::kV + (k & 1) * kKeys * L::kRowV + r * L::kRowV + part * 16),
                     reinterpret_cast<const char *>(vs) + part * 16, off >= 0);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    find_rows(u.k0);
    // the query rows, scaled
    for (int e = tid; e < BM * D; e += kThreads) {
      const int r = e / D, d = e - r * D, tok = r / g, hh = r - tok * g;
      sq[e] = r < rows ? Elem<T>::load(static_cast<const T *>(p.q)[(u.row0 + tok) * p.qs + (long long)(h0 + hh) * D + d]) * p.qscale
                       : 0.f;
    }
    __syncthreads();
    load(u.k0);
    find_rows(u.k0 + 1);

    float m[RM], l[RM], o[RM][NV * VW];
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
      for (int d = 0; d < NV * VW; ++d) o[i][d] = 0.f;
    }
    for (int k = u.k0; k < u.k1; ++k) {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();  // tile k and the row offsets of tile k + 1 are there; tile k - 1 is done with
      load(k + 1);
      if (warp_row < rows) {  // uniform over the warp, whose lanes exchange values below
        const unsigned char *kb = smem + L::kK + (k & 1) * kKeys * L::kRowK;
        const T *vb = reinterpret_cast<const T *>(smem + L::kV + (k & 1) * kKeys * L::kRowV);
        float z[RM][KT];
#pragma unroll
        for (int i = 0; i < RM; ++i)
#pragma unroll
          for (int c = 0; c < KT; ++c) z[i][c] = 0.f;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
          float qf[RM][4], kf[KT][4];
#pragma unroll
          for (int i = 0; i < RM; ++i) lds<4>(sq + (ty * RM + i) * D + d, qf[i]);
#pragma unroll
          for (int c = 0; c < KT; ++c) lds<4>(reinterpret_cast<const T *>(kb + (tx + c * TX) * L::kRowK) + d, kf[c]);
#pragma unroll
          for (int i = 0; i < RM; ++i)
#pragma unroll
            for (int c = 0; c < KT; ++c)
#pragma unroll
              for (int x = 0; x < 4; ++x) z[i][c] = fmaf(qf[i][x], kf[c][x], z[i][c]);
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
#pragma unroll
          for (int d = 0; d < NV * VW; ++d) o[i][d] *= f;
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
            for (int x = 0; x < 4; ++x)
#pragma unroll
              for (int n = 0; n < NV; ++n) {
                float vf[VW];
                lds<VW>(vb + (c + x) * D + (tx + n * TX) * VW, vf);
#pragma unroll
                for (int i = 0; i < RM; ++i)
                  if (!hidden || pf[i][x] >= 0.f)
#pragma unroll
                    for (int y = 0; y < VW; ++y) o[i][n * VW + y] = fmaf(pf[i][x], vf[y], o[i][n * VW + y]);
              }
          }
        }
        __syncwarp();
      }
      find_rows(k + 2);  // into the slot that load(k) used, before the barrier above
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

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
              for (int y = 0; y < VW; ++y) row[(tx + n * TX) * VW + y] = Elem<T>::store(o[i][n * VW + y] * inv);
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
              for (int y = 0; y < VW; ++y) part[r * PS + (tx + n * TX) * VW + y] = o[i][n * VW + y];
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
          float M = -INFINITY, A = 0.f, S = 0.f;
          for (int c = cf; c <= cl; ++c)
            M = fmaxf(M, __ldcg(p.partials + ((long long)c * 2 + (c == cf)) * BM * PS + r * PS + D));
          const float ref = M == -INFINITY ? 0.f : M;
          for (int c = cf; c <= cl; ++c) {
            const float *q = p.partials + ((long long)c * 2 + (c == cf)) * BM * PS + r * PS;
            const float f = exp2f(__ldcg(q + D) - ref);
            S = fmaf(f, __ldcg(q + D + 1), S);
            A = fmaf(f, __ldcg(q + d), A);
          }
          out[(u.row0 + tok) * p.os + (long long)h * D + d] =
              Elem<T>::store(A * sink_reciprocal(S, M, paged_sink_log2(p, h)));
        }
        if (tid == 0) p.tickets[cf] = 0u;
      }
    }
    __syncthreads();  // sq, rowoff and the tiles are reused by the next unit
  }
  pdl_launch_dependents();
}

}  // namespace gqaw
