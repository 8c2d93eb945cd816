// gqaw_paged_warp.cuh -- paged attention of at most 8 query rows per kv head on the CUDA cores:
// decode with fp32 caches, and with bf16 ones that the tensor-core kernels do not take.
//
// Bound: HBM; so everything else is kept out of the way of the loads.  Each warp of a CTA works
// on its own, with its own ring of tiles of 32 keys (warp w takes tiles w, w + W, ... of the
// CTA's part of the unit) and its own softmax state; no barrier of the CTA falls inside a unit.
//   - Each lane looks up the row of one key of a tile, a tile ahead of its loads, and the loads
//     (16-byte cp.async, neighbouring lanes on neighbouring addresses) run kStages - 1 tiles
//     ahead: at 44 bytes per ns and SM a latency of 2 us takes 90 KB under way.
//   - z: a lane has one key against all rows; K rows are padded by 16 bytes, so 32 lanes reading
//     32 rows of K conflict no more than their bytes must.  The rows keep a reference maximum
//     that moves only when exceeded by more than 2^8 (one vote a tile), sums stay in the lanes.
//   - o: a lane has D / 32 dimensions of all rows; the weights of a key come as one broadcast.
// Products are packed pairs of fp32.  At the end of a unit the warps' states are joined in shared
// memory, and a unit cut between CTAs through partial results, as in the other kernels.
#pragma once

#include "gqaw_paged_attend.cuh"

namespace gqaw {

namespace pwarp {
using prow::kKeys;
using prow::kUnitCost;

template <typename T, int D>
struct Lay {
  static constexpr int kRowK = D * (int)sizeof(T) + 16, kRowV = D * (int)sizeof(T);
  static constexpr int kStage = kKeys * (kRowK + kRowV);
  // 4 warps with 3 tiles each where they fit; rows of 512 bytes leave 3 warps with 2
  static constexpr bool kWide = D * (int)sizeof(T) >= 512;
  static constexpr int W = kWide ? 3 : 4, kStages = kWide ? 2 : 3;
  static constexpr int kThreads = 32 * W;
  static constexpr int kQ = W * kStages * kStage;      // [8][D] fp32, scaled
  static constexpr int kP = kQ + 8 * D * 4;            // [W][32 keys][8 rows]
  static constexpr int kTotal = kP + W * kKeys * 8 * 4;
  static constexpr int kPerSm = kTotal + 12 * 1024 <= 110 * 1024 ? 2 : 1;  // resident CTAs
  static_assert(8 * (D + 2) * 4 <= kStages * kStage, "a warp's state fits in its ring");
  static_assert(kTotal + 12 * 1024 <= 232448, "shared memory");
};
}  // namespace pwarp

// RM: 4 or 8 rows.
template <typename T, int D, int RM>
__global__ void __launch_bounds__(pwarp::Lay<T, D>::kThreads, pwarp::Lay<T, D>::kPerSm) paged_warp_attend_kernel(const PagedParams p) {
  using namespace pwarp;
  using namespace prow;
  using L = pwarp::Lay<T, D>;
  constexpr int W = L::W, S = L::kStages, VW = D >= 32 ? D / 32 : 1;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ PSched sched;
  __shared__ int s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float *sq = reinterpret_cast<float *>(smem + L::kQ);
  float *sp = reinterpret_cast<float *>(smem + L::kP) + warp * kKeys * 8;
  unsigned char *ring = smem + warp * S * L::kStage;
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
    auto look_up = [&](int i) {  // this lane's page of the warp's tile i
      const long long j = key0(i) + lane;
      return i < n && j >= jlo && j < jhi ? needed_page(p.table[(long long)u.b * p.width + (int)j / p.page]) : kNotNeeded;
    };
    auto load = [&](int i, int id) {
      if (i < n) {  // uniform over the warp
        constexpr int CPR = D * (int)sizeof(T) / 16;  // 16-byte parts of a row
        const int j = (int)key0(i) + lane;
        long long off = -1;
        if (id != kNotNeeded) {
          if ((unsigned)id < (unsigned)p.npages)
            off = id * p.sp + kvh * p.sh + (long long)(j - j / p.page * p.page) * p.sr;
          else
            pflag(p, GQAW_DEV_BAD_PAGE);
        }
        unsigned char *kb = ring + (i % S) * L::kStage, *vb = kb + kKeys * L::kRowK;
#pragma unroll 8
        for (int c = lane; c < kKeys * CPR; c += 32) {
          const int r = c / CPR, part = c % CPR;
          const long long o = __shfl_sync(0xffffffffu, off, r);
          const T *ks = static_cast<const T *>(p.kp) + (o < 0 ? 0 : o), *vs = static_cast<const T *>(p.vp) + (o < 0 ? 0 : o);
          cp_async16(smem_u32(kb + r * L::kRowK + part * 16), reinterpret_cast<const char *>(ks) + part * 16, o >= 0);
          cp_async16(smem_u32(vb + r * L::kRowV + part * 16), reinterpret_cast<const char *>(vs) + part * 16, o >= 0);
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
    for (int e = tid; e < RM * D; e += L::kThreads) {
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

    float m[RM], l[RM];
    uint64_t o[RM / 2][VW];  // pairs of rows
#pragma unroll
    for (int r = 0; r < RM; ++r) m[r] = -INFINITY, l[r] = 0.f;
#pragma unroll
    for (int r = 0; r < RM / 2; ++r)
#pragma unroll
      for (int d = 0; d < VW; ++d) o[r][d] = 0ull;
    for (int i = 0; i < n; ++i) {
      const int next = look_up(i + S);
      load(i + S - 1, id);
      id = next;
      asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
      __syncwarp();
      const unsigned char *kb = ring + (i % S) * L::kStage, *vb = kb + kKeys * L::kRowK;
      uint64_t z2[RM];
#pragma unroll
      for (int r = 0; r < RM; ++r) z2[r] = 0ull;
      const T *kr = reinterpret_cast<const T *>(kb + lane * L::kRowK);
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        uint64_t k0, k1;
        if constexpr (sizeof(T) == 4) {
          const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(kr + d);
          k0 = v.x, k1 = v.y;
        } else {
          float f[4];
          lds<4>(kr + d, f);
          k0 = pk(f[0], f[1]), k1 = pk(f[2], f[3]);
        }
#pragma unroll
        for (int r = 0; r < RM; ++r) {
          const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(sq + r * D + d);
          z2[r] = fma2(q.x, k0, z2[r]);
          z2[r] = fma2(q.y, k1, z2[r]);
        }
      }
      const long long j0 = key0(i), j = j0 + lane;
      const bool inner = j0 >= jlo && j0 + kKeys - 1 <= u.qpos && (p.W == 0 || j0 >= jhi - p.W);
      float z[RM];
      bool up = false;
#pragma unroll
      for (int r = 0; r < RM; ++r) {
        const float2 f = unpk(z2[r]);
        z[r] = f.x + f.y;
        if (p.capmul != 0.f) z[r] = cap_logit(p, z[r]);
        if (!inner) {
          const long long at = u.qpos + r / g;
          if (r >= rows || j > at || j < jlo || (p.W > 0 && j <= at - p.W)) z[r] = -INFINITY;
        }
        up |= z[r] > m[r] + 8.f;
      }
      if (__any_sync(0xffffffffu, up)) {
        float f[RM];
#pragma unroll
        for (int r = 0; r < RM; ++r) {
          float mx = z[r];
#pragma unroll
          for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
          f[r] = 1.f;
          if (mx > m[r] + 8.f) {
            f[r] = exp2f(m[r] - mx);  // 0 while nothing was seen
            m[r] = mx;
            l[r] *= f[r];
          }
        }
#pragma unroll
        for (int r = 0; r < RM / 2; ++r)
#pragma unroll
          for (int d = 0; d < VW; ++d) o[r][d] = fma2(o[r][d], pk(f[2 * r], f[2 * r + 1]), 0ull);
      }
#pragma unroll
      for (int r = 0; r < RM; ++r) {
        const bool hid = !inner && z[r] == -INFINITY;
        const float pr = exp2f(z[r] - (m[r] == -INFINITY ? 0.f : m[r]));
        l[r] += pr;
        z[r] = hid ? -1.f : pr;  // hidden: its value row is not touched
      }
#pragma unroll
      for (int r = 0; r < RM; r += 4)
        *reinterpret_cast<float4 *>(sp + lane * 8 + r) = make_float4(z[r], z[r + 1], z[r + 2], z[r + 3]);
      __syncwarp();
      if (lane * VW < D) {
        const T *vr = reinterpret_cast<const T *>(vb) + lane * VW;
#pragma unroll 4
        for (int k = 0; k < kKeys; ++k) {
          float v[VW];
          if constexpr (VW == 8) {
            float a[4], b[4];
            lds<4>(vr + k * D, a);
            lds<4>(vr + k * D + 4, b);
#pragma unroll
            for (int d = 0; d < 4; ++d) v[d] = a[d], v[4 + d] = b[d];
          } else {
            lds<VW>(vr + k * D, v);
          }
          uint64_t w[RM / 2];
#pragma unroll
          for (int r = 0; r < RM / 2; r += 2) {
            const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(sp + k * 8 + 2 * r);
            w[r] = x.x, w[r + 1] = x.y;
          }
#pragma unroll
          for (int r = 0; r < RM / 2; ++r) {
            if (inner) {
#pragma unroll
              for (int d = 0; d < VW; ++d) o[r][d] = fma2(w[r], pk(v[d], v[d]), o[r][d]);
            } else {
              const float2 x = unpk(w[r]);
#pragma unroll
              for (int d = 0; d < VW; ++d) {
                float2 a = unpk(o[r][d]);
                if (x.x >= 0.f) a.x = fmaf(x.x, v[d], a.x);
                if (x.y >= 0.f) a.y = fmaf(x.y, v[d], a.y);
                if (!(x.x >= 0.f) && x.x != -1.f) a.x = x.x;  // a weight that is not a number
                if (!(x.y >= 0.f) && x.y != -1.f) a.y = x.y;
                o[r][d] = pk(a.x, a.y);
              }
            }
          }
        }
      }
      __syncwarp();  // the stage and sp are free
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // ---- the warp's state into its ring: [RM][D + 2]
    constexpr int PS = D + 2;
    float *mine = reinterpret_cast<float *>(ring);
    __syncwarp();
#pragma unroll
    for (int r = 0; r < RM; ++r) {
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], s);
      if (lane == 0) {
        mine[r * PS + D] = m[r];
        mine[r * PS + D + 1] = l[r];
      }
    }
    if (lane * VW < D) {
#pragma unroll
      for (int r = 0; r < RM / 2; ++r)
#pragma unroll
        for (int d = 0; d < VW; ++d) {
          const float2 a = unpk(o[r][d]);
          mine[2 * r * PS + lane * VW + d] = a.x;
          mine[(2 * r + 1) * PS + lane * VW + d] = a.y;
        }
    }
    __syncthreads();
    // ---- the warps' states joined
    const bool cut = u.k0 > 0 || u.k1 < u.nt;
    const int cta = blockIdx.x, cf = cut ? walk.owner(u.g0) : cta, cl = cut ? walk.owner(u.g0 + u.nt - 1) : cta;
    T *out = static_cast<T *>(p.out);
    float *part = p.partials + ((long long)cta * 2 + (cta == cf ? 1 : 0)) * 16 * PS;
    for (int e = tid; e < rows * D; e += L::kThreads) {
      const int r = e / D, d = e - r * D, tok = r / g, h = h0 + r - tok * g;
      float M = -INFINITY, A = 0.f, Z = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) M = fmaxf(M, reinterpret_cast<const float *>(smem + w * S * L::kStage)[r * PS + D]);
      const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float *x = reinterpret_cast<const float *>(smem + w * S * L::kStage) + r * PS;
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
          merge_row<D, 1>(cf, cl, d, [&](int c) { return p.partials + ((long long)c * 2 + (c == cf)) * 16 * PS + r * PS; }, M, Z, A);
          out[(u.row0 + tok) * p.os + (long long)h * D + d] = Elem<T>::store(A[0] * sink_reciprocal(Z, M, paged_sink_log2(p, h)));
        }
        if (tid == 0) p.tickets[cf] = 0u;
      }
    }
    __syncthreads();  // sq and the rings are reused by the next unit
  }
  pdl_launch_dependents();
}

}  // namespace gqaw
