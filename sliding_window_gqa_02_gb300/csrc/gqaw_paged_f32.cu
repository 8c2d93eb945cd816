// gqaw_paged_f32.cu -- paged attention of at most 8 query rows per kv head over an fp32 cache
// (decode), head sizes 32, 64 and 128, with pages that tile 16 keys in whole 8-row groups.
//
// The same work as gqaw_paged_warp.cuh (its comment has the formulas and the reasons: a warp on
// its own, a reference maximum that rarely moves), which measured 2000 instructions per 32 keys
// on four warps a SM, many of them address arithmetic of the loads, and ran at a quarter of the
// memory's rate.  Here the tiles come by tensor TMA through the page table, a few instructions
// each, and are half as tall, so that more warps fit (head size 64: 12 warps with two stages each,
// 8 contexts of 8192 with 8 rows 62 us, 67 with 10 warps; three stages and 8 warps 77 before the
// sums of o by halves, 68 then with 12):
//   - a tile is 16 keys; K and V in blocks of 32 dimensions, rows of 128 bytes in the 128-byte
//     swizzle, whose exclusive-or of the 16-byte part with the row is what lets neighbouring
//     lanes read neighbouring keys without a bank conflict;
//   - z: a lane has 4 dimensions of each block (ds) for four keys (kg) and all rows; its part of the
//     queries stays in registers, and the sum over the eight lanes of a key is an exchange of
//     halves that leaves a lane one row of its keys (28 exchanges instead of a reduction each);
//   - o: half a warp has a key, 4 dimensions a lane (head size 128: the whole warp), the weights of a
//     key come as one broadcast; the halves are added at the unit's end.
// Bound: it was what shared memory returns to registers, 128 bytes a cycle: with one key and half
// of the dimensions a lane, the queries from shared memory and two dimensions of o, a tile took 448
// cycles of it, now some 160 (8 contexts of 8192 keys, 8 rows: 89 -> 62 us, 4.3 TB/s; 4 rows 55
// -> 48 us, 5.6 TB/s; head size 128, 4 rows 104 -> 92 us, 5.8 TB/s).  Now it is instruction issue
// and its latencies: 42% of the slots busy, memory 44%.
#include <atomic>

#include "gqaw_paged_attend.cuh"
#include "gqaw_paged_tc.cuh"

namespace gqaw {

namespace pf32 {

using prow::fma2;
using prow::pk;
using prow::unpk;
constexpr int kKeys = 16;
constexpr int kUnitCost = 24;  // see gqaw_paged_sched.cuh; 6 to 64 differ by 8% here

template <int D>
struct Lay {
  static constexpr int B = D / 32;                     // blocks of 32 dimensions
  static constexpr int kBlock = kKeys * 128;           // bytes of a block
  static constexpr int kStage = 2 * B * kBlock;        // K and V
  static constexpr int W = D == 128 ? 6 : D == 64 ? 12 : 8, S = D == 32 ? 4 : 2;
  static constexpr int kThreads = 32 * W;
  static constexpr int kQ = W * S * kStage;            // [8][D] fp32, scaled
  static constexpr int kP = kQ + 8 * D * 4;            // [W][16 keys][8 rows]
  static constexpr int kBars = kP + W * kKeys * 8 * 4;
  static constexpr int kTotal = kBars + W * S * 8 + 1024;  // and room to align the base
  static_assert(8 * (D + 2) * 4 <= S * kStage, "a warp's state fits in its ring");
  static_assert(kTotal + 12 * 1024 <= 232448, "shared memory");
};

}  // namespace pf32

// RM: 4 or 8 rows.
template <int D, int RM>
__global__ void __launch_bounds__(pf32::Lay<D>::kThreads, 1)
    paged_f32_decode_kernel(const PagedParams p, const __grid_constant__ PagedMaps maps) {
  using namespace pf32;
  using L = Lay<D>;
  constexpr int W = L::W, S = L::S, J = D / 32, NZ = RM / 2;
  constexpr int KS = D <= 64 ? 2 : 1, LK = 32 / KS, VW = D / LK;  // o: keys at a time, lanes of a key, dimensions of a lane
  constexpr bool QREG = RM * D / 8 <= 64;  // queries in registers
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ PSched sched;
  __shared__ int s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float *sq = reinterpret_cast<float *>(smem + L::kQ);
  float *sp = reinterpret_cast<float *>(smem + L::kP) + warp * kKeys * 8;
  unsigned char *ring = smem + warp * S * L::kStage;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kBars) + warp * S;  // this warp's stages
  if (tid == 0) {
    ptc::prefetch_map(&maps.k);
    ptc::prefetch_map(&maps.v);
  }
  if (lane == 0) {
    for (int i = 0; i < S; ++i) mbar_init(&full[i], 1);
    mbar_fence_init();
  }
  __syncwarp();
  pdl_wait();
  const PShape shp = shape_of(p, kUnitCost);
  sched_build<kKeys>(p, shp, &sched);
  PWalk<kKeys> walk(shp, &sched);
  PUnit u;
  const uint64_t pol = policy_evict_first();
  const int box = p.page < kKeys ? p.page : kKeys, nbox = kKeys / box;  // rows of a box, boxes of a tile
  int used = 0;      // tiles this warp has loaded, over its units: stage used % S, phase used / S
  bool fine = true;  // no wait of this warp has expired
  while (walk.next(shp, u)) {
    const int g = p.group, rows = u.ntok * g;
    const long long jlo = p.W > 0 && u.qpos - p.W + 1 > 0 ? u.qpos - p.W + 1 : 0, jhi = u.qpos + u.ntok;
    const int n = (u.k1 - u.k0 - warp + W - 1) / W;  // tiles of this warp: k0 + warp, k0 + warp + W, ...
    const int first = used;                          // the number of the unit's first tile
    auto key0 = [&](int i) { return (long long)(u.kt + u.k0 + warp + i * W) * kKeys; };
    // lane b < nbox looks up box b of the warp's tile i: kNotNeeded when no row attends any of its keys
    auto look_up = [&](int i) {
      const long long j = key0(i) + lane * box;
      return i < n && lane < nbox && j < jhi && j + box > jlo ? needed_page(p.table[(long long)u.b * p.width + (int)j / p.page]) : kNotNeeded;
    };
    auto load = [&](int i, int id) {
      if (i >= n) return;  // uniform over the warp
      const int st = (first + i) % S;
      const int j = (int)key0(i) + lane * box, row = j - j / p.page * p.page;
      const bool ok = (unsigned)id < (unsigned)p.npages;
      if (id != kNotNeeded && !ok) pflag(p, GQAW_DEV_BAD_PAGE);
      const uint32_t mask = __ballot_sync(0xffffffffu, ok);
      if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)(__popc(mask) * 2 * L::B * box * 128));
      for (int b = 0; b < nbox; ++b) {
        const int pid = __shfl_sync(0xffffffffu, id, b), prow_ = __shfl_sync(0xffffffffu, row, b);
        if (lane == 0 && ((mask >> b) & 1u)) {
          unsigned char *dst = ring + st * L::kStage + b * box * 128;
#pragma unroll
          for (int c = 0; c < L::B; ++c) {
            ptc::tma_load_4d(dst + c * L::kBlock, &maps.k, c * 32, prow_, u.hu, pid, &full[st], pol);
            ptc::tma_load_4d(dst + (L::B + c) * L::kBlock, &maps.v, c * 32, prow_, u.hu, pid, &full[st], pol);
          }
        }
      }
    };
    int id = look_up(0);
    for (int i = 0; i < S - 1; ++i) {
      const int next = look_up(i + 1);
      load(i, id);
      id = next;
    }
    for (int e = tid; e < RM * D; e += L::kThreads) {
      const int r = e / D, d = e - r * D, tok = r / g, hh = r - tok * g;
      sq[e] = r < rows ? static_cast<const float *>(p.q)[(u.row0 + tok) * p.qs + (long long)(u.hu * g + hh) * D + d] * p.qscale : 0.f;
    }
    __syncthreads();

    // z: a lane has four dimensions of every block (ds) of four keys (kg); its part of the queries
    // stays in registers where they allow
    const int ds = lane & 7, kg = lane >> 3;
    ulonglong2 qr[QREG ? RM : 1][J];
    if (QREG) {
#pragma unroll
      for (int r = 0; r < RM; ++r)
#pragma unroll
        for (int c = 0; c < J; ++c) qr[QREG ? r : 0][c] = *reinterpret_cast<const ulonglong2 *>(sq + r * D + c * 32 + ds * 4);
    }
    // after the sum over the lanes of a key: this lane's row, and its NZ keys
    const int row = RM == 8 ? ds : ds >> 1;
    auto key_of = [&](int i) { return ((RM == 8 ? 0 : 2 * (ds & 1)) + i) * 4 + kg; };
    float m = -INFINITY, l = 0.f;  // of the row; l of this lane's keys
    uint64_t o[RM / 2][VW];  // pairs of rows
#pragma unroll
    for (int r = 0; r < RM / 2; ++r)
#pragma unroll
      for (int d = 0; d < VW; ++d) o[r][d] = 0ull;
    for (int i = 0; i < n; ++i) {
      const int next = look_up(i + S);
      load(i + S - 1, id);
      id = next;
      const int st = (first + i) % S;
      if (!__all_sync(0xffffffffu, fine && mbar_wait(&full[st], ((first + i) / S) & 1))) fine = false;
      const unsigned char *kb = ring + st * L::kStage, *vb = kb + L::B * L::kBlock;
      float z[4][RM];  // this lane's part of four keys' logits
      auto part_of = [&](int c, int key) {
        return *reinterpret_cast<const ulonglong2 *>(kb + c * L::kBlock + key * 128 + ((ds ^ (key & 7)) << 4));
      };
      if constexpr (QREG) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint64_t z2[RM];
#pragma unroll
          for (int c = 0; c < J; ++c) {
            const ulonglong2 kv = part_of(c, k * 4 + kg);
#pragma unroll
            for (int r = 0; r < RM; ++r) {
              z2[r] = fma2(qr[r][c].x, kv.x, c ? z2[r] : 0ull);
              z2[r] = fma2(qr[r][c].y, kv.y, z2[r]);
            }
          }
#pragma unroll
          for (int r = 0; r < RM; ++r) {
            const float2 f = unpk(z2[r]);
            z[k][r] = f.x + f.y;
          }
        }
      } else {
        uint64_t z2[4][RM];
#pragma unroll
        for (int c = 0; c < J; ++c) {
          ulonglong2 kv[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) kv[k] = part_of(c, k * 4 + kg);
#pragma unroll
          for (int r = 0; r < RM; ++r) {
            const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(sq + r * D + c * 32 + ds * 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              z2[k][r] = fma2(q.x, kv[k].x, c ? z2[k][r] : 0ull);
              z2[k][r] = fma2(q.y, kv[k].y, z2[k][r]);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int r = 0; r < RM; ++r) {
            const float2 f = unpk(z2[k][r]);
            z[k][r] = f.x + f.y;
          }
      }
      // the sum over the eight lanes of a key: each step, a lane gives away the half that its
      // partner keeps
      float y[4];
      {
        float a[4][RM / 2], b[4][RM / 4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int r = 0; r < RM / 2; ++r) {
            const float mine = ds & 4 ? z[k][r + RM / 2] : z[k][r], his = ds & 4 ? z[k][r] : z[k][r + RM / 2];
            a[k][r] = mine + __shfl_xor_sync(0xffffffffu, his, 4);
          }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int r = 0; r < RM / 4; ++r) {
            const float mine = ds & 2 ? a[k][r + RM / 4] : a[k][r], his = ds & 2 ? a[k][r] : a[k][r + RM / 4];
            b[k][r] = mine + __shfl_xor_sync(0xffffffffu, his, 2);
          }
#pragma unroll
        for (int k = 0; k < NZ; ++k) {
          float mine, his;
          if constexpr (RM == 8) {
            mine = ds & 1 ? b[k][RM / 4 - 1] : b[k][0];
            his = ds & 1 ? b[k][0] : b[k][RM / 4 - 1];
          } else {
            mine = ds & 1 ? b[k + 2][0] : b[k][0];
            his = ds & 1 ? b[k][0] : b[k + 2][0];
          }
          y[k] = mine + __shfl_xor_sync(0xffffffffu, his, 1);
        }
      }
      const long long j0 = key0(i);
      const bool inner = j0 >= jlo && j0 + kKeys - 1 <= u.qpos && (p.W == 0 || j0 >= jhi - p.W);
      bool up = false;
#pragma unroll
      for (int k = 0; k < NZ; ++k) {
        if (p.capmul != 0.f) y[k] = cap_logit(p, y[k]);
        if (!inner) {
          const long long at = u.qpos + row / g, j = j0 + key_of(k);
          if (row >= rows || j > at || j < jlo || (p.W > 0 && j <= at - p.W)) y[k] = -INFINITY;
        }
        up |= y[k] > m + 8.f;
      }
      if (__any_sync(0xffffffffu, up)) {
        float mx = y[0];
#pragma unroll
        for (int k = 1; k < NZ; ++k) mx = fmaxf(mx, y[k]);
        if (RM == 4) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        float f = 1.f;
        if (mx > m + 8.f) {
          f = exp2f(m - mx);  // 0 while nothing was seen
          m = mx;
          l *= f;
        }
#pragma unroll
        for (int r = 0; r < RM / 2; ++r) {  // rows 2r and 2r + 1: of lanes with kg = 0
          const float f0 = __shfl_sync(0xffffffffu, f, 2 * r * (8 / RM)), f1 = __shfl_sync(0xffffffffu, f, (2 * r + 1) * (8 / RM));
#pragma unroll
          for (int d = 0; d < VW; ++d) o[r][d] = fma2(o[r][d], pk(f0, f1), 0ull);
        }
      }
#pragma unroll
      for (int k = 0; k < NZ; ++k) {
        const float pr = exp2f(y[k] - (m == -INFINITY ? 0.f : m));
        l += pr;
        // a hidden key: its value row is not touched
        sp[key_of(k) * 8 + row] = !inner && y[k] == -INFINITY ? -1.f : pr;
      }
      __syncwarp();
      // this lane's dimensions: VW from lane % LK * VW, of every KS-th key from lane / LK on
      const int d0 = lane % LK * VW, blk = d0 / 32, part = d0 % 32 / 4, byte = d0 % 4 * 4;
#pragma unroll
      for (int k0 = 0; k0 < kKeys; k0 += KS) {
        const int k = k0 + lane / LK;
        float v[VW];
        prow::lds<VW>(reinterpret_cast<const float *>(vb + blk * L::kBlock + k * 128 + ((part ^ (k & 7)) << 4) + byte), v);
        uint64_t w[RM / 2];
#pragma unroll
        for (int r = 0; r < RM / 2; r += 2) {
          const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(sp + k * 8 + 2 * r);
          w[r] = x.x, w[r + 1] = x.y;
        }
        if (inner) {
#pragma unroll
          for (int r = 0; r < RM / 2; ++r)
#pragma unroll
            for (int d = 0; d < VW; ++d) o[r][d] = fma2(w[r], pk(v[d], v[d]), o[r][d]);
        } else {
#pragma unroll
          for (int r = 0; r < RM / 2; ++r) {
            const float2 x = unpk(w[r]);
#pragma unroll
            for (int d = 0; d < VW; ++d) {
              float2 a = unpk(o[r][d]);
              if (x.x != -1.f) a.x = fmaf(x.x, v[d], a.x);
              if (x.y != -1.f) a.y = fmaf(x.y, v[d], a.y);
              o[r][d] = pk(a.x, a.y);
            }
          }
        }
      }
      __syncwarp();  // the stage and sp are free
    }
    used = first + (n > 0 ? n : 0);

    // ---- the warp's state into its ring: [RM][D + 2]
    constexpr int PS = D + 2;
    float *mine = reinterpret_cast<float *>(ring);
    if (RM == 4) l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 8);
    l += __shfl_xor_sync(0xffffffffu, l, 16);
    if (lane == row * (8 / RM)) {
      mine[row * PS + D] = m;
      mine[row * PS + D + 1] = l;
    }
#pragma unroll
    for (int r = 0; r < RM / 2; ++r)
#pragma unroll
      for (int d = 0; d < VW; ++d) {
        float2 a = unpk(o[r][d]);
        if (KS == 2) {
          a.x += __shfl_xor_sync(0xffffffffu, a.x, 16);
          a.y += __shfl_xor_sync(0xffffffffu, a.y, 16);
        }
        if (lane / LK == r % KS) {
          mine[2 * r * PS + lane % LK * VW + d] = a.x;
          mine[(2 * r + 1) * PS + lane % LK * VW + d] = a.y;
        }
      }
    __syncthreads();
    // ---- the warps' states joined
    const bool cut = u.k0 > 0 || u.k1 < u.nt;
    const int cta = blockIdx.x, cf = cut ? walk.owner(u.g0) : cta, cl = cut ? walk.owner(u.g0 + u.nt - 1) : cta;
    float *out = static_cast<float *>(p.out);
    float *part = p.partials + ((long long)cta * 2 + (cta == cf ? 1 : 0)) * 16 * PS;
    for (int e = tid; e < rows * D; e += L::kThreads) {
      const int r = e / D, d = e - r * D, tok = r / g, h = u.hu * g + r - tok * g;
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
        out[(u.row0 + tok) * p.os + (long long)h * D + d] = A * sink_reciprocal(Z, M, paged_sink_log2(p, h));
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
          const int r = e / D, d = e - r * D, tok = r / g, h = u.hu * g + r - tok * g;
          float M, Z, A[1];
          merge_row<D, 1>(cf, cl, d, [&](int c) { return p.partials + ((long long)c * 2 + (c == cf)) * 16 * PS + r * PS; }, M, Z, A);
          out[(u.row0 + tok) * p.os + (long long)h * D + d] = A[0] * sink_reciprocal(Z, M, paged_sink_log2(p, h));
        }
        if (tid == 0) p.tickets[cf] = 0u;
      }
    }
    // the state was written by ordinary stores where the next unit's tiles land by TMA
    tc::fence_proxy_async_smem();
    __syncthreads();  // sq and the rings are reused by the next unit
  }
  // every load that was issued has been waited for, unless a wait expired
  if (!fine) {
    if (lane == 0) {
      pflag(p, GQAW_DEV_TIMEOUT);
      for (int i = used > S ? used - S : 0; i < used; ++i) mbar_wait(&full[i % S], (i / S) & 1);
    }
  }
  pdl_launch_dependents();
}

template <int D, int RM>
cudaError_t launch_paged_f32_one(const PagedParams &p, const PagedMaps &maps, int sms, cudaStream_t stream) {
  using L = pf32::Lay<D>;
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> ready[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(paged_f32_decode_kernel<D, RM>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kTotal);
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
  e = cudaLaunchKernelEx(&cfg, paged_f32_decode_kernel<D, RM>, p, maps);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_paged_f32_decode(const PagedParams &p, const PagedMaps &maps, int rows, int sms, cudaStream_t stream) {
  switch (p.D) {
    case 32: return rows <= 4 ? launch_paged_f32_one<32, 4>(p, maps, sms, stream) : launch_paged_f32_one<32, 8>(p, maps, sms, stream);
    case 64: return rows <= 4 ? launch_paged_f32_one<64, 4>(p, maps, sms, stream) : launch_paged_f32_one<64, 8>(p, maps, sms, stream);
    default: return rows <= 4 ? launch_paged_f32_one<128, 4>(p, maps, sms, stream) : launch_paged_f32_one<128, 8>(p, maps, sms, stream);
  }
}

}  // namespace gqaw
