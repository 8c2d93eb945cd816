// gqaw_paged_rows.cu -- the row-wise part of the paged operators: RMS norm of query and key
// heads, the rotary embedding, and the append of keys and values to the pages, in one pass
// over the new rows.
//
// For a row x of D elements (one head of one token)
//     y = x * rsqrt(mean(x^2) + eps) * w,  then pairs (y1, y2) -> (y1 c - y2 s, y2 c + y1 s)
// with c, s from row `pos` of the tables; everything in fp32, one rounding at the end.
//
// Bound: HBM.  Each row is read once and written once; the tables' row is shared by all heads
// of a token.  So a lane owns 8 consecutive elements of a head (16 or 32 bytes: one or two
// wide loads), D / 8 lanes make a row, and a warp keeps its token's cos and sin (and the
// weights) in registers while it goes over kBatch groups of heads whose loads are all issued
// before the first is used.  The mean is a butterfly over the row's lanes; the partner of a
// split pair (i, i + rd/2) sits at the same place of another lane when rd/2 is a multiple of
// 8, one shuffle per element; other widths pick it out of 8 shuffles.  A lane stores only what
// it loaded, so the norm may work in place.
// Measured on a GB300 (with what bounds each): see the table of figures at the end.
#include <atomic>

#include "gqaw_paged.cuh"

namespace gqaw {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;

template <typename T> struct Oct;  // 8 elements as stored
template <> struct Oct<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const float *s) {
    a = reinterpret_cast<const uint4 *>(s)[0];
    b = reinterpret_cast<const uint4 *>(s)[1];
  }
  __device__ __forceinline__ void store(float *d) const {
    reinterpret_cast<uint4 *>(d)[0] = a;
    reinterpret_cast<uint4 *>(d)[1] = b;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    Elem<float>::unpack(a, f);
    Elem<float>::unpack(b, f + 4);
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    a = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    b = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
  }
};
template <> struct Oct<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16 *s) { a = *reinterpret_cast<const uint4 *>(s); }
  __device__ __forceinline__ void store(__nv_bfloat16 *d) const { *reinterpret_cast<uint4 *>(d) = a; }
  __device__ __forceinline__ void get(float (&f)[8]) const { Elem<__nv_bfloat16>::unpack(a, f); }
  __device__ __forceinline__ static uint32_t pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    a = make_uint4(pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7]));
  }
};

// What one launch does with a token's heads: nq query heads (to qout), nk key heads (to kout,
// or the pages), nv value heads (to the pages).
struct RowsJob {
  int nq, nk, nv;
  bool paged;    // rows belong to sequences; keys go to the pages
  bool vec;      // the tables' rows split into whole vectors for a lane
  int chunks;    // warps per token
  long long warps;
};

// The sequence that row n belongs to: the last b with query_start[b] <= n, searched 32 ways
// at a time by the warp; -1 when there is none.
__device__ __forceinline__ int find_sequence(const PagedParams &p, int n, int lane) {
  int lo = 0, size = p.B;
  bool first = true;
  while (size > 1 || first) {
    first = false;
    const int step = (size + 31) / 32, i = lo + lane * step;
    const bool le = lane * step < size && p.qstart[i] <= n;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    if (c == 0) return -1;
    const int end = lo + size;
    lo += (c - 1) * step;
    size = min(step, end - lo);
  }
  return lo;
}

}  // namespace

template <typename T, int LPR>
__global__ void __launch_bounds__(kThreads) paged_rows_kernel(const PagedParams p, const RowsJob j) {
  constexpr int RPW = 32 / LPR, D = LPR * 8;
  const int lane = threadIdx.x & 31, lr = lane % LPR, sub = lane / LPR;
  const long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  pdl_wait();
  if (w < j.warps) {
    const int n = (int)(w / j.chunks), c0 = (int)(w - (long long)n * j.chunks) * (kBatch * RPW);
    const int heads = j.nq + j.nk + j.nv, e = lr * 8;

    // the rows themselves, ahead of the dependent look-ups
    Oct<T> x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = c0 + i * RPW + sub;
      if (h < heads) {
        const T *src = h < j.nq          ? static_cast<const T *>(p.q) + n * p.qs + h * D
                       : h < j.nq + j.nk ? static_cast<const T *>(p.k) + n * p.ks + (h - j.nq) * D
                                         : static_cast<const T *>(p.v) + n * p.vs + (h - j.nq - j.nk) * D;
        x[i].load(src + e);
      }
    }
    int b = 0;
    long long pos = 0, page_at = -1;
    bool owned = true;
    if (j.paged) {
      b = find_sequence(p, n, lane);
      owned = b >= 0;
      if (owned) {
        const int q0 = p.qstart[b], q1 = p.qstart[b + 1];
        const long long TT = (long long)p.seqlens[b] + 1;
        if (n >= q1) {
          owned = false;  // behind the last sequence
        } else if (q0 < 0 || q1 > p.N || q1 - q0 > p.max_new || TT < q1 - q0 || TT > p.max_len) {
          owned = false;
          if (lane == 0) pflag(p, GQAW_DEV_BAD_SEQLEN);
        } else {
          pos = TT - (q1 - n);
          if (c0 + kBatch * RPW > j.nq) {  // this warp has keys or values
            const int pg = (int)pos / p.page;
            const int id = p.table[(long long)b * p.width + pg];
            if ((unsigned)id < (unsigned)p.npages)
              page_at = id * p.sp + (pos - (long long)pg * p.page) * p.sr;
            else if (lane == 0)
              pflag(p, GQAW_DEV_BAD_PAGE);
          }
        }
      }
    }
    if (owned) {
      float cs[8], sn[8];
      bool turn = p.rot_dim > 0 && c0 < j.nq + j.nk;
      const int half = p.rot_dim / 2;
      if (turn) {
        if (p.pos_ids) pos = p.pos_ids[n];
        if (pos < 0 || pos >= p.rot_len) {
          turn = false;
          if (lane == 0) pflag(p, GQAW_DEV_BAD_POSITION);
        }
      }
      if (turn) {
        const T *tc = static_cast<const T *>(p.rcos) + pos * half, *ts = static_cast<const T *>(p.rsin) + pos * half;
        if (p.rot_inter) {  // pair m of this lane: elements e + 2m, e + 2m + 1, column e/2 + m
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const bool in = e + 2 * m < p.rot_dim;
            cs[2 * m] = cs[2 * m + 1] = in ? Elem<T>::load(tc[e / 2 + m]) : 1.f;
            sn[2 * m] = sn[2 * m + 1] = in ? Elem<T>::load(ts[e / 2 + m]) : 0.f;
          }
        } else if (j.vec) {
          if (e < p.rot_dim) {
            const int col = e < half ? e : e - half;
            Oct<T> u;
            u.load(tc + col);
            u.get(cs);
            u.load(ts + col);
            u.get(sn);
          }
        } else {
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            const int i = e + m, col = i < half ? i : i - half;
            cs[m] = i < p.rot_dim ? Elem<T>::load(tc[col]) : 1.f;
            sn[m] = i < p.rot_dim ? Elem<T>::load(ts[col]) : 0.f;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = c0 + i * RPW + sub;  // lanes past the heads run along: they take part in the shuffles
        const bool isq = h < j.nq, isk = !isq && h < j.nq + j.nk, on = h < heads;
        if (c0 + i * RPW >= heads) break;  // uniform over the warp
        if (c0 + i * RPW < j.nq + j.nk) {  // some row of the group is a query or a key
          float y[8];
          if (on) {
            x[i].get(y);
          } else {
#pragma unroll
            for (int m = 0; m < 8; ++m) y[m] = 0.f;
          }
          const T *wt = static_cast<const T *>(isq ? p.qw : p.kw);
          float ss = 0.f;
#pragma unroll
          for (int m = 0; m < 8; ++m) ss = fmaf(y[m], y[m], ss);
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          if (wt) {
            const float inv = __frsqrt_rn(ss * (1.f / D) + p.eps);
            Oct<T> u;
            float wf[8];
            u.load(wt + e);
            u.get(wf);
#pragma unroll
            for (int m = 0; m < 8; ++m) y[m] = y[m] * inv * wf[m];
          }
          if (turn) {
            if (p.rot_inter) {
#pragma unroll
              for (int m = 0; m < 8; m += 2) {
                if (e + m < p.rot_dim) {
                  const float y1 = y[m], y2 = y[m + 1];
                  y[m] = fmaf(y1, cs[m], -y2 * sn[m]);
                  y[m + 1] = fmaf(y2, cs[m], y1 * sn[m]);
                }
              }
            } else if (half % 8 == 0) {
              const int src = e < half ? lane + half / 8 : e < p.rot_dim ? lane - half / 8 : lane;
#pragma unroll
              for (int m = 0; m < 8; ++m) {
                const float o = __shfl_sync(0xffffffffu, y[m], src);
                if (e < half)
                  y[m] = fmaf(y[m], cs[m], -o * sn[m]);
                else if (e < p.rot_dim)
                  y[m] = fmaf(y[m], cs[m], o * sn[m]);
              }
            } else {
              float o[8];
#pragma unroll
              for (int m = 0; m < 8; ++m) {
                const int el = e + m, other = el < half ? el + half : el < p.rot_dim ? el - half : el;
                const int src = lane - lr + other / 8;
                o[m] = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const float t = __shfl_sync(0xffffffffu, y[k], src);
                  if (other % 8 == k) o[m] = t;
                }
              }
#pragma unroll
              for (int m = 0; m < 8; ++m)
                if (e + m < p.rot_dim) y[m] = fmaf(y[m], cs[m], e + m < half ? -o[m] * sn[m] : o[m] * sn[m]);
            }
          }
          if ((isq || isk) && (wt || turn)) x[i].set(y);  // otherwise the bits as they came
        }
        if (!on) continue;
        if (isq)
          x[i].store(static_cast<T *>(p.qout) + n * p.qos + h * D + e);
        else if (!j.paged)
          x[i].store(static_cast<T *>(p.kout) + n * p.kos + (h - j.nq) * D + e);
        else if (page_at >= 0)
          x[i].store(static_cast<T *>(isk ? p.kp : p.vp) + page_at + (isk ? h - j.nq : h - j.nq - j.nk) * p.sh + e);
      }
    }
  }
  pdl_launch_dependents();
}

template <typename T>
cudaError_t launch_rows_t(const PagedParams &p, const RowsJob &j, const cudaLaunchConfig_t &cfg) {
  switch (p.D) {
    case 8: return cudaLaunchKernelEx(&cfg, paged_rows_kernel<T, 1>, p, j);
    case 16: return cudaLaunchKernelEx(&cfg, paged_rows_kernel<T, 2>, p, j);
    case 32: return cudaLaunchKernelEx(&cfg, paged_rows_kernel<T, 4>, p, j);
    case 64: return cudaLaunchKernelEx(&cfg, paged_rows_kernel<T, 8>, p, j);
    case 128: return cudaLaunchKernelEx(&cfg, paged_rows_kernel<T, 16>, p, j);
    default: return cudaLaunchKernelEx(&cfg, paged_rows_kernel<T, 32>, p, j);
  }
}

// nq / nk / nv: the heads of each tensor that this launch handles (0: none).
cudaError_t launch_paged_rows(const PagedParams &p, int nq, int nk, int nv, bool paged, bool bf16, cudaStream_t stream) {
  RowsJob j;
  j.nq = nq;
  j.nk = nk;
  j.nv = nv;
  j.paged = paged;
  const int half = p.rot_dim / 2;
  j.vec = half % 8 == 0 && reinterpret_cast<uintptr_t>(p.rcos) % 16 == 0 && reinterpret_cast<uintptr_t>(p.rsin) % 16 == 0;
  const int rpw = 32 / (p.D / 8);
  j.chunks = (nq + nk + nv + kBatch * rpw - 1) / (kBatch * rpw);
  j.warps = (long long)p.N * j.chunks;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((j.warps + kThreads / 32 - 1) / (kThreads / 32)));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see pdl_wait()
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = bf16 ? launch_rows_t<__nv_bfloat16>(p, j, cfg) : launch_rows_t<float>(p, j, cfg);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace gqaw
