// gqaw_paged_rows.cu -- the row-wise part of the paged operators: RMS norm of query and key
// heads, the rotary embedding, and the append of keys and values to the pages, in one pass
// over the new rows.
//
// For a row x of D elements (one head of one token)
//     y = x * rsqrt(mean(x^2) + eps) * w,  then pairs (y1, y2) -> (y1 c - y2 s, y2 c + y1 s)
// with c, s from row `pos` of the tables; everything in fp32, one rounding at the end.
//
// Bound: HBM for many tokens, latency for few.  Each row is read once and written once; the
// tables' row and the weights are shared by all heads of a token.  So a lane owns 8 consecutive
// elements of a head (16 or 32 bytes), D / 8 lanes make a row, and what a token's heads share is
// folded once into two coefficients per element: with p the partner of element i in its pair,
//     out_i = r (x_i (w_i c_i) + x_p (w_p s_i)),   s_i = -sin for the first of a pair, sin for the
// second, and r the row's reciprocal root mean square, left for the last multiplication.  Per
// element that is one product, one multiply-add and one product, on packed pairs of fp32.
// The mean is a butterfly over the row's lanes.  The partner of a split pair (i, i + rd/2) sits
// at the same place of another lane when rd/2 is a multiple of 8: its words are exchanged as
// stored (4 shuffles for 8 bf16); other widths pick it out of the neighbours' elements.
// A warp goes over BATCH groups of heads of one tensor, whose loads are all issued before the
// first is used: 4 where there are tokens enough to fill the GPU, 2 where the chain of dependent
// look-ups (sequence, position, tables) is the time.  What hides that chain is many warps, so
// registers are the price: the usual pairing has a kernel of its own that fits 64 of them (32
// warps a SM; 4099 tokens of 40 heads of 128 in bf16: 21.9 us, 3.9 TB/s; with 8 groups and 80
// registers 23.2 us, with every pairing in one kernel 24.0, in CTAs of 256 threads 25.4; 48
// registers spill: 29).  fp32 takes 80: 33.6 us, 5.1 TB/s, against 41.8 with 64.
// A lane stores only what it loaded, so the norm may work in place.
#include <atomic>

#include "gqaw_paged.cuh"

namespace gqaw {

namespace {

constexpr int kThreads = 128;
constexpr long long kManyWarps = 152 * 16;  // 16 warps a SM

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
  __device__ __forceinline__ Oct from(int src) const {  // the octet of another lane
    Oct o;
    o.a = make_uint4(__shfl_sync(~0u, a.x, src), __shfl_sync(~0u, a.y, src), __shfl_sync(~0u, a.z, src), __shfl_sync(~0u, a.w, src));
    o.b = make_uint4(__shfl_sync(~0u, b.x, src), __shfl_sync(~0u, b.y, src), __shfl_sync(~0u, b.z, src), __shfl_sync(~0u, b.w, src));
    return o;
  }
  __device__ __forceinline__ void clear() { a = b = make_uint4(0, 0, 0, 0); }
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
  __device__ __forceinline__ Oct from(int src) const {
    Oct o;
    o.a = make_uint4(__shfl_sync(~0u, a.x, src), __shfl_sync(~0u, a.y, src), __shfl_sync(~0u, a.z, src), __shfl_sync(~0u, a.w, src));
    return o;
  }
  __device__ __forceinline__ void clear() { a = make_uint4(0, 0, 0, 0); }
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
// or the pages), nv value heads (to the pages); cq, ck, cv warps a token for each.
struct RowsJob {
  int nq, nk, nv, cq, ck, cv;
  bool paged;    // rows belong to sequences; keys go to the pages
  bool vec;      // the tables' rows split into whole vectors for a lane
  long long warps;
  int checks;    // warps behind those, which flag malformed sequences, 32 each (no row need be theirs)
};

// How a row's pairs lie for its lanes.
enum Turn { kNoTurn = 0, kOctets = 1, kInside = 2, kAnywhere = 3 };

}  // namespace

// Packed pairs of fp32: one instruction computes both lanes.
__device__ __forceinline__ uint64_t pk(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpk(uint64_t v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// The coefficients of a lane's 8 elements: x_i takes own[i], its partner takes other[i].
struct Coef {
  uint64_t own[4], other[4];
};

// BATCH groups of RPW heads of one tensor, in `x`: norm (wt), turn, store.  Heads [h, nh), D
// elements (in) and `step` elements (out) apart.  SPLIT: with `lo` not 0, what the rounding to
// bf16 leaves is stored too, that many elements on.
template <int MODE, bool SPLIT, typename T, int LPR, int BATCH>
__device__ __forceinline__ void rows_out(const PagedParams &p, Oct<T> (&x)[BATCH], const Coef &c, bool norm, T *dst,
                                         long long step, long long lo, int h, int nh, int e, int src) {
  constexpr int RPW = 32 / LPR, D = LPR * 8;
  const int lane = threadIdx.x & 31, lr = lane % LPR, half = p.rot_dim / 2;
  const int h0 = h - lane / LPR;  // the warp's first head
#pragma unroll
  for (int i = 0; i < BATCH; ++i) {
    if (h0 + i * RPW >= nh) break;  // uniform over the warp; lanes past the heads run along
    if (MODE != kNoTurn || norm) {
      float y[8];
      x[i].get(y);
      uint64_t v[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) v[m] = pk(y[2 * m], y[2 * m + 1]);
      float r = 1.f;
      if (norm) {
        uint64_t s2 = mul2(v[0], v[0]);
#pragma unroll
        for (int m = 1; m < 4; ++m) s2 = fma2(v[m], v[m], s2);
        float s0, s1;
        unpk(s2, s0, s1);
        float ss = s0 + s1;
#pragma unroll
        for (int k = LPR / 2; k > 0; k >>= 1) ss += __shfl_xor_sync(~0u, ss, k);
        r = __frsqrt_rn(ss * (1.f / D) + p.eps);
      }
      uint64_t o[4] = {0ull, 0ull, 0ull, 0ull};
      if (MODE == kInside) {
#pragma unroll
        for (int m = 0; m < 4; ++m)
          if (e + 2 * m < p.rot_dim) o[m] = pk(y[2 * m + 1], y[2 * m]);
      } else if (MODE == kOctets) {
        Oct<T> other = x[i].from(src);
        if (e >= p.rot_dim) other.clear();  // what does not turn takes nothing, not 0 times infinity
        float z[8];
        other.get(z);
#pragma unroll
        for (int m = 0; m < 4; ++m) o[m] = pk(z[2 * m], z[2 * m + 1]);
      } else if (MODE == kAnywhere) {
        float z[8];
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          const int el = e + m, at = el < half ? el + half : el < p.rot_dim ? el - half : el;
          z[m] = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float t = __shfl_sync(~0u, y[k], lane - lr + at / 8);
            if (at % 8 == k && el < p.rot_dim) z[m] = t;
          }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) o[m] = pk(z[2 * m], z[2 * m + 1]);
      }
      const uint64_t r2 = pk(r, r);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        uint64_t t = mul2(v[m], c.own[m]);
        if (MODE != kNoTurn) t = fma2(o[m], c.other[m], t);
        unpk(mul2(t, r2), y[2 * m], y[2 * m + 1]);
      }
      x[i].set(y);
      if (SPLIT && lo) {
        float z[8];
        x[i].get(z);
#pragma unroll
        for (int m = 0; m < 8; ++m) z[m] = fabsf(z[m]) < INFINITY ? y[m] - z[m] : 0.f;
        Oct<T> rest;
        rest.set(z);
        if (h + i * RPW < nh) rest.store(dst + lo + (long long)i * RPW * step);
      }
    } else if (SPLIT && lo) {
      Oct<T> rest;
      rest.clear();
      if (h + i * RPW < nh) rest.store(dst + lo + (long long)i * RPW * step);
    }
    if (h + i * RPW < nh) x[i].store(dst + (long long)i * RPW * step);
  }
}

// OCTETS: pairs lie in octets of other lanes, or nothing turns (the common case, in fewer registers).
template <bool OCTETS, bool SPLIT, typename T, int LPR, int BATCH>
__global__ void __launch_bounds__(kThreads, OCTETS && sizeof(T) == 2 ? 8 : 6)
    paged_rows_kernel(const PagedParams p, const RowsJob j) {
  constexpr int RPW = 32 / LPR, D = LPR * 8;
  const int lane = threadIdx.x & 31, lr = lane % LPR, sub = lane / LPR;
  const long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  pdl_wait();
  if (w < j.warps) {
    const int chunks = j.cq + j.ck + j.cv, n = (int)(w / chunks);
    int c = (int)(w - (long long)n * chunks);
    const int kind = c < j.cq ? 0 : c < j.cq + j.ck ? 1 : 2;  // queries, keys, values
    c -= kind == 0 ? 0 : kind == 1 ? j.cq : j.cq + j.ck;
    const int nh = kind == 0 ? j.nq : kind == 1 ? j.nk : j.nv, h = c * (BATCH * RPW) + sub, e = lr * 8;

    // the rows themselves, ahead of the dependent look-ups
    Oct<T> x[BATCH];
    const T *in = (kind == 0   ? static_cast<const T *>(p.q) + n * p.qs
                   : kind == 1 ? static_cast<const T *>(p.k) + n * p.ks
                               : static_cast<const T *>(p.v) + n * p.vs) + (long long)h * D + e;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      if (h + i * RPW < nh)
        x[i].load(in + i * RPW * D);
      else
        x[i].clear();
    }
    long long pos = 0, page_at = -1;
    bool owned = true;
    if (j.paged) {
      const int b = find_sequence(batch_of(p), n);
      owned = b >= 0;  // else nobody's, or a malformed sequence's
      if (owned) {
        pos = (long long)p.seqlens[b] + 1 - (p.qstart[b + 1] - n);
        if (kind > 0) {
          const int pg = (int)pos / p.page;
          const int id = p.table[(long long)b * p.width + pg];
          if ((unsigned)id < (unsigned)p.npages)
            page_at = id * p.sp + (pos - (long long)pg * p.page) * p.sr;
          else if (lane == 0)
            pflag(p, GQAW_DEV_BAD_PAGE);
          owned = page_at >= 0;
        }
      }
    }
    if (owned) {
      T *dst;
      long long step = D, lo = 0;
      if (kind == 0) {
        dst = static_cast<T *>(p.qout) + n * p.qos;
        if (SPLIT) lo = static_cast<const T *>(p.qlo) - static_cast<const T *>(p.qout);
      } else if (!j.paged) {
        dst = static_cast<T *>(p.kout) + n * p.kos;
      } else {
        dst = static_cast<T *>(kind == 1 ? p.kp : p.vp) + page_at;
        step = p.sh;
      }
      dst += h * step + e;
      const T *wt = static_cast<const T *>(kind == 0 ? p.qw : kind == 1 ? p.kw : nullptr);
      const int half = p.rot_dim / 2;
      bool turn = p.rot_dim > 0 && kind < 2;
      if (turn) {
        if (p.pos_ids) pos = p.pos_ids[n];
        if (pos < 0 || pos >= p.rot_len) {
          turn = false;
          if (lane == 0) pflag(p, GQAW_DEV_BAD_POSITION);
        }
      }
      const int mode = !turn ? kNoTurn : OCTETS ? kOctets : p.rot_inter ? kInside : half % 8 == 0 ? kOctets : kAnywhere;
      float cs[8], sn[8], wo[8], wp[8];
#pragma unroll
      for (int m = 0; m < 8; ++m) cs[m] = 1.f, sn[m] = 0.f, wo[m] = wp[m] = 1.f;
      if (turn && e < p.rot_dim) {
        const T *tc = static_cast<const T *>(p.rcos) + pos * half, *ts = static_cast<const T *>(p.rsin) + pos * half;
        if (mode == kInside) {  // pair m of this lane: elements e + 2m, e + 2m + 1, column e/2 + m
#pragma unroll
          for (int m = 0; m < 4; ++m)
            if (e + 2 * m < p.rot_dim) {
              cs[2 * m] = cs[2 * m + 1] = Elem<T>::load(tc[e / 2 + m]);
              sn[2 * m + 1] = Elem<T>::load(ts[e / 2 + m]);
              sn[2 * m] = -sn[2 * m + 1];
            }
        } else if (j.vec) {
          const int col = e < half ? e : e - half;
          Oct<T> u;
          u.load(tc + col);
          u.get(cs);
          u.load(ts + col);
          u.get(sn);
          if (e < half)
#pragma unroll
            for (int m = 0; m < 8; ++m) sn[m] = -sn[m];
        } else {
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            const int i = e + m, col = i < half ? i : i - half;
            if (i < p.rot_dim) {
              cs[m] = Elem<T>::load(tc[col]);
              sn[m] = Elem<T>::load(ts[col]);
              if (i < half) sn[m] = -sn[m];
            }
          }
        }
      }
      // first element of the partner octet, and the lane that holds it
      const int pe = mode != kOctets || e >= p.rot_dim ? e : e < half ? e + half : e - half, src = lane - lr + pe / 8;
      if (wt) {
        Oct<T> u;
        u.load(wt + e);
        u.get(wo);
        if (mode == kInside) {
#pragma unroll
          for (int m = 0; m < 8; ++m) wp[m] = wo[m ^ 1];
        } else if (mode == kOctets) {
          u.load(wt + pe);
          u.get(wp);
        } else if (mode == kAnywhere) {
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            const int i = e + m;
            wp[m] = Elem<T>::load(wt[i < half ? i + half : i < p.rot_dim ? i - half : i]);
          }
        }
      }
      Coef c;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        c.own[m] = pk(wo[2 * m] * cs[2 * m], wo[2 * m + 1] * cs[2 * m + 1]);
        c.other[m] = pk(wp[2 * m] * sn[2 * m], wp[2 * m + 1] * sn[2 * m + 1]);
      }
      // one loop for each way, so that the one taken is short
      switch (mode) {
        case kNoTurn: rows_out<kNoTurn, SPLIT, T, LPR, BATCH>(p, x, c, wt != nullptr, dst, step, lo, h, nh, e, src); break;
        case kOctets: rows_out<kOctets, SPLIT, T, LPR, BATCH>(p, x, c, wt != nullptr, dst, step, lo, h, nh, e, src); break;
        case kInside: if (!OCTETS) rows_out<kInside, SPLIT, T, LPR, BATCH>(p, x, c, wt != nullptr, dst, step, lo, h, nh, e, src); break;
        default: if (!OCTETS) rows_out<kAnywhere, SPLIT, T, LPR, BATCH>(p, x, c, wt != nullptr, dst, step, lo, h, nh, e, src);
      }
    }
  } else if (w < j.warps + j.checks) {
    const int b = (int)(w - j.warps) * 32 + lane;
    if (b < p.B && malformed(batch_of(p), p.qstart[b], p.qstart[b + 1], p.seqlens[b])) pflag(p, GQAW_DEV_BAD_SEQLEN);
  }
  pdl_launch_dependents();
}

template <bool OCTETS, bool SPLIT, typename T, int BATCH>
cudaError_t launch_rows_t(const PagedParams &p, const RowsJob &j, const cudaLaunchConfig_t &cfg) {
  switch (p.D) {
    case 8: return cudaLaunchKernelEx(&cfg, paged_rows_kernel<OCTETS, SPLIT, T, 1, BATCH>, p, j);
    case 16: return cudaLaunchKernelEx(&cfg, paged_rows_kernel<OCTETS, SPLIT, T, 2, BATCH>, p, j);
    case 32: return cudaLaunchKernelEx(&cfg, paged_rows_kernel<OCTETS, SPLIT, T, 4, BATCH>, p, j);
    case 64: return cudaLaunchKernelEx(&cfg, paged_rows_kernel<OCTETS, SPLIT, T, 8, BATCH>, p, j);
    case 128: return cudaLaunchKernelEx(&cfg, paged_rows_kernel<OCTETS, SPLIT, T, 16, BATCH>, p, j);
    default: return cudaLaunchKernelEx(&cfg, paged_rows_kernel<OCTETS, SPLIT, T, 32, BATCH>, p, j);
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
  auto chunks = [&](int heads, int batch) { return (heads + batch * rpw - 1) / (batch * rpw); };
  const int deep = 4;  // 64 bytes of loads a lane, or 128 of fp32
  const bool many = (long long)p.N * (chunks(nq, deep) + chunks(nk, deep) + chunks(nv, deep)) >= kManyWarps;
  const int batch = many ? deep : 2;
  j.cq = chunks(nq, batch);
  j.ck = chunks(nk, batch);
  j.cv = chunks(nv, batch);
  j.warps = (long long)p.N * (j.cq + j.ck + j.cv);
  cudaLaunchConfig_t cfg = {};
  j.checks = paged ? (p.B + 31) / 32 : 0;
  cfg.gridDim = dim3((unsigned)((j.warps + j.checks + kThreads / 32 - 1) / (kThreads / 32)));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see pdl_wait()
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // p.qlo: a variant of its own, for the rows that need no second part are 6% slower with the choice inside
  const bool octets = !p.rot_inter && half % 8 == 0;
  cudaError_t e;
  if (!bf16)
    e = !many ? launch_rows_t<false, false, float, 2>(p, j, cfg)
        : octets ? launch_rows_t<true, false, float, 4>(p, j, cfg) : launch_rows_t<false, false, float, 4>(p, j, cfg);
  else if (p.qlo)
    e = !many ? launch_rows_t<false, true, __nv_bfloat16, 2>(p, j, cfg)
        : octets ? launch_rows_t<true, true, __nv_bfloat16, 4>(p, j, cfg) : launch_rows_t<false, true, __nv_bfloat16, 4>(p, j, cfg);
  else
    e = !many ? launch_rows_t<false, false, __nv_bfloat16, 2>(p, j, cfg)
        : octets ? launch_rows_t<true, false, __nv_bfloat16, 4>(p, j, cfg) : launch_rows_t<false, false, __nv_bfloat16, 4>(p, j, cfg);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace gqaw
