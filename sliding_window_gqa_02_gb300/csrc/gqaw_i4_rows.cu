// gqaw_i4_rows.cu -- the row-wise part of the operators on 4-bit caches: the append (norm, turn,
// quantize), the queries of a whole step (norm, turn), and reading rows back.
//
// Append, for the D elements x of one head of one token:
//     r = 1 / sqrt(mean(x^2) + eps), y = (x r) w; pairs (y1, y2) -> (y1 c - y2 s, y2 c + y1 s)
//     a = max |y| over 32 elements, s = a / 7 rounded up to five significant bits
//     c = 8 + round(y / s)
// A code is a decision: an element next to the border between two codes falls to either side with the
// last bit of y, and then it is off by a whole step.  So y does not depend on the order of a sum or
// on which products are contracted: the sum of squares is kept in two numbers (48 bits, errors of
// sums and products carried along), r is rounded once, and every other operation is one IEEE
// operation.  The same for queries, so that a step's are those of any other implementation.
//
// Bound: the append by its instructions for many tokens (some 360 for 256 elements; 2689 tokens of 8 key
// and 8 value heads of 128 in bf16 14 us, 70% of the issue slots), by latency for few (32 tokens of a step 5.6
// us).  A lane has 8 consecutive elements of a head (16 or 32 bytes in, 4 bytes out), D / 8 lanes a row; a
// group's maximum is two exchanges among four lanes.  With 32 elements a lane the scale and the steps of the
// sum are computed once and not by four lanes: the 2689 tokens take 12.7 us, but the 32 take 7.0, since a lane's
// chain of operations is longer; the short one stands.
// Reading back is the inverse, a warp for keys and values of a token, whose look-ups were most of its
// instructions: 32768 tokens, 38 MB in and 134 MB out, in 31 us (38 with a warp for each, 5.5 TB/s).
#include "gqaw_i4_tiles.cuh"

namespace gqaw {

namespace i4r {

constexpr int kThreads = 128;
constexpr long long kManyWarps = 152 * 16;  // 16 warps a SM

// Eight elements as stored.
template <typename T> struct Oct;
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
  __device__ __forceinline__ void ones() { a = b = make_uint4(0x3f800000u, 0x3f800000u, 0x3f800000u, 0x3f800000u); }
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
  __device__ __forceinline__ void ones() { a = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u); }
};

// What one launch does with a token's heads: nq query heads (to qout), nk key and nv value heads (to
// the pages); cq, ck, cv warps a token for each.
struct Job {
  int nq, nk, nv, cq, ck, cv;
  bool vec;    // the tables' rows split into whole vectors for a lane
  int batch;   // groups of a warp
  long long warps;
  int checks;  // warps behind those, which flag malformed sequences, 32 each
};

// Packed pairs of fp32: one instruction computes both lanes, each operation rounded by itself.
__device__ __forceinline__ uint64_t pk(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpk(uint64_t v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
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
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) { return fma2(b, 0xbf800000bf800000ull, a); }

// s + e += x, the error of the sum kept (Knuth's two-sum).
__device__ __forceinline__ void add_two(float &s, float &e, float x) {
  const float t = __fadd_rn(s, x), z = __fsub_rn(t, s);
  e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(x, z)));
  s = t;
}
__device__ __forceinline__ void add_two2(uint64_t &s, uint64_t &e, uint64_t x) {
  const uint64_t t = add2(s, x), z = sub2(t, s);
  e = add2(e, add2(sub2(s, sub2(t, z)), sub2(x, z)));
  s = t;
}

// 1 / sqrt(mean of the row's squares + eps), rounded once to fp32 but for ties within 2^-20 of a
// step.  All lanes of the warp call it; LPR lanes hold a row.  EXACT: squares are fp32 numbers (bf16).
template <int LPR, bool EXACT>
__device__ __forceinline__ float row_factor(const float (&x)[8], float eps) {
  // (products that a sum follows are scalar: the packed ones may be contracted with it)
  auto square = [&](int m) { return pk(__fmul_rn(x[m], x[m]), __fmul_rn(x[m + 1], x[m + 1])); };
  uint64_t v = pk(x[0], x[1]), s2 = square(0), e2 = EXACT ? 0ull : fma2(v, v, sub2(0ull, s2));
#pragma unroll
  for (int m = 2; m < 8; m += 2) {
    v = pk(x[m], x[m + 1]);
    const uint64_t sq = square(m);
    if (!EXACT) e2 = add2(e2, fma2(v, v, sub2(0ull, sq)));
    add_two2(s2, e2, sq);
  }
  float s, e, sb, eb;
  unpk(s2, s, sb);
  unpk(e2, e, eb);
  e = __fadd_rn(e, eb);
  add_two(s, e, sb);
#pragma unroll
  for (int k = LPR / 2; k > 0; k >>= 1) {
    const float so = __shfl_xor_sync(~0u, s, k), eo = __shfl_xor_sync(~0u, e, k);
    // both partners take the sums in the same order, so that they stay alike
    const bool low = (threadIdx.x & k) == 0;
    float a = low ? s : so;
    e = __fadd_rn(e, eo);
    add_two(a, e, low ? so : s);
    s = a;
  }
  s *= 1.f / (LPR * 8);
  e *= 1.f / (LPR * 8);
  add_two(s, e, eps);
  const float hi = __fadd_rn(s, e), lo = __fadd_rn(__fsub_rn(s, hi), e);
  const float r0 = rsqrtf(hi);
  // Newton's step: r = r0 + r0 (1 - (hi + lo) r0^2) / 2
  const float ph = __fmul_rn(r0, r0), pl = fmaf(r0, r0, -ph);
  float t = fmaf(-hi, ph, 1.f);
  t = fmaf(-hi, pl, t);
  t = fmaf(-lo, ph, t);
  float r = fmaf(0.5f * r0, t, r0);
  // squares outside the range of fp32, zeros, and what is not finite: in 64 bits
  const bool plain = hi > 1e-30f && hi < 1e30f;
  if (__any_sync(~0u, !plain)) {
    double d = 0.0;
#pragma unroll
    for (int m = 0; m < 8; ++m) d += (double)x[m] * (double)x[m];
#pragma unroll
    for (int k = LPR / 2; k > 0; k >>= 1) d += __shfl_xor_sync(~0u, d, k);
    if (!plain) r = (float)(1.0 / sqrt(d / (LPR * 8) + (double)eps));
  }
  return r;
}

// The larger magnitude; a NaN stays.
__device__ __forceinline__ float max_abs(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// Codes of a lane's 8 elements, and the scale of the 32 that it shares with three other lanes.
//
// The quotient y / s is rounded correctly by Markstein's theorem (1990): with r = 1 / s rounded
// correctly and q = y r rounded, q + (y - q s) r is the rounded quotient, the residue exact in one multiply-add.
// Adding 1.5 2^23 + 8 rounds it to an integer, halves to even, whose last four bits are the code.
__device__ __forceinline__ uint32_t quantize(const float (&y)[8], uint32_t &scale) {
  float top = max_abs(max_abs(max_abs(y[0], y[1]), max_abs(y[2], y[3])), max_abs(max_abs(y[4], y[5]), max_abs(y[6], y[7])));
  top = max_abs(top, __shfl_xor_sync(~0u, top, 1));
  top = max_abs(top, __shfl_xor_sync(~0u, top, 2));
  // up to four stored bits of the mantissa: the other 19 of the 23, rounded up
  const uint32_t bits = __float_as_uint(top);
  constexpr float kSeventh = 1.f / 7.f;
  const float seventh = __fmul_rn(top, kSeventh);
  scale = (__float_as_uint(fmaf(fmaf(-seventh, 7.f, top), kSeventh, seventh)) + 0x7ffffu) & ~0x7ffffu;
  const bool plain = top > 1e-29f && top < 1e30f;  // 1 / s and the residues are normal numbers
  if (!plain) scale = bits >= 0x7f800000u ? 0x7fc00000u : (__float_as_uint(__fdiv_rn(top, 7.f)) + 0x7ffffu) & ~0x7ffffu;
  const float s = __uint_as_float(scale);
  uint32_t word = 0;
  const float r = __frcp_rn(plain ? s : 1.f);
  const uint64_t r2 = pk(r, r), ns2 = pk(-s, -s), c2 = pk(12582920.f, 12582920.f);
#pragma unroll
  for (int m = 0; m < 8; m += 2) {
    const uint64_t v = pk(y[m], y[m + 1]), q = mul2(v, r2), t = add2(fma2(fma2(q, ns2, v), r2, q), c2);
    float a, b;
    unpk(t, a, b);
    // what stands above the last four bits is the same for all: taken off below
    word += __float_as_uint(a) * (1u << (4 * m)) + __float_as_uint(b) * (16u << (4 * m));
  }
  word -= 0x4b400000u * 0x11111111u;
  if (__any_sync(~0u, !plain)) {
    uint32_t w = 0;
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      const float q = fminf(fmaxf(rintf(__fdiv_rn(y[m], s)), -7.f), 7.f);
      const uint32_t c = s > 0.f ? (uint32_t)((int)q + 8) : 8u;
      w |= c << (4 * m);
    }
    if (!plain) word = w;
  }
  return word;
}

// The other element of each pair that turns, for a lane's elements e, e + 1, ... of a row.
template <int LPR>
__device__ __forceinline__ void partners(const float (&y)[8], float (&z)[8], int e, int rot_dim, bool inter) {
  const int lane = threadIdx.x & 31, first = lane - lane % LPR, half = rot_dim / 2;
  if (inter) {
#pragma unroll
    for (int m = 0; m < 8; ++m) z[m] = y[m ^ 1];
  } else if (half % 8 == 0) {
    const int src = first + (e >= rot_dim ? e : e < half ? e + half : e - half) / 8;
#pragma unroll
    for (int m = 0; m < 8; ++m) z[m] = __shfl_sync(~0u, y[m], src);
  } else {
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      const int el = e + m, at = el < half ? el + half : el < rot_dim ? el - half : el;
      z[m] = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float t = __shfl_sync(~0u, y[k], first + at / 8);
        if (at % 8 == k) z[m] = t;
      }
    }
  }
}

}  // namespace i4r

// A warp has `batch` groups of 32 / LPR heads of one tensor of one token, one after the other (unrolled four times
// the loop ran out of the instruction cache), the next one's elements on their way.
template <typename T, int LPR>
__global__ void __launch_bounds__(i4r::kThreads, 5) i4_append_kernel(const I4Params p, const i4r::Job j) {
  using namespace i4r;
  constexpr int RPW = 32 / LPR, D = LPR * 8;
  const int lane = threadIdx.x & 31, lr = lane % LPR, sub = lane / LPR, e = lr * 8;
  const long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  pdl_wait();
  if (w < j.warps) {
    const int chunks = j.cq + j.ck + j.cv, n = (int)((uint32_t)w / (uint32_t)chunks);  // fewer than 2^31 rows
    int c = (int)w - n * chunks;
    const int kind = c < j.cq ? 0 : c < j.cq + j.ck ? 1 : 2;  // queries, keys, values
    c -= kind == 0 ? 0 : kind == 1 ? j.cq : j.cq + j.ck;
    const int nh = kind == 0 ? j.nq : kind == 1 ? j.nk : j.nv, first = c * (j.batch * RPW), h = first + sub;
    const int groups = min(j.batch, (nh - first + RPW - 1) / RPW);
    // the rows themselves, ahead of the dependent look-ups; lanes past the heads run along on ones
    Oct<T> x;
    x.ones();
    const T *in = (kind == 0   ? static_cast<const T *>(p.q) + n * p.qs
                   : kind == 1 ? static_cast<const T *>(p.k) + n * p.ks
                               : static_cast<const T *>(p.v) + n * p.vs) + (long long)h * D + e;
    if (h < nh) x.load(in);
    const int b = find_sequence(batch_of(p), n);
    if (b >= 0) {  // else nobody's, or a malformed sequence's
      long long pos = (long long)p.seqlens[b] + 1 - (p.qstart[b + 1] - n);
      I4Place at{0, 0};
      if (kind > 0) {
        at = i4_place(p, b, pos);
        if (at.page < 0 && lane == 0) pflag(p, GQAW_DEV_BAD_PAGE);
      }
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
      float cs[8], sn[8], wo[8];
#pragma unroll
      for (int m = 0; m < 8; ++m) cs[m] = 1.f, sn[m] = 0.f;
      if (turn) {  // the second factor with the sign that the product has
        const T *tc = static_cast<const T *>(p.rcos) + pos * half, *ts = static_cast<const T *>(p.rsin) + pos * half;
        if (j.vec) {
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
            const int i = e + m, col = p.rot_inter ? i / 2 : i < half ? i : i - half;
            if (i < p.rot_dim) {
              cs[m] = Elem<T>::load(tc[col]);
              sn[m] = Elem<T>::load(ts[col]);
            }
          }
        }
#pragma unroll
        for (int m = 0; m < 8; ++m)
          if (p.rot_inter ? m % 2 == 0 : e + m < half) sn[m] = -sn[m];
      }
      if (wt) {
        Oct<T> u;
        u.load(wt + e);
        u.get(wo);
      }
      if (at.page >= 0) {
#pragma unroll 1
        for (int i = 0; i < groups; ++i) {
          float y[8];
          x.get(y);
          x.ones();
          if (i + 1 < groups && h + (i + 1) * RPW < nh) x.load(in + (i + 1) * RPW * D);
          if (wt) {
            const float r = row_factor<LPR, sizeof(T) == 2>(y, p.eps);
            const uint64_t r2 = pk(r, r);
#pragma unroll
            for (int m = 0; m < 8; m += 2) unpk(mul2(mul2(pk(y[m], y[m + 1]), r2), pk(wo[m], wo[m + 1])), y[m], y[m + 1]);
          }
          if (turn) {
            float z[8];
            partners<LPR>(y, z, e, p.rot_dim, p.rot_inter != 0);
#pragma unroll
            for (int m = 0; m < 8; ++m) {  // scalar: packed products may be contracted with the sum
              const float a = __fadd_rn(__fmul_rn(y[m], cs[m]), __fmul_rn(z[m], sn[m]));
              if (e + m < p.rot_dim) y[m] = a;
            }
          }
          const int head = h + i * RPW;
          if (kind == 0) {
            Oct<T> o;
            o.set(y);
            T *dst = static_cast<T *>(p.qout) + n * p.qos + (long long)head * D + e;
            if (head < nh) o.store(dst);
            if (p.qlo) {  // bf16: what the rounding leaves
              float z[8];
              o.get(z);
#pragma unroll
              for (int m = 0; m < 8; ++m) z[m] = fabsf(z[m]) < INFINITY ? __fsub_rn(y[m], z[m]) : 0.f;
              o.set(z);
              if (head < nh) o.store(dst + (static_cast<const T *>(p.qlo) - static_cast<const T *>(p.qout)));
            }
          } else {
            uint32_t scale;
            const uint32_t word = quantize(y, scale);
            if (head < nh) {
              unsigned char *codes = static_cast<unsigned char *>(kind == 1 ? p.kp : p.vp) + at.page * p.sp + head * p.sh + at.row * p.sr;
              *reinterpret_cast<uint32_t *>(codes + lr * 4) = word;
              if (lr % 4 == 0)
                (kind == 1 ? p.kscale : p.vscale)[at.page * p.tp + head * p.th + at.row * p.tr + lr / 4] = (uint16_t)(scale >> 16);
            }
          }
        }
      }
    }
  } else if (w < j.warps + j.checks) {
    const int b = (int)(w - j.warps) * 32 + lane;
    if (b < p.B && malformed(batch_of(p), p.qstart[b], p.qstart[b + 1], p.seqlens[b])) pflag(p, GQAW_DEV_BAD_SEQLEN);
  }
  pdl_launch_dependents();
}

// A warp has `BATCH` groups of 32 / LPR heads of one token, keys and values.
template <typename T, int LPR, int BATCH>
__global__ void __launch_bounds__(i4r::kThreads) i4_read_kernel(const I4Params p, const i4r::Job j) {
  using namespace i4r;
  constexpr int RPW = 32 / LPR, D = LPR * 8;
  const int lane = threadIdx.x & 31, lr = lane % LPR, sub = lane / LPR;
  const long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  pdl_wait();
  if (w < j.warps) {
    const int n = (int)((uint32_t)w / (uint32_t)j.ck), h = ((int)w - n * j.ck) * (BATCH * RPW) + sub;
    const int b = find_sequence(batch_of(p), n);
    if (b >= 0) {
      const I4Place at = i4_place(p, b, (long long)p.seqlens[b] + 1 - (p.qstart[b + 1] - n));
      if (at.page >= 0) {
        const long long code = at.page * p.sp + at.row * p.sr + lr * 4, scale = at.page * p.tp + at.row * p.tr + lr / 4;
        uint32_t word[2][BATCH], s[2][BATCH];
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
          for (int i = 0; i < BATCH; ++i) {
            const int head = h + i * RPW;
            const bool have = head < (v ? j.nv : j.nk);
            word[v][i] = have ? *reinterpret_cast<const uint32_t *>(static_cast<const unsigned char *>(v ? p.vp : p.kp) + code + head * p.sh) : 0u;
            s[v][i] = have ? (v ? p.vscale : p.kscale)[scale + head * p.th] : 0u;
          }
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
          for (int i = 0; i < BATCH; ++i) {
            const int head = h + i * RPW;
            Oct<T> o;
            if constexpr (sizeof(T) == 2) {  // a product of two bf16 numbers, rounded once
              o.a = i4t::values8<false>(word[v][i], s[v][i] * 0x10001u, 0u, true);
            } else {
              float y[8];
#pragma unroll
              for (int m = 0; m < 8; ++m)  // 2^23 + c less 2^23 + 8
                y[m] = (__uint_as_float(((word[v][i] >> (4 * m)) & 15u) | 0x4b000000u) - 8388616.f) * __uint_as_float(s[v][i] << 16);
              o.set(y);
            }
            if (head < (v ? j.nv : j.nk)) o.store((v ? static_cast<T *>(p.vo) + n * p.vos : static_cast<T *>(p.ko) + n * p.kos) + (long long)head * D + lr * 8);
          }
      } else if (lane == 0) {
        pflag(p, GQAW_DEV_BAD_PAGE);
      }
    }
  } else if (w < j.warps + j.checks) {
    const int b = (int)(w - j.warps) * 32 + lane;
    if (b < p.B && malformed(batch_of(p), p.qstart[b], p.qstart[b + 1], p.seqlens[b])) pflag(p, GQAW_DEV_BAD_SEQLEN);
  }
  pdl_launch_dependents();
}

namespace i4r {

template <bool READ, typename T, int LPR>
cudaError_t launch(const I4Params &p, const Job &j, const cudaLaunchConfig_t &cfg) {
  if constexpr (READ)
    return j.batch == 4 ? cudaLaunchKernelEx(&cfg, i4_read_kernel<T, LPR, 4>, p, j) : cudaLaunchKernelEx(&cfg, i4_read_kernel<T, LPR, 2>, p, j);
  else
    return cudaLaunchKernelEx(&cfg, i4_append_kernel<T, LPR>, p, j);
}

template <bool READ, typename T>
cudaError_t launch_d(const I4Params &p, const Job &j, const cudaLaunchConfig_t &cfg) {
  switch (p.D) {
    case 32: return launch<READ, T, 4>(p, j, cfg);
    case 64: return launch<READ, T, 8>(p, j, cfg);
    case 128: return launch<READ, T, 16>(p, j, cfg);
    default: return launch<READ, T, 32>(p, j, cfg);
  }
}

}  // namespace i4r

// nq: query heads to norm and turn (0: none); nk, nv: key and value heads to append, or to read.
cudaError_t launch_i4_rows(const I4Params &p, int nq, int nk, int nv, bool read, bool bf16, cudaStream_t stream) {
  using namespace i4r;
  Job j;
  j.nq = nq;
  j.nk = nk;
  j.nv = nv;
  const int half = p.rot_dim / 2;
  j.vec = !p.rot_inter && half % 8 == 0 && reinterpret_cast<uintptr_t>(p.rcos) % 16 == 0 && reinterpret_cast<uintptr_t>(p.rsin) % 16 == 0;
  const int rpw = 32 / (p.D / 8);
  auto chunks = [&](int heads, int batch) { return (heads + batch * rpw - 1) / (batch * rpw); };
  auto warps = [&](int batch) {  // a warp that reads has a token's keys and values
    return (long long)p.N * (read ? chunks(nk > nv ? nk : nv, batch) : chunks(nq, batch) + chunks(nk, batch) + chunks(nv, batch));
  };
  j.batch = read ? (warps(4) >= kManyWarps ? 4 : 2) : warps(4) >= kManyWarps ? 4 : warps(2) >= kManyWarps ? 2 : 1;
  j.cq = chunks(nq, j.batch);
  j.ck = chunks(read && nv > nk ? nv : nk, j.batch);
  j.cv = read ? 0 : chunks(nv, j.batch);
  j.warps = warps(j.batch);
  j.checks = (p.B + 31) / 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((j.warps + j.checks + kThreads / 32 - 1) / (kThreads / 32)));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see pdl_wait()
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = read ? (bf16 ? launch_d<true, __nv_bfloat16>(p, j, cfg) : launch_d<true, float>(p, j, cfg))
                             : (bf16 ? launch_d<false, __nv_bfloat16>(p, j, cfg) : launch_d<false, float>(p, j, cfg));
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gqaw
