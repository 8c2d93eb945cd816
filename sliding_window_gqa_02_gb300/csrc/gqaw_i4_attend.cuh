// gqaw_i4_attend.cuh -- attention over a paged cache held in 4 bits, 8 query rows of a kv head at once
// (fp32: 16).
//
//     o_i = sum_j softmax_j(cap(scale q_i k_j)) v_j,  j <= i (and j > i - W), with sinks,
// k = (c - 8) s and v likewise, c the code of an element and s the scale of its 32 elements.
//
// Bound: HBM (72 bytes a row of 128), if what a byte costs in instructions stays below what the SM
// issues meanwhile: at 44 bytes a ns and SM a warp instruction is there for every 2 codes.  So
//   - codes go from shared memory to registers once and are matrix operands as they are: a nibble
//     in the low bits of an fp16 is the subnormal number c 2^-24, one in the next four bits 16 c 2^-24,
//     which the tensor cores take exactly; one AND makes two operands of two nibbles of a word, and the
//     factor of 16 goes to the query.  Converting to bf16 through shared memory, as the
//     5th-generation tensor cores would need it, costs four bytes there for every byte of codes,
//     written and read again: more than its 128 bytes a cycle at the rate of HBM.  (Where several units
//     share their keys through L2, as 32 rows a kv head do, that would not bind: at 0.75 TB/s a seventh of the time.)
//     Hence mma.sync with the keys (dimensions) as M, whose operands are registers, 8 query rows as N; its
//     rate, a product of 16 x 8 x 16 every 2 cycles of an SM, is 2.4 times what the memory feeds;
//   - z = sum over groups g of s_g (sum_d c_d q_d - 8 sum_d q_d): the scale multiplies a group's sum in fp32,
//     and the sum of the queries is where the accumulator starts;
//   - the values are (c - 8) s in fp16: a nibble in the upper bits of the mantissa of 16 is 16 + c, and
//     (16 + c) s - 24 s one multiply-add, exact since 24 s is a number of fp16 (1032 s, of a nibble in the
//     lower bits, is not); a lane's dimensions (16 of 128) share a scale.  (The 8 does not wait for the
//     end as with the keys: 8 sum p s beside a small result would take its last bits.)
//
// Queries come as one or two parts of fp16 (QP; fp32, or turned bf16: two), after a power of two per
// row that puts the largest element at 2^13; weights as one part, or two for fp32 (PP).  A weight is at
// most 2^15, since the row's reference moves when that is exceeded (and then puts the largest at 2^13); a
// value scale is taken relative to the largest power of two of its group so far, which becomes 2^10: no
// product leaves fp16, and with scales up to 2^24 apart each is exact.  What a row does not attend must not
// change it, however large, so scales farther off count as zero there, and the rows that attend them are
// computed again in fp32 (wide_rows()).  Sums and statistics are fp32.  The tensor cores cut what a sum loses,
// which adds up over a long context: for fp32 rows (kExact) the codes of the keys are signed, so that no large
// sum is taken back, a product's values are added outside, the smaller parts come first, and exponents are
// taken near 0 (error against 64 bits at 500 to 12,000 keys 9.6e-7 -> 2e-7, the time the same).  The reference
// moves by whole powers of two and is never rounded.
//
// Each warp works on its own, on tiles of 32 keys through a ring of its own; no barrier of the CTA
// falls inside a unit.  Tiles come by cp.async through the page table, any page size and strides; with
// pages of 16 rows a tile by tensor TMA and bulk copies is eight copies, whose operands took 300
// instructions, and every lane's own look-ups 200.  A unit's first tiles are under way before the last
// unit's rows go out.  Schedule, splits and merges: gqaw_paged.cuh.
//
// Measured: 64 contexts of 4 k to 33 k keys (8 kv heads of 128, 4 query heads each) 262 us, 3.98 TB/s or 59% of
// the copy rate: issue slots are 43 to 52% busy with some 337 instructions for 16 keys of a warp (148 of them keys
// and softmax, 128 values, 37 scales, 24 loads), 12 warps a SM hide no more of each other's latencies, and registers
// (168) allow no more.  A unit's start and end are 4 to 6 us, the schedule 2, a cut 3.5.
//
// Which of 8 rows is which: position x of 8 is key kappa(x) of a tile's, chosen so that the rows of
// the even positions lie in different banks when four lanes read their dimensions of them.
//
// A value scale that is not finite counts as zero in the products, and the tokens that attend it are
// marked: their outputs of that group are NaN, nobody else's.
#pragma once

#include <atomic>
#include <type_traits>

#include "gqaw_i4.cuh"
#include "gqaw_paged_tc.cuh"

namespace gqaw {

namespace i4a {

constexpr int kKeys = 32;      // a warp's tile
// See gqaw_paged_sched.cuh.  20 to 48 tiles a unit, and 32 or 60 a cut, differ by 2%, but for 16 contexts of 8192
// keys and 8 heads, whose units are better whole (58 us with 32, 52 with 60).
constexpr int kUnitCost = 32, kMergeCost = 60, kMinTiles = 12;
constexpr float kTopP = 13.f;  // log2 of the largest weight when the reference moves
constexpr float kMaxP = 15.f;  // ... and of any
constexpr int kTopV = 10;      // a scale's largest power of two becomes 2^kTopV: 24 s < 2^16
// How many powers of two the value scales of a group may lie above and below the largest of a warp's first tile.  In fp16
// the smallest is then 2^-14 or more, and its values are exact; a weight that fp16 rounds to a multiple of 2^-38 of the
// row's largest is off by 2^-14 of any other value.  Rows that attend other scales are computed by wide_rows(); so are those
// of 2^(kEnd + 1) and more, since 2^31 weights of 2^15 times 8 of them would leave fp32.
constexpr int kAbove = 10, kBelow = 14, kEnd = 63, kUsual = -3;
constexpr uint32_t kWide = 1u << 16;
constexpr int kLarge = -64;    // a row's power of two: queries of 2^77 and more

template <int D, int NT, int QP>
struct Lay {
  static constexpr int G = D / kI4Group;                 // groups of a row
  static constexpr int R = 8 * NT;                       // query rows
  static constexpr int kRow = D / 2;                     // bytes of a row's codes
  static constexpr int kCodes = kKeys * kRow;            // of a tile
  static constexpr int kScales = kKeys * G * 2;
  static constexpr int kStage = 2 * kCodes + 2 * kScales;  // K, V, their scales; a multiple of the swizzle's span
  static constexpr int W = NT > 1 || D == 256 ? 8 : 12;
  static constexpr int kFit = 170 * 1024 / (W * kStage), S = kFit > 8 ? 8 : kFit;  // stages
  static_assert(S >= 2, "a tile under way beside the one at hand");
  static constexpr int kThreads = 32 * W;
  static constexpr int PS = D + 4;                       // a row of a warp's state: D sums, reference, sum of weights
  static constexpr bool kAhead = R * PS * 4 <= kStage;   // the state takes one stage's place, the next unit's tiles the others'
  static constexpr int kRing = S * kStage > R * PS * 4 ? S * kStage : (R * PS * 4 + 1023) / 1024 * 1024;
  static constexpr int kNorm = W * kRing;                // per warp: scales as the products take them
  // per warp: keys' scales in fp32, values' in fp16, their factors; in bf16 bits, two groups a word, the largest scale of the
  // largest power of two seen, less the smallest that may come; that; and the largest that may come
  static constexpr int kWords = (G + 1) / 2, kSeen = (kKeys * G * 6 + G * 4 + 15) / 16 * 16;
  static constexpr int kNormBytes = (kSeen + 3 * kWords * 4 + R * 4 + 15) / 16 * 16;
  static constexpr int kQ = kNorm + W * kNormBytes;      // query operands [QP][NT][2 G][32 lanes] of 8 bytes
  static constexpr int kQsum = kQ + QP * NT * 2 * G * 32 * 8;  // [G][R] fp32: where accumulators start
  static constexpr int kQexp = kQsum + R * G * 4;        // [R]: power of two of a row
  static constexpr int kTotal = kQexp + R * 4 + 1024;    // and room to align the base
  static_assert(kTotal + 12 * 1024 + 512 <= 232448, "shared memory");
};

// The key at position x of a tile.
template <int D>
__device__ __forceinline__ int kappa(int x) {
  if (D == 128) return x ^ ((x >> 1) & 1);                                                  // 0 1 3 2 4 5 7 6
  if (D == 64) return (x & ~3) | ((((x & 1) << 1) | ((x >> 1) & 1)) ^ ((x & 4) >> 1));      // 0 2 1 3 6 4 7 5
  return x;
}

// Where 16-byte part `part` of row r's codes lies in a tile: parts are exchanged so that neighbours in the use lie in different banks.
template <int D>
__device__ __forceinline__ int at_part(int r, int part) {
  const int x = D == 256 ? r & 7 : D == 128 ? (r >> 1) & 3 : D == 64 ? (r >> 2) & 1 : 0;
  return r * (D / 2) + ((part ^ x) << 4);
}

// d = a b + c
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                                    const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
// d += a b
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
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
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// (x & mask) | bits
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(x), "r"(mask), "r"(bits));
  return r;
}
using ptc::fast_exp2;
// 2^e for any e, as what fp32 holds of it
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(min(max(e, -126), 127) + 127) << 23); }
// the same, and 0 where that is too small for fp32's normal numbers
__device__ __forceinline__ float pow2_or_0(int e) { return e < -126 ? 0.f : pow2(e); }
// x 2^e without leaving fp32 on the way
__device__ __forceinline__ float times_pow2(float x, int e) {
  const int a = e / 2;
  return x * pow2(a) * pow2(e - a);
}

// N consecutive 32-bit words of shared memory in wide loads.
template <int N>
__device__ __forceinline__ void lds_words(const void *p, uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 x = reinterpret_cast<const uint4 *>(p)[i / 4];
      w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
    }
  } else if constexpr (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2 *>(p);
    w[0] = x.x, w[1] = x.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t *>(p);
  }
}
__device__ __forceinline__ uint32_t lds32(const unsigned char *p) { return *reinterpret_cast<const uint32_t *>(p); }
__device__ __forceinline__ uint32_t lds16(const unsigned char *p) { return *reinterpret_cast<const uint16_t *>(p); }

template <int N>
__device__ __forceinline__ void cp_async(void *dst, const void *src) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async(void *dst, const void *src, bool ok) {
  const int n = ok ? N : 0;  // 0: zeros
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src), "n"(N), "r"(n) : "memory");
}
// A unit, as one thread prepares it for all warps.
struct Unit {
  int b, row0, ntok;           // sequence, first row of query / output, tokens
  int kvh, h0, g, rows;        // kv head, first query head, query heads, rows
  int t0, tiles;               // this CTA's key tiles
  int in_lo, in_hi;            // tiles [in_lo, in_hi) have only keys that every row attends
  uint32_t qpos, jlo, jhi;     // position of the first token; positions that some row attends
  int cut, cf, cl;             // is the unit cut, and the first and last CTA with a part of it
  int more;                    // is this a unit?
  const unsigned char *codes;  // the kv head's key codes and scales
  const uint16_t *scales;
  template <typename Walk>
  __device__ inline void take(const I4Params &p, const PShape &shp, Walk &walk) {
    PUnit u;
    more = walk.next(shp, u);
    if (!more) return;
    b = u.b;
    row0 = u.row0;
    ntok = u.ntok;
    kvh = u.hu / p.hblocks;
    const int hb = u.hu - kvh * p.hblocks;
    h0 = kvh * p.group + hb * p.gb;
    g = min(p.gb, p.group - hb * p.gb);
    rows = ntok * g;
    codes = static_cast<const unsigned char *>(p.kp) + kvh * p.sh;
    scales = p.kscale + kvh * p.th;
    t0 = u.kt + u.k0;
    tiles = u.k1 - u.k0;
    const long long lo = p.W > 0 && u.qpos - p.W + 1 > 0 ? u.qpos - p.W + 1 : 0, hi = u.qpos + u.ntok;
    const long long all = p.W > 0 && hi - p.W > lo ? hi - p.W : lo;  // the last token's first key
    qpos = (uint32_t)u.qpos;
    jlo = (uint32_t)lo;
    jhi = (uint32_t)hi;
    in_lo = (int)((all + kKeys - 1) / kKeys);
    in_hi = (int)((u.qpos + 1) / kKeys);
    cut = u.k0 > 0 || u.k1 < u.nt;
    cf = cut ? walk.owner(u.g0) : 0;
    cl = cut ? walk.owner(u.g0 + u.nt - 1) : 0;
  }
};

// Pages of any size: every lane copies its own rows' codes of the tile that begins at position j0 to kb.  Returns
// whether the row of key `lane` is needed and has a page, and where its scales are.  Out of line, for
// the tiles' usual way is short of instruction cache.
template <int D>
__device__ __noinline__ bool load_rows(const I4Params &p, const Unit &x, unsigned char *kb, uint32_t j0, int lane, const uint16_t *&scales) {
  constexpr int CPR = D / 32, RPC = 32 / CPR;
  const int crow = lane / CPR, cpart = lane % CPR;
  const int32_t *table = p.table + (long long)x.b * p.width;
  auto page_of = [&](uint32_t j) { return (uint32_t)(((uint64_t)j * p.div_mul) >> p.div_shift); };
  auto page_at = [&](uint32_t j) {
    const int id = j >= x.jlo && j < x.jhi ? needed_page(table[page_of(j)]) : kNotNeeded;
    if (id != kNotNeeded && (unsigned)id >= (unsigned)p.npages) pflag(p, GQAW_DEV_BAD_PAGE);
    return (unsigned)id < (unsigned)p.npages ? id : -1;
  };
#pragma unroll 1
  for (int c = 0; c < CPR; ++c) {
    const uint32_t j = j0 + c * RPC + crow, row = j - page_of(j) * p.page;
    const int id = page_at(j);
    const unsigned char *at = id >= 0 ? x.codes + (((uint64_t)(uint32_t)id * p.sp16 + (uint64_t)row * p.sr16 + cpart) << 4) : x.codes;
    unsigned char *to = kb + at_part<D>(c * RPC + crow, cpart);
    cp_async<16>(to, at, id >= 0);
    cp_async<16>(to + kKeys * (D / 2), at + p.to_values, id >= 0);
  }
  const uint32_t j = j0 + lane, row = j - page_of(j) * p.page;
  const int id = page_at(j);
  scales = id >= 0 ? x.scales + ((uint64_t)(uint32_t)id * p.tpg + (uint64_t)row * p.trg) * (D / kI4Group) : x.scales;
  return id >= 0;
}

// What the value scales of a warp's first tile of a unit say of the others.  Out of line, which leaves the loop over the
// tiles its registers (64 long contexts 262 us, 264 to 267 otherwise).
template <int D, int kWords>
__device__ __noinline__ void first_scales(const I4Params &p, const Unit &x, const uint16_t *scales, uint32_t *seen_at, float *vf, int warp, int lane) {
  constexpr int G = D / kI4Group;
  const int key = (lane & ~7) | kappa<D>(lane & 7);
  const long long j = (long long)(x.t0 + warp) * kKeys + key, last = (long long)x.qpos + x.ntok - 1;
  // The largest of the keys that all rows attend, if one is not zero: what only some of them attend is not to say how
  // the others are computed.  A group of zeros, like those of padding, may have scales around 2^kUsual after that.
  const bool some = j >= x.jlo && j < x.jhi, all = j <= (long long)x.qpos && j >= (long long)x.jlo && (p.W == 0 || j > last - p.W);
  const uint16_t *vs = scales + key * G;
#pragma unroll
  for (int gr = 0; gr < G; ++gr) {
    const uint32_t h = vs[gr] & 0x7fffu, fin = h < 0x7f80u ? h : 0u;
    uint32_t mx = __reduce_max_sync(0xffffffffu, all ? fin : 0u);
    if (mx == 0u) mx = __reduce_max_sync(0xffffffffu, some ? fin : 0u);
    const int e = mx ? (int)(mx >> 7) : 127 + kUsual, low = max(min(e, 127 + kEnd) - kBelow, 0) << 7;
    const uint32_t roof = (uint32_t)(min(e + kAbove, 127 + kEnd) << 7 | 0x7f);
    if (lane == 0) {
      uint16_t *to = reinterpret_cast<uint16_t *>(seen_at) + gr;
      to[0] = (uint16_t)(mx ? min(mx | 0x7fu, roof) - low : 0u);  // (none: as if the smallest had been seen)
      to[2 * kWords] = (uint16_t)low;
      to[4 * kWords] = (uint16_t)roof;
      vf[gr] = pow2(kTopV + 127 - (mx ? min(e, 127 + kEnd) : low >> 7));
    }
  }
  if (G == 1 && lane == 0)  // the other half of the only word
    reinterpret_cast<uint16_t *>(seen_at)[1] = reinterpret_cast<uint16_t *>(seen_at)[3] = reinterpret_cast<uint16_t *>(seen_at)[5] = 0;
  __syncwarp();
}

// The state of a warp's tiles of a unit in fp32 throughout, for the rows of `rows` alone, which attend value scales too
// far apart for one power of two in fp16, or have queries of 2^77 and more.  The large scales may be another row's, or under next to no weight, so every row
// and lane has a power of two of its own: a sum holds 2^ro of what it stands for, ro going down for a product above 2^88
// (2^31 of them stay in fp32, and beside them what is 2^-200 of the largest) and up when a tile begins with less than 1.  At the end the reference moves so that the weights add up to 2^-13: no sum
// of warps and CTAs leaves fp32 where the average does not.
//
// Out of line and written for few registers, since ordinary caches do not come here: a lane has a key for the logits (its
// scales relative to the largest's power of two) and D / 32 dimensions for the values.  The queries are the operands of the products (put_query()).  Bound by its own
// instructions: 64 contexts of 4 k to 33 k keys that all have such scales take 6.8 ms, and 0.262 without.
template <typename T, int D, int NT, int QP>
__device__ __noinline__ void wide_rows(const I4Params &p, const Unit &x, const unsigned char *smem, float *mine, uint32_t rows, uint32_t marked,
                                       int warp, int lane) {
  using L = Lay<D, NT, QP>;
  constexpr int G = L::G, R = L::R, PS = L::PS, DL = D / 32, kNone = 1 << 20, kHigh = 80;
  const int my_group = lane * DL / kI4Group;
  const uint2 *sq = reinterpret_cast<const uint2 *>(smem + L::kQ);
  const int *sqexp = reinterpret_cast<const int *>(smem + L::kQexp);
  float o[R][DL], l[R], m[R];  // the reference is a whole number
  int ro[R];
  __syncwarp();  // the other rows' state is written
#pragma unroll
  for (int r = 0; r < R; ++r) {
    l[r] = 0.f;
    m[r] = -INFINITY;
    ro[r] = kNone;
#pragma unroll
    for (int d = 0; d < DL; ++d) o[r][d] = 0.f;
  }
#pragma unroll 1
  for (int t = x.t0 + warp; t < x.t0 + x.tiles; t += L::W) {
    const uint32_t j = (uint32_t)t * kKeys + lane;
    const bool in = j >= x.jlo && j < x.jhi;
    const I4Place at = in ? i4_place(p, x.b, j) : I4Place{-1, 0};
    const bool ok = at.page >= 0;  // else a row of zeros
    const unsigned char *codes = x.codes + (ok ? at.page * p.sp + at.row * p.sr : 0ll);
    const uint16_t *scales = x.scales + (ok ? at.page * p.tp + at.row * p.tr : 0ll);
    int ks = -126;  // the power of two of the key's largest scale
#pragma unroll 1
    for (int gr = 0; gr < G; ++gr) ks = max(ks, ok ? (int)(scales[gr] >> 7 & 0xffu) - 127 : -126);
    float w[R];  // logits, then weights
#pragma unroll
    for (int r = 0; r < R; ++r) w[r] = 0.f;
#pragma unroll 1
    for (int gr = 0; gr < G; ++gr) {
      const float s = ok ? times_pow2(__uint_as_float((uint32_t)scales[gr] << 16), -ks) : 0.f;
      float acc[R];
#pragma unroll
      for (int r = 0; r < R; ++r) acc[r] = 0.f;
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {  // eight dimensions
        const uint32_t word = ok ? *reinterpret_cast<const uint32_t *>(codes + gr * 16 + b * 4) : 0x88888888u;
        float c[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {  // odd ones count 16 times, their queries a sixteenth
          const float y = (float)((int)((word >> (4 * k)) & 15u) - 8);
          c[k] = k & 1 ? 16.f * y : y;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if (!((rows >> r) & 1u)) continue;
#pragma unroll
          for (int q = QP - 1; q >= 0; --q)
#pragma unroll
            for (int step = 0; step < 2; ++step) {
              const uint2 y = sq[((q * NT + r / 8) * 2 * G + 2 * gr + step) * 32 + (r & 7) * 4 + b];
              const float2 even = floats_of(y.x), odd = floats_of(y.y);
              acc[r] = fmaf(c[2 * step], even.x, acc[r]);
              acc[r] = fmaf(c[2 * step + 4], even.y, acc[r]);
              acc[r] = fmaf(c[2 * step + 1], odd.x, acc[r]);
              acc[r] = fmaf(c[2 * step + 5], odd.y, acc[r]);
            }
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) w[r] = fmaf(s, acc[r], w[r]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (!((rows >> r) & 1u)) continue;
      float z = times_pow2(w[r] * p.qscale, ks - sqexp[r]);
      if (p.capmul != 0.f) z = sizeof(T) == 4 ? cap_logit(p, z) : p.capmul * ptc::fast_tanh(z);
      const long long pos = (long long)x.qpos + r / x.g;
      if (!(r < x.rows && in && j <= pos && (p.W == 0 || j > pos - p.W))) z = -INFINITY;
      float mx = z;
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
      float top = 0.f;
      if (mx > m[r]) {
        const float to = rintf(mx), f = m[r] == -INFINITY ? 0.f : fast_exp2(m[r] - to);
        m[r] = to;
        l[r] *= f;
#pragma unroll
        for (int d = 0; d < DL; ++d) o[r][d] *= f;
      }
      w[r] = fast_exp2(z - (m[r] == -INFINITY ? 0.f : m[r]));
      l[r] += w[r];
#pragma unroll
      for (int d = 0; d < DL; ++d) top = fmaxf(top, fabsf(o[r][d]));
      if (top == 0.f) {
        ro[r] = kNone;
      } else if (top < 1.f) {
        const int up = kHigh - ((int)(__float_as_uint(top) >> 23) - 127);
        ro[r] += up;
#pragma unroll
        for (int d = 0; d < DL; ++d) o[r][d] = times_pow2(o[r][d], up);
      }
    }
#pragma unroll 1
    for (int key = 0; key < kKeys; ++key) {
      const unsigned char *vc = reinterpret_cast<const unsigned char *>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(codes), key)) + p.to_values;
      const unsigned char *vs = reinterpret_cast<const unsigned char *>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(scales), key)) + p.to_value_scales;
      const bool have = __shfl_sync(0xffffffffu, ok, key);
      const uint32_t bits = have ? reinterpret_cast<const uint16_t *>(vs)[my_group] : 0u;
      const bool some = (bits & 0x7fffu) != 0u && (bits & 0x7fffu) < 0x7f80u;  // one that is not finite: `marked`
      uint32_t word = 0;
      if (some) {
        if constexpr (DL == 8) word = reinterpret_cast<const uint32_t *>(vc)[lane];
        else if constexpr (DL == 4) word = reinterpret_cast<const uint16_t *>(vc)[lane];
        else if constexpr (DL == 2) word = vc[lane];
        else word = vc[lane / 2] >> (4 * (lane & 1));
      }
      const int es = max((int)(bits >> 7 & 0xffu), 1) - 127;
      const float s = times_pow2(__uint_as_float(bits << 16), -es);  // its power of two taken off
      float v[DL];
#pragma unroll
      for (int d = 0; d < DL; ++d) v[d] = s * (float)((int)((word >> (4 * d)) & 15u) - 8);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (!((rows >> r) & 1u)) continue;
        const float pr = __shfl_sync(0xffffffffu, w[r], key);
        if (some && pr != 0.f) {
          const int over = (int)(__float_as_uint(pr) >> 23 & 0xffu) - 127 + es + ro[r];  // the product's power of two
          if (over > kHigh + 8) {
            const int down = over - kHigh;
            ro[r] -= down;
#pragma unroll
            for (int d = 0; d < DL; ++d) o[r][d] = times_pow2(o[r][d], -down);
          }
          const float u = times_pow2(pr, ro[r] + es);
#pragma unroll
          for (int d = 0; d < DL; ++d) o[r][d] = fmaf(u, v[d], o[r][d]);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float sum = l[r];
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    int e = sum > 0.f && sum < INFINITY ? (int)(__float_as_uint(sum) >> 23) - 127 + 13 : 0;
    if (!(m[r] + (float)e - m[r] == (float)e)) e = 0;  // a reference too large for that
    const bool bad = (__shfl_sync(0xffffffffu, marked, r) >> my_group) & 1u;
    if (!((rows >> r) & 1u)) continue;
#pragma unroll
    for (int d = 0; d < DL; ++d) mine[r * PS + lane * DL + d] = bad ? NAN : times_pow2(o[r][d], -ro[r] - e);
    if (lane == 0) {
      mine[r * PS + D] = m[r] + (float)e;
      mine[r * PS + D + 1] = times_pow2(sum, -e);
    }
  }
}

}  // namespace i4a

// NT: operands of 8 query rows.  T: type of the rows outside the cache.
template <typename T, int D, int NT, int QP>
__global__ void __launch_bounds__(i4a::Lay<D, NT, QP>::kThreads, 1)
    i4_attend_kernel(const __grid_constant__ I4Params p) {
  using namespace i4a;
  using L = Lay<D, NT, QP>;
  constexpr int W = L::W, S = L::S, G = L::G, R = L::R, PS = L::PS;
  constexpr int PP = sizeof(T) == 4 ? 2 : 1;         // parts of a weight
  constexpr bool kExact = sizeof(T) == 4;            // see above
  // Exponents of fp32 rows are taken near 0, where they have most bits, and the power of two comes after
  constexpr float kTopZ = kExact ? 0.f : kTopP, kMaxZ = kExact ? kMaxP - kTopP : kMaxP;
  constexpr bool kQreg = NT * QP * G <= 8;           // query operands in registers
  constexpr int SB = NT == 1 ? 2 : 1;                  // blocks of 16 keys at once
  constexpr int VW = D >= 64 ? D / 64 : 1;           // words of a lane's codes of a value row (D = 32: half of one)
  constexpr int VT = D / 16;                         // operands of 16 dimensions
  constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u, kTop = 0x03c003c0u;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ PSched sched;
  __shared__ int s_last, s_state[W];  // ...; where each warp's state lies
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, t4 = lane & 3;
  unsigned char *ring = smem + warp * L::kRing;
  float *nk = reinterpret_cast<float *>(smem + L::kNorm + warp * L::kNormBytes);  // [G / 4][position][4]
  uint16_t *nv = reinterpret_cast<uint16_t *>(nk + kKeys * G);                    // [G][position]
  float *vf = reinterpret_cast<float *>(nv + kKeys * G);  // of each group: the factor that takes the largest scale's power of two to 2^kTopV
  uint32_t *seen_at = reinterpret_cast<uint32_t *>(smem + L::kNorm + warp * L::kNormBytes + L::kSeen);
  // of each row: groups in which it attends a scale that is not finite; kWide: it attends one too far off, or its queries are so
  // large that the smallest scales, 2^-133, would leave fp32 beside acc < 1 (a factor for these would make the others' logits
  // leave it)
  uint32_t *marks = seen_at + 3 * L::kWords;
  const uint2 *sq = reinterpret_cast<const uint2 *>(smem + L::kQ);
  float *sqsum = reinterpret_cast<float *>(smem + L::kQsum);
  int *sqexp = reinterpret_cast<int *>(smem + L::kQexp);
  pdl_wait();
  PShape shp = shape_of(p, kUnitCost);
  shp.merge_tiles = kMergeCost;
  shp.min_tiles = kMinTiles;
  sched_build<kKeys>(p, shp, &sched);
  __shared__ Unit units[3];  // the unit at hand, the next and the one behind it
  const int my_group = gid * (D / 8) / kI4Group;  // of this lane's dimensions, gid D / 8 and on

  // A copy of the warp has 16 bytes of codes a lane: CPR lanes a row, a block of RPC rows, CPR copies a tile.
  // Where blocks lie in one page each, a lane finds one block's addresses: those of TPB tiles at once, a
  // hundredth of what every lane for its own rows takes, and hands them out by shuffles.
  constexpr int CPR = D / 32, RPC = 32 / CPR, TPB = 32 / CPR;
  const int crow = lane / CPR, cpart = lane % CPR;
  auto page_of = [&](uint32_t j) { return (uint32_t)(((uint64_t)j * p.div_mul) >> p.div_shift); };
  const unsigned char *bcodes = nullptr;  // this lane's block of the batch of tiles at hand: codes
  const uint16_t *bscales = nullptr;      // ... and scales, of keys
  uint32_t bok = 0;                       // the lanes whose block is needed and has a page
  int bid = kNotNeeded, bn = 0;                   // the page of its block of the next batch; tiles of this batch loaded
  // its place in the batch that begins with tile t
  auto block_at = [&](int t) { return (uint32_t)(t + lane / CPR * W) * kKeys + lane % CPR * RPC; };
  auto look_up = [&](const Unit &x, int t, int end) {
    const uint32_t j = block_at(t);
    return t + lane / CPR * W < end && j < x.jhi && j + RPC > x.jlo ? needed_page(p.table[(long long)x.b * p.width + page_of(j)]) : kNotNeeded;
  };
  auto resolve = [&](const Unit &x, int t) {
    const uint32_t j = block_at(t), row = j - page_of(j) * p.page;
    const bool ok = (unsigned)bid < (unsigned)p.npages;
    if (!ok && bid != kNotNeeded) pflag(p, GQAW_DEV_BAD_PAGE);
    bok = __ballot_sync(0xffffffffu, ok);
    bcodes = x.codes + (ok ? ((uint64_t)(uint32_t)bid * p.sp16 + (uint64_t)row * p.sr16) << 4 : 0ull);
    bscales = x.scales + (ok ? ((uint64_t)(uint32_t)bid * p.tpg + (uint64_t)row * p.trg) * G : 0ull);
  };
  const uint32_t code_off = (crow * p.sr16 + cpart) << 4, scale_off = lane % RPC * p.trg * G;
  // key tile t into stage st; rows that nobody needs become zeros
  auto load = [&](const Unit &x, int t, int end, int st) {
    if (t < end) {  // uniform over the warp
      unsigned char *kb = ring + st * L::kStage, *sb = kb + 2 * L::kCodes;
      const uint32_t j0 = (uint32_t)t * kKeys;
      const bool whole = j0 >= x.jlo && j0 + kKeys <= x.jhi;
      unsigned char *dst = kb + at_part<D>(crow, cpart);
      const uint16_t *ks = x.scales;
      bool key_ok = false, plain = false;
      if (p.blocks) {
        constexpr uint32_t kAll = CPR == 32 ? ~0u : (1u << CPR) - 1u;
        const uint32_t ok = bok >> (bn * CPR);
        plain = whole && (ok & kAll) == kAll;
#pragma unroll
        for (int c = 0; c < CPR; ++c) {
          const unsigned char *at =
              reinterpret_cast<const unsigned char *>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(bcodes), bn * CPR + c)) + code_off;
          unsigned char *to = D == 256 ? kb + at_part<D>(c * RPC + crow, cpart) : dst + c * RPC * L::kRow;
          if (plain) {
            cp_async<16>(to, at);
            cp_async<16>(to + L::kCodes, at + p.to_values);
          } else {
            const uint32_t j = j0 + c * RPC + crow;
            const bool need = ((ok >> c) & 1u) && (whole || (j >= x.jlo && j < x.jhi));
            at = need ? at : x.codes;
            cp_async<16>(to, at, need);
            cp_async<16>(to + L::kCodes, at + p.to_values, need);
          }
        }
        const int src = bn * CPR + lane / RPC;
        ks = reinterpret_cast<const uint16_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(bscales), src)) + scale_off;
        key_ok = plain || (((bok >> src) & 1u) && (whole || (j0 + lane >= x.jlo && j0 + lane < x.jhi)));
        if (!key_ok) ks = x.scales;
        if (++bn == TPB) {  // the next batch
          resolve(x, t + W);
          bid = look_up(x, t + (TPB + 1) * W, end);
          bn = 0;
        }
      } else {
        key_ok = load_rows<D>(p, x, kb, j0, lane, ks);
      }
      const void *vs = reinterpret_cast<const unsigned char *>(ks) + p.to_value_scales;
      if constexpr (G >= 2) {
        if (plain) {
          cp_async<2 * G>(sb + lane * 2 * G, ks);
          cp_async<2 * G>(sb + L::kScales + lane * 2 * G, vs);
        } else {
          cp_async<2 * G>(sb + lane * 2 * G, ks, key_ok);
          cp_async<2 * G>(sb + L::kScales + lane * 2 * G, vs, key_ok);
        }
      } else {  // two bytes: too few for a copy
        reinterpret_cast<uint16_t *>(sb)[lane] = key_ok ? *ks : (uint16_t)0;
        reinterpret_cast<uint16_t *>(sb + L::kScales)[lane] = key_ok ? *static_cast<const uint16_t *>(vs) : (uint16_t)0;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto bump = [](int st) { return st + 1 == S ? 0 : st + 1; };
  // a unit's first tiles, from stage st on; id: first_page() of it
  auto first_page = [&](const Unit &x) { return p.blocks && x.more ? look_up(x, x.t0 + warp, x.t0 + x.tiles) : kNotNeeded; };
  auto load_first = [&](const Unit &x, int st, int id) {
    const int t = x.t0 + warp, end = x.t0 + x.tiles;
    if (p.blocks) {
      bid = id;
      resolve(x, t);
      bid = look_up(x, t + TPB * W, end);
      bn = 0;
    }
#pragma unroll 1
    for (int i = 0; i < S - 1; ++i) {
      load(x, t + i * W, end, st);
      st = bump(st);
    }
  };
  // one element of every group of row r
  auto query_row = [&](const Unit &x, int r, float (&y)[G]) {
    const int tok = r / x.g, hh = r - tok * x.g;
#pragma unroll
    for (int i = 0; i < G; ++i) {
      y[i] = 0.f;
      if (r < x.rows) {
        const long long at = (x.row0 + tok) * p.qs + (long long)(x.h0 + hh) * D + i * 32 + lane;
        y[i] = Elem<T>::load(static_cast<const T *>(p.q)[at]);
        if (QP == 2 && sizeof(T) == 2) y[i] += Elem<T>::load(static_cast<const T *>(p.qlo)[at]);
      }
    }
  };
  // a warp's row as operands
  auto put_query = [&](int r, const float (&x)[G]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < G; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
    top = __reduce_max_sync(0xffffffffu, top);
    // x 2^e: the largest at 2^13; a row that is not finite stays so and takes no part in what rows share
    const int e = top && top < 0x7f800000u ? min(140 - (int)(top >> 23), 126) : 0;
    const int nib = lane & 7, step = (nib >> 1) & 1;
    const float f = nib & 1 ? 0.0625f : 1.f, back = nib & 1 ? -8.f * 16.f / 16777216.f : -8.f / 16777216.f;  // a code of an odd nibble counts 16 times
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
      if constexpr (!kExact) {
        sum *= back;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        if (lane == 0) sqsum[i * R + r] = sum;
      }
    }
    if (lane == 0) sqexp[r] = e;
  };

  // One thread walks the units, two ahead, of the warp that has least to do beside it; its walker is kept
  // out of everybody's registers
  constexpr int kWalkThread = L::kThreads - 32;
  __shared__ __align__(16) unsigned char walker[sizeof(PWalk<kKeys>)];
  PWalk<kKeys> *walk = reinterpret_cast<PWalk<kKeys> *>(walker);
  if (tid == 0) {
    *walk = PWalk<kKeys>(shp, &sched);
    units[0].take(p, shp, *walk);
  }
  __syncthreads();
  int st = 0;  // stage of the next tile
  if (units[0].more) {
    float q[G];
    query_row(units[0], min(warp, R - 1), q);
    load_first(units[0], 0, first_page(units[0]));
    if (tid == kWalkThread) units[1].take(p, shp, *walk);
    put_query(min(warp, R - 1), q);
    for (int r = warp + W; r < R; r += W) {
      query_row(units[0], r, q);
      put_query(r, q);
    }
    __syncthreads();
  }
  for (int un = 0; units[un].more;) {
    const Unit &x = units[un];
    const int rows = x.rows, end = x.t0 + x.tiles, in_lo = x.in_lo, in_hi = x.in_hi;
    uint2 qr[kQreg ? QP * NT * 2 * G : 1];
    float qs[kQreg ? NT * G : 1][4];  // where this lane's accumulators start
    if constexpr (kQreg) {
#pragma unroll
      for (int i = 0; i < QP * NT * 2 * G; ++i) qr[i] = sq[i * 32 + lane];
#pragma unroll
      for (int i = 0; i < NT * G; ++i) {
        const float2 y = *reinterpret_cast<const float2 *>(sqsum + (i % G) * R + i / G * 8 + 2 * t4);
        qs[i][0] = qs[i][2] = y.x;
        qs[i][1] = qs[i][3] = y.y;
      }
    }
    // z = (sum s acc) 2^(24 - e) qscale, e the row's power of two
    float qf[NT][2], nb[NT][2], th[NT][2], l[NT][2];  // factor; minus the reference; what a logit less the reference may be
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        qf[nt][c] = p.qscale * pow2_or_0(24 - sqexp[nt * 8 + 2 * t4 + c]);
        nb[nt][c] = 0.f;
        th[nt][c] = -INFINITY;
        l[nt][c] = 0.f;
      }
    float o[NT][VT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < VT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[nt][i][c] = 0.f;
    if (x.t0 + warp < end) {
      asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
      __syncwarp();
      first_scales<D, L::kWords>(p, x, reinterpret_cast<const uint16_t *>(ring + st * L::kStage + 2 * L::kCodes + L::kScales), seen_at, vf, warp, lane);
    }
    if (lane < R) marks[lane] = lane < rows && sqexp[lane] < kLarge ? kWide : 0u;
    __syncwarp();

    // lane-constant places in a tile: keys' codes of positions gid and gid + 8, 16, 24; values' of this lane's dimensions
    int koff[G], voff[2];
#pragma unroll
    for (int gr = 0; gr < G; ++gr) koff[gr] = at_part<D>(kappa<D>(gid), gr) + t4 * 4;
#pragma unroll
    for (int c = 0; c < 2; ++c) voff[c] = L::kCodes + at_part<D>(kappa<D>(2 * t4 + c), gid * (D / 16) / 16) + gid * (D / 16) % 16;

    const int nid = first_page(units[un == 2 ? 0 : un + 1]);  // long before it is wanted
    for (int t = x.t0 + warp; t < end; t += W) {
      load(x, t + (S - 1) * W, end, st == 0 ? S - 1 : st - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
      __syncwarp();
      const unsigned char *kb = ring + st * L::kStage, *sb = kb + 2 * L::kCodes;
      const bool inner = t >= in_lo && t < in_hi;

      // ---- scales: a lane has a position
      {
        const int key = (lane & ~7) | kappa<D>(lane & 7);
        uint32_t kw[(G + 1) / 2], vw[(G + 1) / 2];
        if constexpr (G == 1) {
          kw[0] = reinterpret_cast<const uint16_t *>(sb)[key];
          vw[0] = reinterpret_cast<const uint16_t *>(sb + L::kScales)[key];
        } else {
          lds_words(sb + key * 2 * G, kw);
          lds_words(sb + L::kScales + key * 2 * G, vw);
        }
        if (!inner && ((uint32_t)t * kKeys + key < x.jlo || (uint32_t)t * kKeys + key >= x.jhi)) {  // a row of nobody in the unit, whatever it holds
#pragma unroll
          for (int y = 0; y < (G + 1) / 2; ++y) vw[y] = 0u;
        }
        uint32_t seen[2 * L::kWords], fac[G];
        lds_words(seen_at, seen);
        bool outside = false;  // above the largest so far, or below what may come (zeros among these)
#pragma unroll
        for (int y = 0; y < L::kWords; ++y) {
          // of both halves at once: a lower one that takes from the upper is below its range, and found by itself
          const uint32_t d = (vw[y] & 0x7fff7fffu) - seen[L::kWords + y];
          outside |= __vmaxu2(d, seen[y]) != seen[y];
        }
        if (__any_sync(0xffffffffu, outside)) {
          const float before = vf[my_group];
          __syncwarp();
          uint32_t bad = 0;  // of this lane's key: groups with a scale that is not finite; kWide: with one that lies too far off
#pragma unroll
          for (int y = 0; y < L::kWords; ++y) {
            const uint32_t low = seen[L::kWords + y], roof = seen_at[2 * L::kWords + y], top = seen[y] + low;
            uint32_t x2 = vw[y] & 0x7fff7fffu;
            const uint32_t less = ((x2 | 0x80008000u) - 0x00010001u) ^ 0x80008000u;  // by one, zeros on top
            const uint32_t off = (__vmaxu2(x2, roof) ^ roof) | (__vminu2(less, low) ^ low);
            if (off) {
#pragma unroll
              for (int hf = 0; hf < 2; ++hf)
                if (off >> (16 * hf) & 0xffffu) {
                  bad |= (x2 >> (16 * hf) & 0xffffu) >= 0x7f80u ? 1u << (2 * y + hf) : kWide;
                  vw[y] &= ~(0xffffu << (16 * hf));
                }
              x2 = vw[y] & 0x7fff7fffu;
            }
            const uint32_t mx = __vmaxu2(__reduce_max_sync(0xffffffffu, x2 & 0xffffu) | __reduce_max_sync(0xffffffffu, x2 >> 16) << 16 | 0x007f007fu, top);
            if (lane == 0) seen_at[y] = mx - low;
            if (lane < 2 && 2 * y + lane < G) vf[2 * y + lane] = pow2(kTopV + 127 - (int)((mx >> (16 * lane + 7)) & 0xffu));
          }
          __syncwarp();
          const float down = vf[my_group] / before;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int v = 0; v < VT; ++v)
#pragma unroll
              for (int c = 0; c < 4; ++c) o[nt][v][c] *= down;
          uint32_t who = __ballot_sync(0xffffffffu, bad != 0u);
          while (who) {  // mark the rows that attend such a key
            const int src = __ffs((int)who) - 1;
            who &= who - 1u;
            const long long j = (long long)t * kKeys + __shfl_sync(0xffffffffu, key, src), at = (long long)x.qpos + lane / x.g;
            const uint32_t groups = __shfl_sync(0xffffffffu, bad, src);
            if (lane < rows && j <= at && (p.W == 0 || j > at - p.W)) marks[lane] |= groups;
          }
        }
        lds_words(vf, fac);
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
          const uint32_t ka = gr & 1 ? kw[gr / 2] & 0xffff0000u : kw[gr / 2] << 16;
          const uint32_t va = gr & 1 ? vw[gr / 2] & 0xffff0000u : vw[gr / 2] << 16;
          // (signed codes are not multiples of 2^-24)
          nk[(gr / 4) * (kKeys * 4) + lane * (G < 4 ? G : 4) + gr % 4] = kExact ? __uint_as_float(ka) * (1.f / 16777216.f) : __uint_as_float(ka);
          nv[gr * kKeys + lane] = __half_as_ushort(__float2half_rn(__uint_as_float(va) * __uint_as_float(fac[gr])));
        }
      }
      __syncwarp();

#pragma unroll
      for (int b0 = 0; b0 < 2; b0 += SB) {
        // ---- logits of SB blocks of 16 keys: this lane has positions gid and gid + 8, rows 2 t4 and 2 t4 + 1
        float z[SB][NT][4];
#pragma unroll
        for (int b = 0; b < SB; ++b) {
          constexpr int GV = G < 4 ? G : 4;
#pragma unroll
          for (int g0 = 0; g0 < G; g0 += GV) {
            uint32_t s0[GV], s1[GV];
            const float *ns = nk + (g0 / 4) * (kKeys * 4) + ((b0 + b) * 16 + gid) * GV;
            lds_words(ns, s0);
            lds_words(ns + 8 * GV, s1);
#pragma unroll
            for (int gg = 0; gg < GV; ++gg) {
              const int gr = g0 + gg;
              const unsigned char *kc = kb + koff[gr] + (b0 + b) * 16 * L::kRow;
              const uint32_t w0 = lds32(kc), w1 = lds32(kc + 8 * L::kRow), x0 = w0 >> 8, x1 = w1 >> 8;
              uint32_t a[8];  // even and odd nibbles of the lower and upper bytes
              if constexpr (kExact) {  // 1024 + c less 1032; 1024 + 16 c less 1152: 16 (c - 8)
                auto even = [&](uint32_t w) { return hadd2(and_or(w, kLow, 0x64006400u), 0xe408e408u); };
                auto odd = [&](uint32_t w) { return hadd2(and_or(w, kHigh, 0x64006400u), 0xe480e480u); };
                a[0] = even(w0), a[1] = even(w1), a[2] = odd(w0), a[3] = odd(w1);
                a[4] = even(x0), a[5] = even(x1), a[6] = odd(x0), a[7] = odd(x1);
              } else {
                a[0] = w0 & kLow, a[1] = w1 & kLow, a[2] = w0 & kHigh, a[3] = w1 & kHigh;
                a[4] = x0 & kLow, a[5] = x1 & kLow, a[6] = x0 & kHigh, a[7] = x1 & kHigh;
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float c[4];
                if constexpr (kExact) {
                  c[0] = c[1] = c[2] = c[3] = 0.f;
                } else if constexpr (!kQreg) {
                  const float2 y = *reinterpret_cast<const float2 *>(sqsum + gr * R + nt * 8 + 2 * t4);
                  c[0] = c[2] = y.x;
                  c[1] = c[3] = y.y;
                }
#pragma unroll
                for (int q = QP - 1; q >= 0; --q) {  // the smaller part first
                  const int at = (q * NT + nt) * 2 * G + 2 * gr;
                  const uint2 qa = kQreg ? qr[kQreg ? at : 0] : sq[at * 32 + lane], qb = kQreg ? qr[kQreg ? at + 1 : 0] : sq[(at + 1) * 32 + lane];
                  if (kQreg && q == QP - 1 && !kExact)
                    mma(c, a[0], a[1], a[2], a[3], qa.x, qa.y, qs[kQreg ? nt * G + gr : 0]);
                  else
                    mma(c, a[0], a[1], a[2], a[3], qa.x, qa.y);
                  mma(c, a[4], a[5], a[6], a[7], qb.x, qb.y);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float s = __uint_as_float(e < 2 ? s0[gg] : s1[gg]);
                  z[b][nt][e] = gr ? fmaf(s, c[e], z[b][nt][e]) : s * c[e];
                }
              }
            }
          }
        }
        // ---- softmax: logits less the reference
        if (p.capmul != 0.f) {
#pragma unroll
          for (int b = 0; b < SB; ++b)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const float y = z[b][nt][c] * qf[nt][c & 1];
                z[b][nt][c] = (sizeof(T) == 4 ? cap_logit(p, y) : p.capmul * ptc::fast_tanh(y)) + nb[nt][c & 1];
              }
        } else {
#pragma unroll
          for (int b = 0; b < SB; ++b)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 4; ++c) z[b][nt][c] = fmaf(z[b][nt][c], qf[nt][c & 1], nb[nt][c & 1]);
        }
        if (!inner) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int r = nt * 8 + 2 * t4 + c;
              // this row's keys, relative to the position of this lane's first one
              const long long at = (long long)x.qpos + r / x.g, j = (long long)t * kKeys + b0 * 16 + kappa<D>(gid);
              const int hi = r < rows ? (int)min(max(at - j, -1ll), 63ll) : -1;
              const long long low = p.W > 0 ? max((long long)x.jlo, at - p.W + 1) : (long long)x.jlo;
              const int lo = (int)min(max(low - j, 0ll), 64ll);
#pragma unroll
              for (int b = 0; b < SB; ++b)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
                  if (b * 16 + hf * 8 > hi || b * 16 + hf * 8 < lo) z[b][nt][2 * hf + c] = -INFINITY;
            }
        }
        bool up = false;
#pragma unroll
        for (int b = 0; b < SB; ++b)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) up |= z[b][nt][c] > th[nt][c & 1];
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float mx = fmaxf(z[0][nt][c], z[0][nt][c + 2]);
              if (SB == 2) mx = fmaxf(mx, fmaxf(z[SB - 1][nt][c], z[SB - 1][nt][c + 2]));
#pragma unroll
              for (int s = 4; s < 32; s <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
              if (mx > th[nt][c]) {  // the same in the eight lanes of a row
                // whole powers of two, so that neither the reference nor what was summed is rounded
                const float by = rintf(mx - kTopZ), f = th[nt][c] == -INFINITY ? 0.f : fast_exp2(-by);
                nb[nt][c] -= by;
                th[nt][c] = kMaxZ;
                l[nt][c] *= f;
#pragma unroll
                for (int v = 0; v < VT; ++v) o[nt][v][c] *= f, o[nt][v][c + 2] *= f;
#pragma unroll
                for (int b = 0; b < SB; ++b) z[b][nt][c] -= by, z[b][nt][c + 2] -= by;
              }
            }
        }
#pragma unroll
        for (int b = 0; b < SB; ++b) {
          // ---- weights: rows of positions become rows of queries
          uint32_t pb[NT][PP][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              float w0 = fast_exp2(z[b][nt][2 * hf]), w1 = fast_exp2(z[b][nt][2 * hf + 1]);
              if (kExact) w0 *= 8192.f, w1 *= 8192.f;  // 2^kTopP
              l[nt][0] += w0;
              l[nt][1] += w1;
              const uint32_t h = half2_of(w0, w1);
              pb[nt][0][hf] = transpose(h);
              if (PP == 2) {
                const float2 back = floats_of(h);
                pb[nt][PP - 1][hf] = transpose(half2_of(w0 - back.x, w1 - back.y));
              }
            }
          // ---- values: this lane's D / 8 dimensions of positions 2 t4, + 1, + 8, + 9
          const int pos = (b0 + b) * 16 + 2 * t4;
          const uint32_t sa = *reinterpret_cast<const uint32_t *>(nv + my_group * kKeys + pos);
          const uint32_t sc = *reinterpret_cast<const uint32_t *>(nv + my_group * kKeys + pos + 8);
          const uint32_t na = hmul2(sa, 0xce00ce00u), nc = hmul2(sc, 0xce00ce00u);  // -24 s
          uint32_t w[4][VW];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const unsigned char *vr = kb + voff[c & 1] + ((b0 + b) * 16 + (c & 2) * 4) * L::kRow;
            if constexpr (D == 32)
              w[c][0] = lds16(vr);
            else
              lds_words(vr, w[c]);
          }
#pragma unroll
          for (int y = 0; y < VW; ++y)
#pragma unroll
            for (int hf = 0; hf < (D == 32 ? 1 : 2); ++hf) {
              // four dimensions of two positions, in one word each
              const uint32_t xa = __byte_perm(w[0][y], w[1][y], hf ? 0x7632 : 0x5410), xb = __byte_perm(w[2][y], w[3][y], hf ? 0x7632 : 0x5410);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                // a nibble in the upper bits of the mantissa of 16: 16 + c, times the scale, less 24 of it
                const uint32_t v0 = hfma2(and_or(k ? xa >> 2 : xa << 6, kTop, 0x4c004c00u), sa, na);
                const uint32_t v1 = hfma2(and_or(k ? xa >> 6 : xa << 2, kTop, 0x4c004c00u), sa, na);
                const uint32_t v2 = hfma2(and_or(k ? xb >> 2 : xb << 6, kTop, 0x4c004c00u), sc, nc);
                const uint32_t v3 = hfma2(and_or(k ? xb >> 6 : xb << 2, kTop, 0x4c004c00u), sc, nc);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  float(&acc)[4] = o[nt][(y * 2 + hf) * 2 + k];
                  if constexpr (kExact) {
                    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
                    float part[4];
                    mma(part, v0, v1, v2, v3, pb[nt][PP - 1][0], pb[nt][PP - 1][1], zero);
                    mma(part, v0, v1, v2, v3, pb[nt][0][0], pb[nt][0][1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[e] += part[e];
                  } else {
                    mma(acc, v0, v1, v2, v3, pb[nt][0][0], pb[nt][0][1]);
                  }
                }
              }
            }
        }
      }
      __syncwarp();  // the stage and the scales are free
      st = bump(st);
    }

    // ---- the next unit's tiles and queries are on their way while this one's rows go out
    const Unit &nx = units[un == 2 ? 0 : un + 1];
    const bool more = nx.more;
    float q[G];
    if (more) {
      query_row(nx, min(warp, R - 1), q);
      if constexpr (L::kAhead) load_first(nx, st, nid);
    }

    // ---- the warp's state: [R][D + 4], in the stage that no tile is under way to
    const int state = L::kAhead ? (st == 0 ? S - 1 : st - 1) * L::kStage : 0;
    float *mine = reinterpret_cast<float *>(ring + state);
    // vf is a power of two, and its reciprocal one
    const int ve = 127 - (int)(__float_as_uint(vf[my_group]) >> 23);
    const float v1 = pow2(ve / 2), v2 = pow2(ve - ve / 2);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = nt * 8 + 2 * t4 + c;
        float sum = l[nt][c];
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        const bool bad = (marks[r] >> my_group) & 1u;
        if (gid == 0) {
          mine[r * PS + D] = th[nt][c] == -INFINITY ? -INFINITY : -nb[nt][c] - (kExact ? kTopP : 0.f);
          mine[r * PS + D + 1] = sum;
        }
        float *to = mine + r * PS + gid * (D / 8);
#pragma unroll
        for (int v = 0; v < VT; v += 2) {
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = bad ? NAN : o[nt][v + e / 2][c + 2 * (e & 1)] * v1 * v2;
          *reinterpret_cast<float4 *>(to + 2 * v) = make_float4(y[0], y[1], y[2], y[3]);
        }
      }
    const uint32_t marked = marks[lane % R], wide = __ballot_sync(0xffffffffu, lane < R && (marked & kWide));
    if (wide) wide_rows<T, D, NT, QP>(p, x, smem, mine, wide, marked, warp, lane);
    if (lane == 0) s_state[warp] = warp * L::kRing + state;
    __syncthreads();
    if (tid == kWalkThread) {  // the unit behind the next one, in the place of the last
      Unit &y = units[un == 0 ? 2 : un - 1];
      y.more = 0;
      if (more) y.take(p, shp, *walk);
    }
    if (more) {
      put_query(min(warp, R - 1), q);
      for (int r = warp + W; r < R; r += W) {
        query_row(nx, r, q);
        put_query(r, q);
      }
    }
    // ---- the warps' states joined
    const bool cut = x.cut;
    const int cta = blockIdx.x, cf = x.cf, cl = x.cl, g = x.g, row0 = x.row0, h0 = x.h0;
    T *out = static_cast<T *>(p.out);
    float *part = p.partials + ((long long)cta * 2 + (cta == cf ? 1 : 0)) * R * PS;
    for (int e = tid; e < rows * (D / 4); e += L::kThreads) {  // four dimensions of a row
      const int r = e / (D / 4), d = (e - r * (D / 4)) * 4, tok = r / g, h = h0 + r - tok * g;
      float M = -INFINITY, Z = 0.f, m[W], A[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < W; ++w) {
        m[w] = reinterpret_cast<const float *>(smem + s_state[w])[r * PS + D];
        M = fmaxf(M, m[w]);
      }
      const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float *y = reinterpret_cast<const float *>(smem + s_state[w]) + r * PS;
        const float f = fast_exp2(m[w] - ref);
        const float4 a = *reinterpret_cast<const float4 *>(y + d);
        Z = fmaf(f, y[D + 1], Z);
        A[0] = fmaf(f, a.x, A[0]);
        A[1] = fmaf(f, a.y, A[1]);
        A[2] = fmaf(f, a.z, A[2]);
        A[3] = fmaf(f, a.w, A[3]);
      }
      if (cut) {
        *reinterpret_cast<float4 *>(part + r * PS + d) = make_float4(A[0], A[1], A[2], A[3]);
        if (d == 0) *reinterpret_cast<float2 *>(part + r * PS + D) = make_float2(M, Z);
      } else {
        const float inv = sink_reciprocal(Z, M, paged_sink_log2(p, h));
        T *to = out + (row0 + tok) * p.os + (long long)h * D + d;
        if constexpr (sizeof(T) == 4)
          *reinterpret_cast<float4 *>(to) = make_float4(A[0] * inv, A[1] * inv, A[2] * inv, A[3] * inv);
        else
          *reinterpret_cast<uint2 *>(to) = make_uint2(tc::pack_bf16x2(A[0] * inv, A[1] * inv), tc::pack_bf16x2(A[2] * inv, A[3] * inv));
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
          out[(row0 + tok) * p.os + (long long)h * D + d] = Elem<T>::store(A[0] * sink_reciprocal(Z, M, paged_sink_log2(p, h)));
        }
        if (tid == 0) p.tickets[cf] = 0u;
      }
    }
    __syncthreads();
    if (!L::kAhead && more) load_first(nx, st, nid);
    un = un == 2 ? 0 : un + 1;
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

// nt: operands of 8 query rows, 1 or (fp32 at head sizes up to 128) 2.
template <typename T, int QP>
cudaError_t launch_i4_attend_t(const I4Params &p, int nt, int sms, cudaStream_t stream) {
  auto pick = [&](auto d) {
    constexpr int D = decltype(d)::value;
    if constexpr (sizeof(T) == 4 && D <= 128)
      if (nt == 2) return launch_i4_attend_one<T, D, 2, QP>(p, sms, stream);
    return launch_i4_attend_one<T, D, 1, QP>(p, sms, stream);
  };
  switch (p.D) {
    case 32: return pick(std::integral_constant<int, 32>());
    case 64: return pick(std::integral_constant<int, 64>());
    case 128: return pick(std::integral_constant<int, 128>());
    default: return pick(std::integral_constant<int, 256>());
  }
}

}  // namespace gqaw
