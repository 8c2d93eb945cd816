// gqaw_paged.cuh -- parameters of the paged operators and the list of work that their
// attention kernels share.
#pragma once

#include "gqaw_internal.cuh"
#include "gqaw_paged_sched.cuh"

namespace gqaw {

constexpr int kPagedTickets = 1024;         // one per CTA
constexpr size_t kPagedTicketOffset = 256;  // after the status word
constexpr size_t kPagedPartialOffset = kPagedTicketOffset + kPagedTickets * 4;

struct PagedParams {
  const void *q, *k, *v;
  const void *qlo;                  // bf16: what rounding left of turned queries, laid out as q; NULL: q is all
  void *out;
  void *kp, *vp;
  long long qs, ks, vs, os;         // elements between tokens
  long long sp, sh, sr;             // elements between pages, heads, rows of the cache
  const int32_t *table, *qstart, *seqlens;
  const float *sink;
  int sink_mode;
  int B, N, max_new, max_len, Nq, Nkv, D, page, npages, width, W;  // W: 0 without a window
  int group, hblocks, gb;           // query heads per kv head; head blocks of gb heads per kv head
  int tpt;                          // tokens per query tile
  int s_lo, s_hi;                   // only sequences of [s_lo, s_hi] new tokens are this launch's
  float qscale, capmul;             // as in Params
  uint32_t *status, *tickets;
  float *partials;
  // norm and rotation (gqaw_paged_rows.cu)
  const void *qw, *kw, *rcos, *rsin;
  const long long *pos_ids;
  int rot_dim, rot_inter, rot_len;
  float eps;
  void *qout, *kout;                // gqaw_qk_norm_rotary: where the rows go
  long long qos, kos;
};

__device__ __forceinline__ PShape shape_of(const PagedParams &p, int unit_cost) {
  return PShape{p.tpt, p.W, p.Nkv * p.hblocks, unit_cost};
}

__device__ __forceinline__ PBatch batch_of(const PagedParams &p) {
  return PBatch{p.qstart, p.seqlens, p.B, p.N, p.max_new, p.max_len};
}

__device__ __forceinline__ void pflag(const PagedParams &p, uint32_t bits) { atomicOr(p.status, bits); }

// Builds the list and this CTA's start; all threads of the CTA call it, and it ends with a
// barrier.  One warp does it all, since what it takes is a chain of latencies: spread over the
// CTA, barriers and the sums over warps made it longer (2.7 us for one sequence).  CTA 0
// flags the malformed sequences.
template <int KEYS>
__device__ inline void sched_build(const PagedParams &p, const PShape &shp, PSched *s) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, heads = shp.heads;
    long long base = 0, units = 0;
    int count = 0, longest = 0;
    auto at = [&](const int32_t *x, int b, int end) { return b < end ? x[b] : 0; };
    int q0 = at(p.qstart, lane, p.B + 1), q1 = at(p.qstart, lane + 1, p.B + 1), len = at(p.seqlens, lane, p.B);
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int b = b0 + lane, S = q1 - q0, qs = q0;
      const long long TT = (long long)len + 1;
      const bool bad = b < p.B && malformed(batch_of(p), q0, q1, len);
      if (b0 + 32 < p.B) {  // the next ones, ahead of the arithmetic
        q0 = at(p.qstart, b + 32, p.B + 1);
        q1 = at(p.qstart, b + 33, p.B + 1);
        len = at(p.seqlens, b + 32, p.B);
      }
      long long n = 0, u = 0;
      int mx = 0;
      const bool has = b < p.B && !bad && S >= p.s_lo && S <= p.s_hi;
      if (bad && blockIdx.x == 0) pflag(p, GQAW_DEV_BAD_SEQLEN);
      if (has) {
        const PTiles<KEYS> t(shp, (int)TT, S);
        n = t.before(t.rt) * heads;
        u = (long long)t.rt * heads;
        mx = t.most();
      }
      const uint32_t vote = __ballot_sync(0xffffffffu, has);
      if (!vote) continue;
      long long in = n, iu = u;  // inclusive scans
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, in, o);
        const long long y = __shfl_up_sync(0xffffffffu, iu, o);
        if (lane >= o) in += x, iu += y;
      }
      if (has) s->items[count + __popc(vote & ((1u << lane) - 1u))] = PItem{base + in - n, units + iu - u, b, (int)TT, qs, S};
      count += __popc(vote);
      longest = max(longest, __reduce_max_sync(0xffffffffu, mx));
      base += __shfl_sync(0xffffffffu, in, 31);
      units += __shfl_sync(0xffffffffu, iu, 31);
    }
    if (lane == 0) {
      s->V = base;
      s->n = count;
      s->U = units;
      s->longest = longest;
    }
    __syncwarp();
    const PStart w = sched_start<KEYS>(shp, s, blockIdx.x, gridDim.x);
    if (lane == 0) s->start = w;
  }
  __syncthreads();
}

// Row offset (elements) of position j of sequence b, kv head h; -1 when its table entry is bad.
__device__ __forceinline__ long long cache_row(const PagedParams &p, int b, int h, int j) {
  const int pg = j / p.page;
  const int id = p.table[(long long)b * p.width + pg];
  if ((unsigned)id >= (unsigned)p.npages) return -1;
  return id * p.sp + h * p.sh + (long long)(j - pg * p.page) * p.sr;
}

__device__ __forceinline__ float paged_sink_log2(const PagedParams &p, int h) {
  if (p.sink_mode == 1) return p.sink[h] * kLog2e;
  return p.sink_mode == 2 ? 0.f : -INFINITY;
}

// A row of a cut unit from the partial results of CTAs [cf, cl], for this thread's elements d, d +
// 128, ...: at(c) is the row in CTA c's block, D weighted sums and behind them the row's maximum
// (log2) and sum of weights.  Eight parts are loaded before the first is used, since each is a
// round trip to L2 (19 parts one after the other took 20 us); their order is fixed.
template <int D, int ND, typename At>
__device__ __forceinline__ void merge_row(int cf, int cl, int d, At at, float &M, float &S, float (&A)[ND]) {
  M = -INFINITY;
  S = 0.f;
#pragma unroll
  for (int k = 0; k < ND; ++k) A[k] = 0.f;
  for (int c0 = cf; c0 <= cl; c0 += 8) {
    float m[8], s[8], a[8][ND];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool in = c0 + i <= cl;
      const float *q = at(in ? c0 + i : cl);
      m[i] = in ? __ldcg(q + D) : -INFINITY;
      s[i] = in ? __ldcg(q + D + 1) : 0.f;
#pragma unroll
      for (int k = 0; k < ND; ++k) a[i][k] = in && d + k * 128 < D ? __ldcg(q + d + k * 128) : 0.f;
    }
    float top = M;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, m[i]);
    const float ref = top == -INFINITY ? 0.f : top, f0 = exp2f(M - ref);
    S *= f0;
#pragma unroll
    for (int k = 0; k < ND; ++k) A[k] *= f0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = exp2f(m[i] - ref);
      S = fmaf(f, s[i], S);
#pragma unroll
      for (int k = 0; k < ND; ++k) A[k] = fmaf(f, a[i][k], A[k]);
    }
    M = top;
  }
}

// softcap: tanh with its own saturation; an absolute error of about 1e-7
__device__ __forceinline__ float cap_logit(const PagedParams &p, float x) { return p.capmul * tanhf(x); }

}  // namespace gqaw
