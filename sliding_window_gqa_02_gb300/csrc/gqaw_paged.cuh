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

__device__ __forceinline__ void pflag(const PagedParams &p, uint32_t bits) { atomicOr(p.status, bits); }

// Builds the list and this CTA's start; all `nt` threads of the CTA (a multiple of 32) call
// it, and it ends with a barrier.  CTA 0 flags the malformed sequences.
template <int KEYS>
__device__ inline void sched_build(const PagedParams &p, const PShape &shp, PSched *s, int nt) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
  const int heads = p.Nkv * p.hblocks;
  long long base = 0, units = 0;
  int count = 0, longest = 0;
  for (int b0 = 0; b0 < p.B; b0 += nt) {
    const int b = b0 + tid;
    long long n = 0, u = 0;
    int mx = 0, has = 0, T = 0, q0 = 0, S = 0;
    if (b < p.B) {
      q0 = p.qstart[b];
      const int q1 = p.qstart[b + 1];
      const long long TT = (long long)p.seqlens[b] + 1;
      S = q1 - q0;
      if (q0 < 0 || q1 < q0 || q1 > p.N || S > p.max_new || TT < S || TT > p.max_len) {
        if (blockIdx.x == 0) pflag(p, GQAW_DEV_BAD_SEQLEN);
      } else if (S >= p.s_lo && S <= p.s_hi) {
        T = (int)TT;
        const PTiles<KEYS> t(shp, T, S);
        has = 1;
        n = t.before(t.rt) * heads;
        u = (long long)t.rt * heads;
        mx = t.most();
      }
    }
    long long in = n, iu = u;  // inclusive scans over the warp, then over the warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, in, o);
      const long long y = __shfl_up_sync(0xffffffffu, iu, o);
      if (lane >= o) in += x, iu += y;
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    const uint32_t vote = __ballot_sync(0xffffffffu, has);
    if (lane == 31) {
      s->wsum[warp] = in;
      s->wunits[warp] = iu;
      s->wcnt[warp] = __popc(vote);
      s->wmax[warp] = mx;
    }
    __syncthreads();
    long long at = base + in - n, au = units + iu - u;
    int ac = count + __popc(vote & ((1u << lane) - 1u));
    for (int w = 0; w < nw; ++w) {
      if (w < warp) at += s->wsum[w], au += s->wunits[w], ac += s->wcnt[w];
      base += s->wsum[w];
      units += s->wunits[w];
      count += s->wcnt[w];
      longest = max(longest, s->wmax[w]);
    }
    if (has) s->items[ac] = PItem{at, au, b, T, q0, S};
    __syncthreads();
  }
  if (tid == 0) {
    s->V = base;
    s->n = count;
    s->U = units;
    s->longest = longest;
    sched_start<KEYS>(shp, s, blockIdx.x, gridDim.x);
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

// softcap: tanh with its own saturation; an absolute error of about 1e-7
__device__ __forceinline__ float cap_logit(const PagedParams &p, float x) { return p.capmul * tanhf(x); }

}  // namespace gqaw
