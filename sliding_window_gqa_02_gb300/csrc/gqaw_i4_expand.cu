// gqaw_i4_expand.cu -- the rows of a 4-bit cache that prompt chunks attend, as bf16 pages of 128 rows in the
// workspace, with a page table of their own: what the prompt kernels for bf16 caches then read.
//
// Worth it where a sequence has more than one query tile: in the kernel that takes codes
// (gqaw_i4_tiles.cuh) every query tile converts all its key tiles again, beside the softmax and on the same
// issue slots, while here each is converted once (8 chunks of 512 tokens with a window of 4096: 479 us
// there, 365 here, of which this pass is 43).
//
// Bound: HBM, mostly the writes (3.6 times the bytes of the codes).  A task is 128 rows of one head, keys or
// values; a warp has 32 of them, a lane 16 bytes of codes a row and 64 bytes of values, all loads ahead of the
// first use.  The list of tasks is made on the device, as the attention's schedule is: every CTA counts the
// tiles of the batch's sequences.
#include "gqaw_i4_tiles.cuh"

namespace gqaw {

namespace {
constexpr int kThreads = 128;
}

// Where the expanded pages go.
struct I4Expand {
  __nv_bfloat16 *k, *v;  // (pages, kv heads, 128, D)
  int32_t *table;        // (B, width)
  int width, pages;
};

template <int D>
__global__ void __launch_bounds__(kThreads) i4_expand_kernel(const I4Params p, const I4Expand x) {
  constexpr int CPR = D / 32, RPC = 32 / CPR;  // lanes of a row, rows of a load
  __shared__ int s_first[kPagedItems + 1], s_lo[kPagedItems];  // pages before a sequence's; its first tile
  __shared__ uint32_t s_from[kPagedItems], s_to[kPagedItems];  // positions that it attends
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  if (warp == 0) {
    int base = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int b = b0 + lane;
      int n = 0;
      if (b < p.B) {
        const int q0 = p.qstart[b], q1 = p.qstart[b + 1], len = p.seqlens[b], S = q1 - q0;
        if (!malformed(batch_of(p), q0, q1, len) && S >= p.s_lo && S <= p.s_hi) {
          const long long T = (long long)len + 1, first = p.W > 0 && T - S - p.W + 1 > 0 ? T - S - p.W + 1 : 0;
          s_from[b] = (uint32_t)first;
          s_to[b] = (uint32_t)T;
          s_lo[b] = (int)(first / 128);
          n = (int)((T - 1) / 128) + 1 - s_lo[b];
        }
      }
      int in = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, in, o);
        if (lane >= o) in += y;
      }
      if (b < p.B) s_first[b] = base + in - n;
      base += __shfl_sync(0xffffffffu, in, 31);
    }
    if (lane == 0) s_first[p.B] = base;
  }
  __syncthreads();
  const int pages = min(s_first[p.B], x.pages);  // the workspace holds what the sizes allow
  const long long tasks = (long long)pages * p.Nkv * 2;
  const int row = lane / CPR, part = lane % CPR;
  for (long long t = blockIdx.x; t < tasks; t += gridDim.x) {
    const int pg = (int)(t / (p.Nkv * 2)), rest = (int)(t - (long long)pg * (p.Nkv * 2)), kvh = rest >> 1;
    const bool value = rest & 1;
    int b = 0;  // the last sequence with s_first[b] <= pg, and so one with pages
    for (int lo = 0, hi = p.B; lo < hi;) {
      const int mid = (lo + hi) / 2;
      if (s_first[mid] <= pg)
        b = mid, lo = mid + 1;
      else
        hi = mid;
    }
    const int tile = s_lo[b] + pg - s_first[b];
    if (rest == 0 && tid == 0) x.table[(long long)b * x.width + tile] = pg;
    const uint32_t j0 = (uint32_t)tile * 128 + warp * 32 + row, from = s_from[b], to = s_to[b];
    const int32_t *table = p.table + (long long)b * p.width;
    int id[CPR];
#pragma unroll
    for (int c = 0; c < CPR; ++c) {
      const uint32_t j = j0 + c * RPC;
      id[c] = j >= from && j < to ? needed_page(__ldg(table + (uint32_t)(((uint64_t)j * p.div_mul) >> p.div_shift))) : kNotNeeded;
    }
    uint4 codes[CPR];
    uint32_t scale[CPR];
    const uint4 *base = reinterpret_cast<const uint4 *>(static_cast<const unsigned char *>(value ? p.vp : p.kp) + kvh * p.sh);
    const uint16_t *sbase = (value ? p.vscale : p.kscale) + kvh * p.th + part;
    bool bad = false;
#pragma unroll
    for (int c = 0; c < CPR; ++c) {
      const uint32_t j = j0 + c * RPC, r = j - (uint32_t)(((uint64_t)j * p.div_mul) >> p.div_shift) * p.page;
      const bool ok = (unsigned)id[c] < (unsigned)p.npages;
      bad |= !ok && id[c] != kNotNeeded;
      codes[c] = make_uint4(0u, 0u, 0u, 0u);
      scale[c] = 0u;
      if (ok) {
        codes[c] = __ldcs(base + ((uint64_t)(uint32_t)id[c] * p.sp16 + (uint64_t)r * p.sr16 + part));
        scale[c] = __ldg(sbase + ((uint64_t)(uint32_t)id[c] * p.tpg + (uint64_t)r * p.trg) * (D / kI4Group));
      }
    }
    if (bad) pflag(p, GQAW_DEV_BAD_PAGE);
    uint4 *out = reinterpret_cast<uint4 *>((value ? x.v : x.k) + (((long long)pg * p.Nkv + kvh) * 128 + warp * 32 + row) * D) + part * 4;
#pragma unroll
    for (int c = 0; c < CPR; ++c) {
      const uint32_t s2 = scale[c] * 0x10001u;
      const uint32_t w[4] = {codes[c].x, codes[c].y, codes[c].z, codes[c].w};
#pragma unroll
      for (int y = 0; y < 4; ++y) out[c * RPC * (D / 8) + y] = i4t::values8<false>(w[y], s2, 0u, true);
    }
  }
  pdl_launch_dependents();
}

cudaError_t launch_i4_expand(const I4Params &p, void *k, void *v, int32_t *table, int width, int pages, int sms, cudaStream_t stream) {
  const I4Expand x{static_cast<__nv_bfloat16 *>(k), static_cast<__nv_bfloat16 *>(v), table, width, pages};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sms * 8));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see pdl_wait()
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  switch (p.D) {
    case 64: e = cudaLaunchKernelEx(&cfg, i4_expand_kernel<64>, p, x); break;
    case 128: e = cudaLaunchKernelEx(&cfg, i4_expand_kernel<128>, p, x); break;
    default: e = cudaLaunchKernelEx(&cfg, i4_expand_kernel<256>, p, x);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gqaw
