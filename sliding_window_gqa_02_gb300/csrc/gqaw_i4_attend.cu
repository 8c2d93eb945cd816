// gqaw_i4_attend.cu -- attention over a paged cache held in 4 bits.
//
//     o_i = sum_j softmax_j(cap(scale q_i k_j)) v_j,  j <= i (and j > i - W), with sinks,
// k and v being (c - 8) s of their codes.  A warp has one query head of one token and goes over
// the keys one by one; a lane has D / 32 dimensions.
#include "gqaw_i4.cuh"

namespace gqaw {

template <typename T, int D>
__global__ void __launch_bounds__(128) i4_attend_kernel(const I4Params p) {
  constexpr int VW = D / 32;
  const int lane = threadIdx.x & 31;
  pdl_wait();
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < p.B; b += blockDim.x)
      if (malformed(batch_of(p), p.qstart[b], p.qstart[b + 1], p.seqlens[b])) pflag(p, GQAW_DEV_BAD_SEQLEN);
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int n = (int)(w / p.Nq), h = (int)(w - (long long)n * p.Nq), kvh = h / p.group;
  const int b = n < p.N ? find_sequence(batch_of(p), n) : -1;
  if (b >= 0) {
    const long long i = (long long)p.seqlens[b] + 1 - (p.qstart[b + 1] - n), lo = p.W > 0 && i - p.W + 1 > 0 ? i - p.W + 1 : 0;
    float q[VW], o[VW], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int d = 0; d < VW; ++d) {
      const long long at = n * p.qs + (long long)h * D + lane * VW + d;
      q[d] = Elem<T>::load(static_cast<const T *>(p.q)[at]);
      if (p.qlo) q[d] += Elem<T>::load(static_cast<const T *>(p.qlo)[at]);
      q[d] *= p.qscale;
      o[d] = 0.f;
    }
    auto value = [&](const unsigned char *row, float s, int d) {
      const int el = lane * VW + d;
      return (float)((int)((row[el / 2] >> (4 * (el & 1))) & 15) - 8) * s;
    };
    for (long long j = lo; j <= i; ++j) {
      const I4Place at = i4_place(p, b, j);
      if (at.page < 0) {
        if (lane == 0) pflag(p, GQAW_DEV_BAD_PAGE);
        break;
      }
      const long long codes = at.page * p.sp + kvh * p.sh + at.row * p.sr, scales = at.page * p.tp + kvh * p.th + at.row * p.tr + lane * VW / kI4Group;
      const float ks = __uint_as_float((uint32_t)p.kscale[scales] << 16), vs = __uint_as_float((uint32_t)p.vscale[scales] << 16);
      float z = 0.f;
#pragma unroll
      for (int d = 0; d < VW; ++d) z = fmaf(q[d], value(static_cast<const unsigned char *>(p.kp) + codes, ks, d), z);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) z += __shfl_xor_sync(~0u, z, x);
      if (p.capmul != 0.f) z = cap_logit(p, z);
      const float top = fmaxf(m, z), base = top == -INFINITY ? 0.f : top, f = exp2f(m - base), e = exp2f(z - base);
      m = top;
      l = fmaf(l, f, e);
#pragma unroll
      for (int d = 0; d < VW; ++d) o[d] = fmaf(e, value(static_cast<const unsigned char *>(p.vp) + codes, vs, d), o[d] * f);
    }
    const float inv = sink_reciprocal(l, m, paged_sink_log2(p, h));
#pragma unroll
    for (int d = 0; d < VW; ++d) static_cast<T *>(p.out)[n * p.os + (long long)h * D + lane * VW + d] = Elem<T>::store(o[d] * inv);
  }
  pdl_launch_dependents();
}

template <typename T>
cudaError_t launch_i4_attend_t(const I4Params &p, const cudaLaunchConfig_t &cfg) {
  switch (p.D) {
    case 32: return cudaLaunchKernelEx(&cfg, i4_attend_kernel<T, 32>, p);
    case 64: return cudaLaunchKernelEx(&cfg, i4_attend_kernel<T, 64>, p);
    case 128: return cudaLaunchKernelEx(&cfg, i4_attend_kernel<T, 128>, p);
    default: return cudaLaunchKernelEx(&cfg, i4_attend_kernel<T, 256>, p);
  }
}

cudaError_t launch_i4_attend(const I4Params &p, bool bf16, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((long long)p.N * p.Nq + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see pdl_wait()
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = bf16 ? launch_i4_attend_t<__nv_bfloat16>(p, cfg) : launch_i4_attend_t<float>(p, cfg);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gqaw
