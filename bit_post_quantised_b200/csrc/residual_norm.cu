// residual_norm.cu -- the gated residual update of a transformer block with
// the norm before the next one, in one pass over HBM.
//
// Per token row m, g = m / tokens_per_row:
//   r = residual_scale * x[m] + gate[g] * post(o[m])      (gate or tanh(gate); 1 where none is given)
//   x_out[m] = r
//   h[m] = pre(r) * (1 + scale[g]) + shift[g]
// with post and pre each nothing, RMS normalisation or layer normalisation,
// with an optional weight per channel.  Unfused that is two normalisations,
// a product, a sum and a modulation, each reading and writing the stream;
// here x and o are read once and x_out and h written once (8 bytes per
// element: bound by HBM).  The row stays in registers in fp32 between the
// steps: h is taken from r before r is rounded for x_out, and each output is
// rounded once.
//
// A row is spread over `warps` warps of one CTA (one warp for short rows, and
// then eight rows a CTA), NV 16-byte groups a thread: 3 groups keep x, o and
// r in registers at an occupancy that covers HBM's latency.  Layer norms take
// the mean first and then the variance about it.
#include "internal.h"
#include "kernel_common.cuh"
#include "ptx.cuh"

namespace tern {

namespace {

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ void unpack8(uint4 v, float* f) {
  f[0] = lo_f(v.x), f[1] = hi_f(v.x), f[2] = lo_f(v.y), f[3] = hi_f(v.y);
  f[4] = lo_f(v.z), f[5] = hi_f(v.z), f[6] = lo_f(v.w), f[7] = hi_f(v.w);
}

// Sum over the threads of a row: the warp, then (WIDE) the CTA's warps
// through shared memory.  `buf` alternates between calls so that one barrier
// a call is enough.
template <bool WIDE>
__device__ __forceinline__ float row_sum(float v, float* buf, int warps) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if constexpr (WIDE) {
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < warps; ++w) v += buf[w];
  }
  return v;
}

// Normalises the row in f (groups past n8 hold zeros and stay out of the
// variance), then multiplies by the weight.
template <int NV, bool WIDE>
__device__ __forceinline__ void normalise(float (&f)[NV][8], int kind, float eps, const uint16_t* weight, int K, int n8,
                                          int first, int step, float* buf, int warps) {
  if (kind == kNormNone) return;
  float mean = 0.f;
  if (kind == kNormLayer) {
    float sum = 0.f;
#pragma unroll
    for (int t = 0; t < NV; ++t)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += f[t][e];
    mean = row_sum<WIDE>(sum, buf, warps) / float(K);
  }
  float sq = 0.f;
#pragma unroll
  for (int t = 0; t < NV; ++t)
    if (first + t * step < n8)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[t][e] -= mean;
        sq = fmaf(f[t][e], f[t][e], sq);
      }
  const float rstd = rsqrtf(row_sum<WIDE>(sq, buf + 32, warps) / float(K) + eps);
#pragma unroll
  for (int t = 0; t < NV; ++t) {
    const int i = first + t * step;
    if (i < n8) {
      float w[8];
      if (weight) unpack8(__ldg(reinterpret_cast<const uint4*>(weight) + i), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[t][e] = f[t][e] * rstd * (weight ? w[e] : 1.f);
    }
  }
}

template <int NV, bool WIDE>
__global__ void __launch_bounds__(WIDE ? 1024 : 256) gated_residual_norm_kernel(const __grid_constant__ ResNormArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ float buf[WIDE ? 128 : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long m = WIDE ? (long long)blockIdx.x : (long long)blockIdx.x * 8 + warp;
  if (m >= a.M) return;
  const int first = WIDE ? int(threadIdx.x) : lane, step = WIDE ? int(blockDim.x) : 32;
  const int warps = WIDE ? int(blockDim.x) >> 5 : 1, n8 = a.K >> 3;
  const long long g = m / a.tokens_per_row;
  uint4 xv[NV];
  float f[NV][8];
  const uint4* x = reinterpret_cast<const uint4*>(a.x + m * a.ld_x);
  const uint4* o = reinterpret_cast<const uint4*>(a.o + m * a.ld_o);
  {
    uint4 ov[NV];
#pragma unroll
    for (int t = 0; t < NV; ++t) {
      const int i = first + t * step;
      ov[t] = i < n8 ? o[i] : make_uint4(0u, 0u, 0u, 0u);
      xv[t] = i < n8 ? x[i] : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int t = 0; t < NV; ++t) unpack8(ov[t], f[t]);
  }
  normalise<NV, WIDE>(f, a.post, a.post_eps, a.post_weight, a.K, n8, first, step, buf, warps);
  uint4* xo = reinterpret_cast<uint4*>(a.x_out + m * a.ld_xo);
#pragma unroll
  for (int t = 0; t < NV; ++t) {
    const int i = first + t * step;
    if (i < n8) {
      float xf[8], gt[8];
      unpack8(xv[t], xf);
      if (a.gate) {
        unpack8(__ldg(reinterpret_cast<const uint4*>(a.gate + g * a.mod_ld) + i), gt);
        if (a.gate_tanh)
#pragma unroll
          for (int e = 0; e < 8; ++e) gt[e] = tanhf(gt[e]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) f[t][e] = fmaf(a.residual_scale, xf[e], a.gate ? gt[e] * f[t][e] : f[t][e]);
      xo[i] = make_uint4(pack2(f[t][0], f[t][1]), pack2(f[t][2], f[t][3]), pack2(f[t][4], f[t][5]),
                         pack2(f[t][6], f[t][7]));
    }
  }
  if (!a.h) return;
  normalise<NV, WIDE>(f, a.pre, a.pre_eps, a.pre_weight, a.K, n8, first, step, buf + 64, warps);
  uint4* h = reinterpret_cast<uint4*>(a.h + m * a.ld_h);
#pragma unroll
  for (int t = 0; t < NV; ++t) {
    const int i = first + t * step;
    if (i < n8) {
      if (a.scale) {
        float sc[8], sh[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(a.scale + g * a.mod_ld) + i), sc);
        unpack8(__ldg(reinterpret_cast<const uint4*>(a.shift + g * a.mod_ld) + i), sh);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[t][e] = fmaf(f[t][e], 1.f + sc[e], sh[e]);
      }
      h[i] = make_uint4(pack2(f[t][0], f[t][1]), pack2(f[t][2], f[t][3]), pack2(f[t][4], f[t][5]),
                        pack2(f[t][6], f[t][7]));
    }
  }
}

template <int NV, bool WIDE>
cudaError_t launch_one(const ResNormArgs& a, int warps, cudaStream_t stream) {
  const long long grid = WIDE ? a.M : (a.M + 7) / 8;
  return launch_pdl(gated_residual_norm_kernel<NV, WIDE>, dim3(unsigned(grid)), dim3(WIDE ? warps * 32 : 256), 0, stream,
                    1, a);
}

}  // namespace

cudaError_t launch_gated_residual_norm(const ResNormArgs& a, cudaStream_t stream) {
  const int n8 = a.K >> 3;
  if (n8 <= 32) return launch_one<1, false>(a, 1, stream);
  if (n8 <= 64) return launch_one<2, false>(a, 1, stream);
  if (n8 <= 96) return launch_one<3, false>(a, 1, stream);
  return launch_one<3, true>(a, (n8 + 95) / 96, stream);
}

}  // namespace tern
