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
// A row is spread over the warps of one CTA (one warp for short rows, and
// then four rows a CTA), NV 16-byte groups a thread.  The grid is as many
// CTAs as fit the GPU, each walking over rows, so the next row's loads are in
// flight while this row is reduced.  What a modulation row and the weights
// bring, as three fp32 vectors
//   A = gate' * post_weight,  B = pre_weight * (1 + scale),  C = shift,
// is worked out once per modulation row (with its tanh) and kept in shared
// memory, each thread its own channels (no barrier; unpacking them per row
// instead was a third of the instructions, which bound the kernel).
// On long walks the row after the next is asked into L2 meanwhile, so that the
// registers' one row of loads need not cover HBM's latency: 14,042 x 2312
// between two norms 58.8 -> 55.5 us, 51,000 x 144 23.2 -> 21.2, 4608 x 3072 the
// same.  Below seven rows a CTA it only adds requests to the first rows' (2000 x
// 5120 19.0 -> 19.4 us, 4096 x 1152 13.3 -> 13.8).
// Statistics take one barrier a norm: each warp's mean and sum of squares
// about it, merged exactly, so a row far from zero keeps its digits.
#include "internal.h"
#include "kernel_common.cuh"
#include "ptx.cuh"

namespace tern {

namespace {

constexpr int kNarrowRows = 4;     // rows (warps) of a CTA where a warp holds a row
constexpr int kWideThreads = 512;  // 128 registers a thread; 16384 channels are 2048 groups, four a thread

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ void unpack8(uint4 v, float2 (&f)[4]) {
  f[0] = make_float2(lo_f(v.x), hi_f(v.x)), f[1] = make_float2(lo_f(v.y), hi_f(v.y));
  f[2] = make_float2(lo_f(v.z), hi_f(v.z)), f[3] = make_float2(lo_f(v.w), hi_f(v.w));
}
__device__ __forceinline__ uint4 pack8(const float2 (&f)[4]) {
  return make_uint4(pack2(f[0].x, f[0].y), pack2(f[1].x, f[1].y), pack2(f[2].x, f[2].y), pack2(f[3].x, f[3].y));
}

// (mean, biased variance about it) of a row, or (0, mean square) for RMS, from
// each thread's groups: within the warp by shuffles, then over the CTA's
// warps (WIDE) through `buf`, one barrier.  A warp holds `mine` values.
template <int NV, bool WIDE>
__device__ __forceinline__ float2 row_stats(const float2 (&f)[NV][4], bool layer, float inv_k, int n8, int first, int step,
                                            float mine, float inv_mine, float4* buf) {
  float mean = 0.f;
  if (layer) {
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int t = 0; t < NV; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) s = add2(s, f[t][e]);  // absent groups are zeros
    float sum = s.x + s.y;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    mean = sum * inv_mine;
  }
  float2 q = make_float2(0.f, 0.f);
  const float2 neg = make_float2(-mean, -mean);
#pragma unroll
  for (int t = 0; t < NV; ++t)
    if (first + t * step < n8)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 d = add2(f[t][e], neg);
        q = fma2(d, d, q);
      }
  float sq = q.x + q.y;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, off);
  if constexpr (WIDE) {
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = make_float4(mine, mean, sq, 0.f);
    __syncthreads();
    const int warps = int(blockDim.x) >> 5;
    if (layer) {
      float total = 0.f;
      for (int w = 0; w < warps; ++w) total = fmaf(buf[w].x, buf[w].y, total);
      mean = total * inv_k;
    }
    sq = 0.f;
    for (int w = 0; w < warps; ++w) {
      const float4 v = buf[w];
      const float d = v.y - mean;
      sq += fmaf(v.x * d, d, v.z);
    }
  }
  return make_float2(mean, sq * inv_k);
}

// f <- (f - mean) / sqrt(var + eps)
template <int NV, bool WIDE>
__device__ __forceinline__ void normalise(float2 (&f)[NV][4], int kind, float eps, float inv_k, int n8, int first, int step,
                                          float mine, float inv_mine, float4* buf) {
  if (kind == kNormNone) return;
  const float2 st = row_stats<NV, WIDE>(f, kind == kNormLayer, inv_k, n8, first, step, mine, inv_mine, buf);
  const float r = rsqrtf(st.y + eps);
  const float2 neg = make_float2(-st.x, -st.x), rstd = make_float2(r, r);
#pragma unroll
  for (int t = 0; t < NV; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) f[t][e] = mul2(add2(f[t][e], neg), rstd);
}

template <int NV, bool WIDE>
__global__ void __launch_bounds__(WIDE ? kWideThreads : kNarrowRows * 32, WIDE ? 1 : 4)
    gated_residual_norm_kernel(const __grid_constant__ ResNormArgs a) {
  __shared__ float4 buf[WIDE ? 4 : 1][WIDE ? kWideThreads / 32 : 1];  // [row parity, post or pre]
  extern __shared__ float4 mod_smem[];  // [3 vectors][NV groups][2][threads]
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n8 = a.K >> 3;
  const int first = WIDE ? int(threadIdx.x) : lane, step = WIDE ? int(blockDim.x) : 32;
  int groups = 0;  // of this warp's lanes
#pragma unroll
  for (int t = 0; t < NV; ++t) groups += max(0, min(32, n8 - (first - lane) - t * step));
  const float mine = 8.f * float(groups), inv_mine = groups > 0 ? 1.f / mine : 0.f, inv_k = 1.f / float(a.K);
  unsigned m = WIDE ? blockIdx.x : blockIdx.x * kNarrowRows + warp;
  const unsigned M = unsigned(a.M), rows = WIDE ? gridDim.x : gridDim.x * kNarrowRows;
  // This thread's first group of the row, in steps of `rows` rows (bytes).
  const uint8_t* xp = reinterpret_cast<const uint8_t*>(a.x + m * a.ld_x) + 16 * first;
  const uint8_t* op = reinterpret_cast<const uint8_t*>(a.o + m * a.ld_o) + 16 * first;
  uint8_t* xop = reinterpret_cast<uint8_t*>(a.x_out + m * a.ld_xo) + 16 * first;
  uint8_t* hp = reinterpret_cast<uint8_t*>(a.h + m * a.ld_h) + 16 * first;
  const long long x_step = 2 * a.ld_x * rows, o_step = 2 * a.ld_o * rows, xo_step = 2 * a.ld_xo * rows,
                  h_step = 2 * a.ld_h * rows;
  uint4 xv[NV], ov[NV];
  auto load = [&]() {
#pragma unroll
    for (int t = 0; t < NV; ++t) {
      const bool in = first + t * step < n8;
      ov[t] = in ? *reinterpret_cast<const uint4*>(op + 16 * t * step) : make_uint4(0u, 0u, 0u, 0u);
      xv[t] = in ? *reinterpret_cast<const uint4*>(xp + 16 * t * step) : make_uint4(0u, 0u, 0u, 0u);
    }
    xp += x_step;
    op += o_step;
  };
  // This thread's part of A, B and C.
  auto vec = [&](int v, int t, int half) -> float4& {
    return mod_smem[((v * NV + t) * 2 + half) * blockDim.x + threadIdx.x];
  };
  auto put = [&](int v, int t, const float2 (&f)[4]) {
    vec(v, t, 0) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    vec(v, t, 1) = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
  };
  auto get = [&](int v, int t, float2 (&f)[4]) {
    const float4 p = vec(v, t, 0), q = vec(v, t, 1);
    f[0] = make_float2(p.x, p.y), f[1] = make_float2(p.z, p.w), f[2] = make_float2(q.x, q.y), f[3] = make_float2(q.z, q.w);
  };
  const bool has_a = a.gate || a.post_weight, has_b = a.scale || a.pre_weight;
  if (m < M) load();
  const bool ahead = M > 7 * rows && (WIDE ? threadIdx.x == 0 : lane == 0);
  unsigned g_end = m;  // first row past the modulation row that A, B and C hold
  const float2 alpha = make_float2(a.residual_scale, a.residual_scale), one = make_float2(1.f, 1.f);
  for (int parity = 0; m < M; m += rows, parity ^= 2, xop += xo_step, hp += h_step) {
    if (m >= g_end) {
      const unsigned T = unsigned(a.tokens_per_row), q = m / T;
      const long long g = q;
      g_end = (M - q * T > T) ? (q + 1) * T : M;
      for (int t = 0; t < NV; ++t) {
        const int i = first + t * step;
        if (i >= n8) break;
        float2 f[4], w[4];
        if (has_a) {
          f[0] = f[1] = f[2] = f[3] = one;
          if (a.gate) {
            unpack8(__ldg(reinterpret_cast<const uint4*>(a.gate + g * a.mod_ld) + i), f);
            if (a.gate_tanh)
#pragma unroll
              for (int e = 0; e < 4; ++e) f[e] = make_float2(tanhf(f[e].x), tanhf(f[e].y));
          }
          if (a.post_weight) {
            unpack8(__ldg(reinterpret_cast<const uint4*>(a.post_weight) + i), w);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = mul2(f[e], w[e]);
          }
          put(0, t, f);
        }
        if (has_b) {
          f[0] = f[1] = f[2] = f[3] = one;
          if (a.scale) {
            unpack8(__ldg(reinterpret_cast<const uint4*>(a.scale + g * a.mod_ld) + i), f);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = add2(f[e], one);
          }
          if (a.pre_weight) {
            unpack8(__ldg(reinterpret_cast<const uint4*>(a.pre_weight) + i), w);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = mul2(f[e], w[e]);
          }
          put(1, t, f);
          f[0] = f[1] = f[2] = f[3] = make_float2(0.f, 0.f);
          if (a.shift) unpack8(__ldg(reinterpret_cast<const uint4*>(a.shift + g * a.mod_ld) + i), f);
          put(2, t, f);
        }
      }
    }
    float2 f[NV][4];
#pragma unroll
    for (int t = 0; t < NV; ++t) unpack8(ov[t], f[t]);
    normalise<NV, WIDE>(f, a.post, a.post_eps, inv_k, n8, first, step, mine, inv_mine, buf[WIDE ? parity : 0]);
#pragma unroll
    for (int t = 0; t < NV; ++t) {
      const int i = first + t * step;
      float2 xf[4];
      unpack8(xv[t], xf);
      if (i < n8) {
        if (has_a) {
          float2 v[4];
          get(0, t, v);
#pragma unroll
          for (int e = 0; e < 4; ++e) f[t][e] = mul2(f[t][e], v[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) f[t][e] = fma2(alpha, xf[e], f[t][e]);
        *reinterpret_cast<uint4*>(xop + 16 * t * step) = pack8(f[t]);
      } else {
        f[t][0] = f[t][1] = f[t][2] = f[t][3] = make_float2(0.f, 0.f);
      }
    }
    if (rows < M - m) load();
    if (ahead && 2 * rows < M - m) {
      const long long row = m + 2 * (long long)rows;
      prefetch_l2_bulk(a.x + row * a.ld_x, uint32_t(a.K) * 2);
      prefetch_l2_bulk(a.o + row * a.ld_o, uint32_t(a.K) * 2);
    }
    if (!a.h) continue;
    normalise<NV, WIDE>(f, a.pre, a.pre_eps, inv_k, n8, first, step, mine, inv_mine, buf[WIDE ? parity + 1 : 0]);
#pragma unroll
    for (int t = 0; t < NV; ++t) {
      const int i = first + t * step;
      if (i < n8) {
        if (has_b) {
          float2 v[4], w[4];
          get(1, t, v);
          get(2, t, w);
#pragma unroll
          for (int e = 0; e < 4; ++e) f[t][e] = fma2(f[t][e], v[e], w[e]);
        }
        *reinterpret_cast<uint4*>(hp + 16 * t * step) = pack8(f[t]);
      }
    }
  }
}

template <int NV, bool WIDE>
cudaError_t launch_one(const ResNormArgs& a, int warps, int sms, cudaStream_t stream) {
  const int threads = WIDE ? warps * 32 : kNarrowRows * 32;
  const int smem = 96 * NV * threads;
  // Once per device: shared memory above 48 KB; once per block size as well: how many CTAs fit an SM.
  static thread_local int ready_dev = -1, ready_threads = 0, ctas = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (ready_dev != dev || ready_threads != threads) {
    e = cudaFuncSetAttribute(gated_residual_norm_kernel<NV, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             96 * NV * (WIDE ? kWideThreads : kNarrowRows * 32));
    if (e != cudaSuccess) return e;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, gated_residual_norm_kernel<NV, WIDE>, threads, smem);
    if (e != cudaSuccess) return e;
    ready_dev = dev, ready_threads = threads;
  }
  const long long need = WIDE ? a.M : (a.M + kNarrowRows - 1) / kNarrowRows, fit = (long long)max(ctas, 1) * sms;
  return launch_pdl(gated_residual_norm_kernel<NV, WIDE>, dim3(unsigned(need < fit ? need : fit)), dim3(threads), smem,
                    stream, 1, a);
}

}  // namespace

cudaError_t launch_gated_residual_norm(const ResNormArgs& a, int sms, cudaStream_t stream) {
  const int n8 = a.K >> 3;
  if (n8 <= 32) return launch_one<1, false>(a, 1, sms, stream);
  if (n8 <= 64) return launch_one<2, false>(a, 1, sms, stream);
  if (n8 <= 96) return launch_one<3, false>(a, 1, sms, stream);
  // Three groups a thread: at 4608 x 3072 22.5 us, against 26 with two (more
  // warps in each reduction) and 24.8 with four (fewer rows on an SM).
  if (n8 <= 3 * kWideThreads) return launch_one<3, true>(a, (n8 + 95) / 96, sms, stream);
  return launch_one<4, true>(a, (n8 + 127) / 128, sms, stream);
}

}  // namespace tern
