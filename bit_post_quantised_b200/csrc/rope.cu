// rope.cu -- rotary position embedding with several axes (time, height,
// width): the (cos, sin) table of token positions, and the rotation of query
// and key heads by it.
//
// Table: pair j of axis a (d_a channels, d_a / 2 pairs, i = the pair's place
// on its axis) of token m turns by ids[m, a] * theta^(-2 i / d_a).  Far
// positions turn by thousands of radians, where one fp32 ulp of the angle is
// already visible in its cosine, so the angle and its reduction to
// [-pi/4, pi/4] are in 64 bits.  There the sine and cosine are their Taylor
// polynomials (degrees 11 and 12: truncation below 7e-12), rounded once to
// fp32.  One thread owns one pair and walks over tokens, so its frequency
// stays in registers; stores are 8 bytes per lane, consecutive.
//
// Rotation: bound by HBM (each element read once, written once).  A thread
// owns one 16-byte group of channels of a token (or, for half-split pairs,
// the two groups that turn together) and walks over the heads of q and k, so
// the table, shared by all heads, is read once per token and stays in
// registers.  fp32 products, one rounding to bf16.
#include "internal.h"
#include "kernel_common.cuh"
#include "ptx.cuh"

namespace tern {

namespace {

// ------------------------------------------------------------------- table
constexpr int kTableThreads = 256;
constexpr int kTableRows = 4;  // token rows per thread

// cos and sin of `a`, |a| < 2^31 pi / 2, each rounded to fp32.
__device__ __forceinline__ float2 cos_sin(double a) {
  // n = the nearest multiple of pi/2, r = a - n pi/2 (pi/2 as two doubles).
  const double n = rint(a * 0.63661977236758134308);
  double r = fma(-n, 1.57079632679489661923, a);
  r = fma(-n, 6.12323399573676603587e-17, r);
  const double z = r * r;
  double s = fma(z, -1.0 / 39916800.0, 1.0 / 362880.0);
  s = fma(z, s, -1.0 / 5040.0);
  s = fma(z, s, 1.0 / 120.0);
  s = fma(z, s, -1.0 / 6.0);
  s = fma(z * r, s, r);
  double c = fma(z, 1.0 / 479001600.0, -1.0 / 3628800.0);
  c = fma(z, c, 1.0 / 40320.0);
  c = fma(z, c, -1.0 / 720.0);
  c = fma(z, c, 1.0 / 24.0);
  c = fma(z, c, -0.5);
  c = fma(z, c, 1.0);
  const float fs = float(s), fc = float(c);
  const int q = __double2int_rn(n) & 3;  // quarter turns
  const float cc = (q & 1) ? fs : fc, ss = (q & 1) ? fc : fs;
  return make_float2((q == 1 || q == 2) ? -cc : cc, (q >= 2) ? -ss : ss);
}

__global__ void __launch_bounds__(kTableThreads)
    rope_table_kernel(const float* __restrict__ ids, long long L, const __grid_constant__ RopeFreqs f, float2* cs) {
  pdl_wait();
  pdl_trigger();
  const int P = f.pairs;
  const int rows = kTableThreads / P;  // token rows side by side
  const int j = threadIdx.x % P, r = threadIdx.x / P;
  if (r >= rows) return;
  const double omega = f.omega[j];
  const int axis = f.axis[j];
  const long long m0 = (long long)blockIdx.x * (rows * kTableRows) + r;
#pragma unroll
  for (int t = 0; t < kTableRows; ++t) {
    const long long m = m0 + t * rows;
    if (m < L) cs[m * P + j] = cos_sin(double(ids[m * f.n_axes + axis]) * omega);
  }
}

// ---------------------------------------------------------------- rotation
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// The adjacent pair (a, b) of one word turned by (c, s).
__device__ __forceinline__ uint32_t turn(uint32_t w, float c, float s) {
  const float a = lo_f(w), b = hi_f(w);
  return pack2(a * c - b * s, a * s + b * c);
}

// Threads of a block: slot = tid / units owns (token row of the block, first
// head), unit = tid % units one group of channels; both fixed, so the table
// entries stay in registers while the thread walks over heads.
template <bool HALVES>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ RopeArgs a) {
  pdl_wait();
  pdl_trigger();
  const int unit = threadIdx.x % a.units, slot = threadIdx.x / a.units;
  const int row = slot / a.heads_par, h0 = slot - row * a.heads_par;
  const long long m = (long long)blockIdx.x * a.rows_par + row;
  if (row >= a.rows_par || m >= a.rows) return;
  const long long b = m / a.L, l = m - b * a.L;
  const bool turned = unit < a.turned_units;
  // First channel of this thread's group; half-split: of its first half.
  const int c0 = turned ? 8 * unit : (HALVES ? a.rot + 8 * (unit - a.turned_units) : 8 * unit);
  constexpr int NC = HALVES ? 8 : 4;  // pairs per thread
  float c[NC], s[NC];
  if (turned) {
    const float4* t = reinterpret_cast<const float4*>(a.cs + ((a.cs_per_batch ? m : l) * (a.rot / 2) + NC * unit) * 2);
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) {
      const float4 v = __ldg(t + i);
      c[2 * i] = v.x, s[2 * i] = v.y, c[2 * i + 1] = v.z, s[2 * i + 1] = v.w;
    }
  }
#pragma unroll 4
  for (int hh = h0; hh < a.heads; hh += a.heads_par) {
    int t = 0, h = hh;
#pragma unroll
    for (int i = 0; i + 1 < kRopeTensors; ++i)
      if (t == i && h >= a.t[i].heads) h -= a.t[i].heads, t = i + 1;
    const RopeTensor& T = a.t[t];
    const uint16_t* x = T.x + b * T.x_b + l * T.x_l + h * T.x_h + c0;
    uint16_t* y = T.y + b * T.y_b + l * T.y_l + h * T.y_h + c0;
    uint4 v = *reinterpret_cast<const uint4*>(x);
    if (!turned) {
      *reinterpret_cast<uint4*>(y) = v;
    } else if constexpr (!HALVES) {
      v.x = turn(v.x, c[0], s[0]);
      v.y = turn(v.y, c[1], s[1]);
      v.z = turn(v.z, c[2], s[2]);
      v.w = turn(v.w, c[3], s[3]);
      *reinterpret_cast<uint4*>(y) = v;
    } else {
      uint4 w = *reinterpret_cast<const uint4*>(x + a.rot / 2);
      uint32_t* pv = &v.x;
      uint32_t* pw = &w.x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a0 = lo_f(pv[i]), a1 = hi_f(pv[i]), b0 = lo_f(pw[i]), b1 = hi_f(pw[i]);
        pv[i] = pack2(a0 * c[2 * i] - b0 * s[2 * i], a1 * c[2 * i + 1] - b1 * s[2 * i + 1]);
        pw[i] = pack2(a0 * s[2 * i] + b0 * c[2 * i], a1 * s[2 * i + 1] + b1 * c[2 * i + 1]);
      }
      *reinterpret_cast<uint4*>(y) = v;
      *reinterpret_cast<uint4*>(y + a.rot / 2) = w;
    }
  }
}

}  // namespace

cudaError_t launch_rope_table(const float* ids, long long L, const RopeFreqs& f, float* cs, cudaStream_t stream) {
  const long long rows = (kTableThreads / f.pairs) * kTableRows;
  const long long grid = (L + rows - 1) / rows;
  return launch_pdl(rope_table_kernel, dim3(unsigned(grid)), dim3(kTableThreads), 0, stream, 1, ids, L, f,
                    reinterpret_cast<float2*>(cs));
}

cudaError_t launch_rope(RopeArgs a, bool halves, cudaStream_t stream) {
  a.turned_units = halves ? a.rot / 16 : a.rot / 8;
  a.units = halves ? a.rot / 16 + (a.head_dim - a.rot) / 8 : a.head_dim / 8;
  const int slots = 256 / a.units;
  // As few passes over the heads as the slots allow, each of them full.
  const int passes = (a.heads + slots - 1) / slots;
  a.heads_par = (a.heads + passes - 1) / passes;
  a.rows_par = slots / a.heads_par;
  const long long grid = (a.rows + a.rows_par - 1) / a.rows_par;
  const unsigned threads = unsigned((a.units * a.heads_par * a.rows_par + 31) / 32 * 32);
  return halves ? launch_pdl(rope_kernel<true>, dim3(unsigned(grid)), dim3(threads), 0, stream, 1, a)
                : launch_pdl(rope_kernel<false>, dim3(unsigned(grid)), dim3(threads), 0, stream, 1, a);
}

}  // namespace tern
