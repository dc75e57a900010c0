// rope.cu -- rotary position embedding with several axes (time, height,
// width): the (cos, sin) table of token positions, and the rotation of query
// and key heads by it.
//
// Table: pair j of axis a (d_a channels, d_a / 2 pairs, i = the pair's place
// on its axis) of token m turns by ids[m, a] * theta^(-2 i / d_a).  Far
// positions turn by thousands of radians, where one fp32 ulp of the angle is
// already visible in its cosine, so the angle is counted in quarter turns and
// reduced to [-1/2, 1/2] in 64 bits.  There the sine and cosine are their
// Taylor polynomials (degrees 11 and 12: truncation below 7e-12), rounded
// once to fp32.  A lane owns a token and its warp walks over pairs, so the
// frequency is one constant operand for the warp (a frequency per lane, read
// from the parameters, serialised 32 constant reads: 21 us for 57,677 tokens
// of 64 pairs); the block's 32 rows are turned around in shared memory so
// that stores are consecutive.
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
constexpr int kTableRows = 32;  // token rows per block, one per lane

// cos and sin of x * w quarter turns, each rounded once to fp32 (|x w| < 2^50).
__device__ __forceinline__ float2 cos_sin(double x, double w) {
  // Adding 1.5 * 2^52 leaves the nearest integer n (its low bits count the
  // quarter turns); the remainder x w - n, in [-1/2, 1/2], is rounded once.
  const double magic = 6755399441055744.0;
  const double u = fma(x, w, magic);
  const int q = __double2loint(u);
  const double f = fma(x, w, magic - u);
  const double z = f * f;
  // sin(pi/2 f) / f and cos(pi/2 f): Taylor coefficients (pi/2)^k / k!, alternating.
  constexpr double h = 1.57079632679489661923, h2 = h * h;
  constexpr double s1 = h * h2 / 6, s2 = s1 * h2 / 20, s3 = s2 * h2 / 42, s4 = s3 * h2 / 72, s5 = s4 * h2 / 110;
  constexpr double c1 = h2 / 2, c2 = c1 * h2 / 12, c3 = c2 * h2 / 30, c4 = c3 * h2 / 56, c5 = c4 * h2 / 90,
                   c6 = c5 * h2 / 132;
  const double s = f * fma(z, fma(z, fma(z, fma(z, fma(z, -s5, s4), -s3), s2), -s1), h);
  const double c = fma(z, fma(z, fma(z, fma(z, fma(z, fma(z, c6, -c5), c4), -c3), c2), -c1), 1.0);
  const float fs = float(s), fc = float(c);
  const float cc = (q & 1) ? fs : fc, ss = (q & 1) ? fc : fs;
  // cos changes its sign for quarter turns 1 and 2, sin for 2 and 3.
  return make_float2(__uint_as_float(__float_as_uint(cc) ^ (uint32_t(q + 1) << 30 & 0x80000000u)),
                     __uint_as_float(__float_as_uint(ss) ^ (uint32_t(q) << 30 & 0x80000000u)));
}

__global__ void __launch_bounds__(kTableThreads)
    rope_table_kernel(const float* __restrict__ ids, int L, const __grid_constant__ RopeFreqs f, float2* cs) {
  extern __shared__ float2 tile[];  // [kTableRows][pairs + 1]: a column of lanes meets every bank
  pdl_wait();
  pdl_trigger();
  const int P = f.pairs, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m0 = int(blockIdx.x) * kTableRows, rows = min(kTableRows, L - m0);
  double x[4];  // this lane's token
#pragma unroll
  for (int a = 0; a < 4; ++a) x[a] = a < f.n_axes && lane < rows ? double(ids[(long long)(m0 + lane) * f.n_axes + a]) : 0.0;
  for (int j = warp; j < P; j += kTableThreads / 32) {
    const int axis = f.axis[j];
    tile[lane * (P + 1) + j] = cos_sin(axis == 0 ? x[0] : axis == 1 ? x[1] : axis == 2 ? x[2] : x[3], f.turns[j]);
  }
  __syncthreads();
  float2* out = cs + (long long)m0 * P;
  for (int r = warp; r < rows; r += kTableThreads / 32)
    for (int j = lane; j < P; j += 32) out[r * P + j] = tile[r * (P + 1) + j];
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

cudaError_t launch_rope_table(const float* ids, int L, const RopeFreqs& f, float* cs, cudaStream_t stream) {
  const unsigned grid = unsigned((L + kTableRows - 1) / kTableRows);
  return launch_pdl(rope_table_kernel, dim3(grid), dim3(kTableThreads), kTableRows * (f.pairs + 1) * sizeof(float2), stream,
                    1, ids, L, f, reinterpret_cast<float2*>(cs));
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
